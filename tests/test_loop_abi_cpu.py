"""Refusals of the calls between two attention steps, on the host (fake pointers, never dereferenced)."""
import pytest

from load_balanced_paged_02_gb300 import _build
from load_balanced_paged_02_gb300 import binding as hb

FAKE, OTHER = 0x10000, 0x20000
ODD = 0x10004
OK, INVALID, UNSUPPORTED = 0, 1, 2
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return hb.lib()


def test_attn_weights_refusals(L):
    def call(q=FAKE, k=FAKE, ks=None, dt=0, pages=16, pt=FAKE, stride=4, qs=FAKE, sl=FAKE, rc=None, win=0, lse=FAKE, B=2, T=10, Hq=8,
             Hkv=1, D=128, P=64, decay=1.0, w=FAKE, ws=256):
        return L.hpc_attn_weights(q, k, ks, dt, pages, pt, stride, qs, sl, rc, win, lse, B, T, Hq, Hkv, D, P, decay, w, ws, None, None)
    assert call(D=64) == UNSUPPORTED and call(P=16) == UNSUPPORTED and call(Hq=4) == UNSUPPORTED and call(dt=2) == UNSUPPORTED
    for name in ("q", "k", "pt", "sl", "lse", "w"):
        assert call(**{name: None}) == INVALID, name
    assert call(q=ODD) == INVALID and call(k=ODD) == INVALID
    assert call(dt=1) == INVALID and call(dt=1, ks=ODD) == INVALID                  # e4m3 without scales
    assert call(pages=0) == INVALID and call(pages=2147483647 // 64) == INVALID
    assert call(stride=0) == INVALID and call(win=-1) == INVALID and call(T=-1) == INVALID
    assert call(B=0) == INVALID and call(B=16385) == INVALID
    assert call(Hkv=0) == INVALID and call(Hkv=257, Hq=2056) == INVALID and call(Hq=0) == INVALID
    assert call(decay=-0.5) == INVALID and call(decay=1.5) == INVALID and call(decay=NAN) == INVALID
    assert call(ws=255) == INVALID                                                  # shorter than the table's row
    assert call(qs=None, T=11) == INVALID                                           # not as many rows for each
    assert call(T=0, q=None, lse=None) == OK                                        # nothing to enqueue


def test_kv_select_refusals(L):
    def call(w=FAKE, ws=256, sl=FAKE, B=2, H=1, n=64, first=4, recent=8, keep=FAKE, kl=FAKE):
        return L.hpc_kv_select(w, ws, sl, B, H, n, first, recent, keep, kl, None, None)
    for name in ("w", "sl", "keep", "kl"):
        assert call(**{name: None}) == INVALID, name
    assert call(B=0) == INVALID and call(B=16385) == INVALID and call(H=0) == INVALID and call(H=257) == INVALID
    assert call(ws=0) == INVALID and call(ws=(1 << 30) + 1) == INVALID and call(n=0) == INVALID
    assert call(first=-1) == INVALID and call(recent=-1) == INVALID
    assert call(first=60, recent=5) == INVALID and call(first=2147483647, recent=2147483647) == INVALID


def test_kv_compact_refusals(L):
    def call(k=FAKE, v=FAKE, ks=None, vs=None, dt=0, pages=16, pt=FAKE, stride=4, keep=FAKE, n=64, kl=FAKE, nt=FAKE, ns=1, B=2, H=1, D=128,
             P=64, w=None, ws=0, nw=None, nws=0):
        return L.hpc_kv_compact(k, v, ks, vs, dt, pages, pt, stride, keep, n, kl, nt, ns, B, H, D, P, w, ws, nw, nws, None, None)
    assert call(D=64) == UNSUPPORTED and call(P=16) == UNSUPPORTED and call(dt=2) == UNSUPPORTED
    for name in ("k", "v", "pt", "keep", "kl", "nt"):
        assert call(**{name: None}) == INVALID, name
    assert call(k=ODD) == INVALID and call(v=ODD) == INVALID and call(dt=1) == INVALID and call(dt=1, ks=FAKE) == INVALID
    assert call(stride=0) == INVALID and call(n=0) == INVALID and call(ns=0) == INVALID and call(pages=0) == INVALID
    assert call(B=0) == INVALID and call(H=0) == INVALID and call(B=16385) == INVALID and call(H=257) == INVALID
    assert call(w=FAKE, ws=256) == INVALID and call(nw=FAKE, nws=64) == INVALID     # one without the other
    assert call(w=FAKE, ws=256, nw=FAKE, nws=64) == INVALID                         # onto itself
    assert call(w=FAKE, ws=255, nw=OTHER, nws=64) == INVALID
    assert call(w=FAKE, ws=256, nw=OTHER, nws=63) == INVALID


def test_verify_refusals(L):
    def call(p=FAKE, ps=100, q=FAKE, qs=100, dt=0, d=FAKE, c=None, u=FAKE, us=FAKE, B=2, n=3, V=100, acc=FAKE, tok=FAKE, sl=None, kl=None):
        return L.hpc_verify_drafts(p, ps, q, qs, dt, d, c, u, us, B, n, V, acc, tok, sl, kl, None, None)
    for name in ("p", "d", "u", "us", "acc", "tok"):
        assert call(**{name: None}) == INVALID, name
    assert call(dt=2) == UNSUPPORTED and call(B=0) == INVALID and call(B=16385) == INVALID
    assert call(n=-1) == INVALID and call(n=32) == INVALID and call(V=0) == INVALID
    assert call(ps=99) == INVALID and call(qs=99) == INVALID and call(p=0x10002) == INVALID and call(q=0x10001, dt=1) == INVALID
    assert call(kl=FAKE) == INVALID                                                 # new lengths of no lengths


def test_sizes_that_leave_32_bits(L):
    def weights(stride, ws):
        return L.hpc_attn_weights(FAKE, FAKE, None, 0, 16, FAKE, stride, FAKE, FAKE, None, 0, FAKE, 2, 10, 8, 1, 128, 64, 1.0, FAKE, ws, None,
                                  None)
    assert weights((1 << 24) + 1, ((1 << 24) + 1) * 64) == INVALID and weights(2147483647, 2147483647 * 64) == INVALID
    for n in ((1 << 30) + 1, 2147483647):
        assert L.hpc_kv_select(FAKE, 256, OTHER, 2, 1, n, 4, 8, FAKE, FAKE, None, None) == INVALID
        assert L.hpc_kv_compact(FAKE, FAKE, None, None, 0, 16, FAKE, 4, FAKE, n, FAKE, FAKE, 1, 2, 1, 128, 64, None, 0, None, 0, None,
                                None) == INVALID


def test_outputs_that_other_blocks_still_read(L):
    assert L.hpc_kv_select(FAKE, 256, OTHER, 2, 1, 64, 4, 8, FAKE, OTHER, None, None) == INVALID    # lengths in place
    assert L.hpc_verify_drafts(FAKE, 100, FAKE, 100, 0, FAKE, OTHER, FAKE, FAKE, 2, 3, 100, OTHER, FAKE, None, None, None, None) == INVALID
