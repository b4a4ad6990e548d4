"""Outputs of the calls between two attention steps that overlap what other blocks read or write: refused on the host
(fake pointers, never dereferenced; every call here is refused)."""
import pytest

from load_balanced_paged_02_gb300 import _build
from load_balanced_paged_02_gb300 import binding as hb

INVALID, UNSUPPORTED = 1, 2
P, Q, D, U, US, ACC, TOK, CNT, LEN, KEPT = (0x100000 * (i + 1) for i in range(10))


@pytest.fixture(scope="module")
def L():
    _build.build()
    return hb.lib()


def verify(L, p=P, ps=100, q=Q, qs=100, dt=0, d=D, c=CNT, u=U, us=US, B=2, n=3, V=100, acc=ACC, tok=TOK, sl=LEN, kl=KEPT):
    return L.hpc_verify_drafts(p, ps, q, qs, dt, d, c, u, us, B, n, V, acc, tok, sl, kl, None, None)


def test_verify(L):
    # arrays of 2 (counts, lengths, accepted), 6 (drafts) and 8 (tokens) numbers
    for other, words in ((D, 6), (CNT, 2), (LEN, 2), (TOK, 8)):
        for step in (0, 4, 4 * (words - 1), -4):
            assert verify(L, acc=other + step) == INVALID, (other, step)
            if other != LEN or step:
                assert verify(L, kl=other + step) == INVALID, (other, step)
    for other, words in ((D, 6), (CNT, 2), (LEN, 2)):
        for step in (0, 4, 4 * (words - 1), -4, -28):
            assert verify(L, tok=other + step) == INVALID, (other, step)
    assert verify(L, acc=KEPT) == INVALID and verify(L, acc=KEPT + 4) == INVALID
    # one request: its drafts' own place, and no other over them
    for step in (4, -4, 8, -12):
        assert verify(L, B=1, tok=D + step) == INVALID
    # the same lengths in place beside another fault
    assert verify(L, kl=LEN, V=0) == INVALID and verify(L, kl=LEN, sl=None) == INVALID


def test_select(L):
    def call(sl=LEN, keep=TOK, kl=KEPT, B=2, H=3, n=10, w=P, first=1, recent=2):
        return L.hpc_kv_select(w, 256, sl, B, H, n, first, recent, keep, kl, None, None)
    for step in (0, 4, -4):
        assert call(kl=LEN + step) == INVALID
    for step in (0, 4, 59 * 4, -4):
        assert call(sl=TOK + step) == INVALID and call(kl=TOK + step) == INVALID
    assert call(B=1, kl=LEN) == INVALID


def test_other_refusals_with_arrays_apart(L):
    for name in ("p", "d", "u", "us", "acc", "tok"):
        assert verify(L, **{name: None}) == INVALID, name
    assert verify(L, dt=2) == UNSUPPORTED and verify(L, B=0) == INVALID and verify(L, B=16385) == INVALID
    assert verify(L, n=-1) == INVALID and verify(L, n=32) == INVALID and verify(L, V=0) == INVALID
    assert verify(L, ps=99) == INVALID and verify(L, qs=99) == INVALID and verify(L, p=P + 2) == INVALID and verify(L, q=Q + 1, dt=1) == INVALID
