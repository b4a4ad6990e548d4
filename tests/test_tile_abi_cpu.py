"""Refusals of the prompt, shared-prefix and cache calls, on the host (fake pointers, never
dereferenced), and their size functions."""
import ctypes

import pytest

from load_balanced_paged_02_gb300 import _build
from load_balanced_paged_02_gb300 import binding as hb

FAKE = 0x10000
ODD = 0x10004
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    _build.build()
    return hb.lib()


def tile_plan(mode=0, seqs=2, tokens=10, heads=1, workers=4, tile=32, q_len=1, stride=4, buf=FAKE, nbytes=1 << 20):
    return hb.TilePlanStruct(buf, nbytes, seqs, tokens, heads, workers, mode, tile, q_len, stride)


def test_sizes(L):
    assert L.hpc_tile_plan_bytes(1, 1) == 4 * (16 + 2 * 8 + 4 + 4)
    assert L.hpc_tile_plan_bytes(7, 152) == 4 * (16 + 153 * 8 + 7 * 4 + 8 * 2)
    for bad in ((0, 1), (16385, 1), (1, 0), (1, 4097), (-1, 5)):
        assert L.hpc_tile_plan_bytes(*bad) == 0
    assert L.hpc_prefill_split_rows(152) == 2 * 152 * 256
    assert L.hpc_prefill_split_rows(0) == 0 and L.hpc_prefill_split_rows(4097) == 0
    assert L.hpc_prefix_split_rows(1, 64, 1, 8, 152) == ((64 // 32 + 2) * 8 + 152) * 256
    for bad in ((0, 1, 1, 1, 1), (1, 0, 1, 1, 1), (1, 1, 0, 1, 1), (1, 1, 9, 1, 1), (1, 1, 1, 0, 1), (1, 1, 1, 257, 1), (1, 1, 1, 1, 0)):
        assert L.hpc_prefix_split_rows(*bad) == 0
    assert L.hpc_prefill_workspace_bytes(4, 152) >= L.hpc_tile_plan_bytes(4, 152) + L.hpc_prefill_split_rows(152) * 516
    assert L.hpc_prefill_workspace_bytes(0, 152) == 0
    need = L.hpc_decode_shared_prefix_workspace_bytes(2, 64, 1, 8, 152, 152)
    assert need >= L.hpc_prefix_split_rows(2, 64, 1, 8, 152) * 516 + L.hpc_decode_split_capacity(64, 8, 152) * 8 * 516
    for bad in ((0, 1, 1, 1, 1, 1), (1, 0, 1, 1, 1, 1), (1, 1, 9, 1, 1, 1), (1, 1, 1, 300, 1, 1), (1, 1, 1, 1, 5000, 1), (1, 1, 1, 1, 1, 0)):
        assert L.hpc_decode_shared_prefix_workspace_bytes(*bad) == 0


def test_plan_refusals(L):
    def prefill(qs=FAKE, sl=FAKE, B=2, T=10, H=1, stride=4, C=4, m=1, tt=0, plan="new", nbytes=1 << 20, buf=FAKE):
        p = hb.TilePlanStruct(buf, nbytes, 0, 0, 0, 0, 0, 0, 0, 0) if plan == "new" else None
        return L.hpc_prefill_plan(qs, sl, B, T, H, stride, C, m, tt, None if p is None else ctypes.byref(p), None)
    assert prefill(qs=None) == INVALID and prefill(sl=None) == INVALID and prefill(plan=None) == INVALID
    assert prefill(buf=None) == INVALID and prefill(buf=ODD) == INVALID
    assert prefill(B=0) == INVALID and prefill(B=16385) == INVALID and prefill(T=-1) == INVALID
    assert prefill(H=0) == INVALID and prefill(H=257) == INVALID and prefill(stride=0) == INVALID
    assert prefill(C=0) == INVALID and prefill(C=4097) == INVALID and prefill(m=-1) == INVALID
    assert prefill(tt=16) == INVALID and prefill(tt=128) == INVALID
    assert prefill(T=2147483647, H=256) == INVALID  # tile numbers past int32
    assert prefill(nbytes=64) == SMALL

    def prefix(gs=FAKE, pl=FAKE, G=1, B=4, q=1, H=1, stride=4, C=4, m=1, tt=0, nbytes=1 << 20):
        p = hb.TilePlanStruct(FAKE, nbytes, 0, 0, 0, 0, 0, 0, 0, 0)
        return L.hpc_prefix_plan(gs, pl, G, B, q, H, stride, C, m, tt, ctypes.byref(p), None)
    assert prefix(gs=None) == INVALID and prefix(pl=None) == INVALID and prefix(G=0) == INVALID
    assert prefix(B=0) == INVALID and prefix(B=16385) == INVALID and prefix(q=0) == INVALID and prefix(q=9) == INVALID
    assert prefix(nbytes=8) == SMALL


def attn(L, fn, plan, q=FAKE, k=FAKE, v=FAKE, ks=None, vs=None, dt=0, pages=16, pt=FAKE, stride=4, Hq=8, Hkv=1, D=128,
         P=64, so=FAKE, sl=FAKE, out=FAKE):
    ref = None if plan is None else ctypes.byref(plan)
    if fn == "prefill":
        return L.hpc_prefill_attn(q, k, v, ks, vs, dt, pages, pt, stride, Hq, Hkv, D, P, ref, so, sl, out, None, None)
    return L.hpc_prefix_attn(q, k, v, ks, vs, dt, pages, pt, stride, Hq, Hkv, D, P, ref, so, sl, None)


@pytest.mark.parametrize("fn", ["prefill", "prefix"])
def test_attn_refusals(L, fn):
    mode = 0 if fn == "prefill" else 1
    good = tile_plan(mode)
    assert attn(L, fn, good, D=64) == UNSUPPORTED and attn(L, fn, good, P=16) == UNSUPPORTED
    assert attn(L, fn, good, Hq=4) == UNSUPPORTED and attn(L, fn, good, dt=2) == UNSUPPORTED
    assert attn(L, fn, good, Hkv=0) == INVALID and attn(L, fn, good, Hkv=257, Hq=2056) == INVALID
    for name in ("q", "k", "v", "pt", "so", "sl"):
        assert attn(L, fn, good, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "so"):
        assert attn(L, fn, good, **{name: ODD}) == INVALID, name
    assert attn(L, fn, good, dt=1) == INVALID                       # e4m3 without scales
    assert attn(L, fn, good, dt=1, ks=FAKE, vs=ODD) == INVALID
    assert attn(L, fn, good, pages=0) == INVALID
    assert attn(L, fn, good, pages=2147483647 // 64) == INVALID     # the page after the last must have a coordinate
    assert attn(L, fn, good, stride=5) == INVALID                   # another table than the plan's
    assert attn(L, fn, None) == INVALID
    assert attn(L, fn, tile_plan(1 - mode)) == INVALID              # the other kind of map
    assert attn(L, fn, tile_plan(mode, heads=2)) == INVALID
    assert attn(L, fn, tile_plan(mode, nbytes=16)) == INVALID
    assert attn(L, fn, tile_plan(mode, tile=48)) == INVALID
    assert attn(L, fn, tile_plan(mode, workers=0)) == INVALID
    if fn == "prefill":
        assert attn(L, fn, good, out=None) == INVALID and attn(L, fn, good, out=ODD) == INVALID
        assert attn(L, fn, tile_plan(mode, tokens=0)) == OK         # nothing to enqueue
        assert attn(L, fn, tile_plan(mode, tokens=0), q=None, out=None) == OK


def test_combine_refusals(L):
    p = tile_plan(0)
    args = dict(so=FAKE, sl=FAKE, out=FAKE, Hq=8, Hkv=1, D=128)

    def call(plan=p, **kw):
        a = dict(args, **kw)
        return L.hpc_prefill_combine(ctypes.byref(plan), a["so"], a["sl"], a["out"], None, a["Hq"], a["Hkv"], a["D"], None)
    assert call(D=64) == UNSUPPORTED and call(so=None) == INVALID and call(sl=None) == INVALID
    assert call(out=None) == INVALID and call(out=ODD) == INVALID and call(plan=tile_plan(1)) == INVALID
    assert call(plan=tile_plan(0, tokens=0)) == OK

    pre, own = tile_plan(1, tokens=4, q_len=2), hb.PlanStruct(FAKE, 1 << 20, 2, 1, 4, 2, 0, 10)

    def prefix(plan=own, pplan=pre, po=FAKE, pl=FAKE, so=FAKE, sl=FAKE, out=FAKE, B=2, q=2, Hq=8, Hkv=1, D=128):
        return L.hpc_prefix_combine(ctypes.byref(pplan), po, pl, ctypes.byref(plan), so, sl, out, None, B, q, Hq, Hkv, D, None)
    assert prefix(D=32) == UNSUPPORTED and prefix(B=3) == INVALID and prefix(q=1) == INVALID and prefix(q=9) == INVALID
    for name in ("po", "pl", "so", "sl", "out"):
        assert prefix(**{name: None}) == INVALID, name
    assert prefix(po=ODD) == INVALID and prefix(so=ODD) == INVALID
    assert prefix(plan=hb.PlanStruct(FAKE, 1 << 20, 3, 1, 4, 2, 0, 10)) == INVALID
    assert prefix(plan=hb.PlanStruct(FAKE, 8, 2, 1, 4, 2, 0, 10)) == INVALID
    assert prefix(pplan=tile_plan(0, tokens=4)) == INVALID


def test_one_call_refusals(L):
    p = hb.TilePlanStruct()
    need = L.hpc_prefill_workspace_bytes(2, 4)

    def prefill(q=FAKE, k=FAKE, dt=0, pt=FAKE, stride=4, qs=FAKE, sl=FAKE, B=2, T=10, Hq=8, Hkv=1, D=128, C=4, tt=0,
                ws=FAKE, nbytes=need, plan=p, out=FAKE):
        return L.hpc_prefill(q, k, FAKE, None, None, dt, 16, pt, stride, qs, sl, B, T, Hq, Hkv, D, 64, C, 1, tt, ws, nbytes,
                             None if plan is None else ctypes.byref(plan), out, None, None)
    assert prefill(nbytes=need - 1) == SMALL
    assert prefill(ws=None) == INVALID and prefill(ws=0x10010) == INVALID and prefill(plan=None) == INVALID
    for name in ("q", "k", "pt", "qs", "sl", "out"):
        assert prefill(**{name: None}) == INVALID, name
    assert prefill(B=0) == INVALID and prefill(C=0) == INVALID and prefill(D=96) == UNSUPPORTED
    assert prefill(dt=1) == INVALID and prefill(dt=3) == UNSUPPORTED and prefill(stride=0) == INVALID and prefill(tt=1) == INVALID

    own = hb.PlanStruct()
    need2 = L.hpc_decode_shared_prefix_workspace_bytes(1, 2, 1, 1, 4, 4)

    def shared(q=FAKE, k=FAKE, dt=0, pt=FAKE, sl=FAKE, ptab=FAKE, pl=FAKE, gs=FAKE, G=1, B=2, ql=1, Hq=8, Hkv=1, D=128, C=4,
               m=2, PC=4, ws=FAKE, nbytes=need2, out=FAKE):
        return L.hpc_decode_shared_prefix(q, k, FAKE, None, None, dt, 16, pt, 4, sl, ptab, 4, pl, gs, G, B, ql, Hq, Hkv, D, 64,
                                          C, m, PC, 1, 0, ws, nbytes, ctypes.byref(p), ctypes.byref(own), out, None, None)
    assert shared(nbytes=need2 - 1) == SMALL
    for name in ("q", "k", "pt", "sl", "ptab", "pl", "gs", "out", "ws"):
        assert shared(**{name: None}) == INVALID, name
    assert shared(G=0) == INVALID and shared(B=0) == INVALID and shared(ql=9) == INVALID and shared(m=-1) == INVALID
    assert shared(Hq=16) == UNSUPPORTED and shared(D=64) == UNSUPPORTED and shared(dt=1) == INVALID and shared(PC=0) == INVALID


def test_cache_refusals(L):
    def write(k=FAKE, v=FAKE, ks=128, vs=128, slots=FAKE, T=3, H=1, D=128, P=64, kc=FAKE, vc=FAKE, kss=None, vss=None, dt=0,
              pages=4):
        return L.hpc_kv_write(k, v, ks, vs, slots, T, H, D, P, kc, vc, kss, vss, dt, pages, None, None)
    assert write(T=0) == OK and write(T=0, k=None, v=None, slots=None) == OK and write(T=-1) == INVALID and write(D=64) == UNSUPPORTED and write(P=32) == UNSUPPORTED
    assert write(ks=120) == INVALID and write(vs=132) == INVALID and write(H=2, ks=128) == INVALID and write(ks=-128) == INVALID
    for name in ("k", "v", "slots", "kc", "vc"):
        assert write(**{name: None}) == INVALID, name
    assert write(k=ODD) == INVALID and write(v=ODD) == INVALID and write(kc=ODD) == INVALID
    assert write(dt=1) == INVALID and write(dt=5) == UNSUPPORTED and write(pages=0) == INVALID and write(H=300) == INVALID

    def read(kc=FAKE, vc=FAKE, kss=None, vss=None, dt=0, pages=4, pt=FAKE, stride=2, starts=FAKE, B=1, rows=3, H=1, D=128,
             P=64, ko=FAKE, vo=FAKE):
        return L.hpc_kv_read(kc, vc, kss, vss, dt, pages, pt, stride, None, starts, B, rows, H, D, P, ko, vo, None, None)
    assert read(rows=0) == OK and read(rows=0, ko=None, vo=None) == OK and read(rows=-1) == INVALID and read(D=64) == UNSUPPORTED and read(P=32) == UNSUPPORTED
    for name in ("kc", "vc", "pt", "starts", "ko", "vo"):
        assert read(**{name: None}) == INVALID, name
    assert read(ko=ODD) == INVALID and read(stride=0) == INVALID and read(B=0) == INVALID and read(dt=1) == INVALID


def test_read_error_refuses_null(L):
    w = ctypes.c_int(0)
    assert L.hpc_tile_read_error(None, ctypes.byref(w)) == INVALID
    assert L.hpc_tile_read_error(ctypes.byref(tile_plan()), None) == INVALID
