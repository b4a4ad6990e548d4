"""Values of V that are not finite, in prompts: they reach the rows that see their token, in their own dimension,
and no other row, whatever block of keys the token shares with the row's own."""
import numpy as np
import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb
import _tiles as tl

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def poison(c, kv, b, t, h, d, x):
    """V of sequence b, token t, head h: dimension d (None: all) set to x. Over e4m3 a NaN code; an infinity comes
    from the token's scale and needs codes that are not zero."""
    page, slot = int(c["tables"][0][b, t // 64]), t % 64
    if kv == "bf16":
        if d is None:
            c["v_cache"][page, slot, h] = x
        else:
            c["v_cache"][page, slot, h, d] = x
    elif d is None:
        codes = c["v_cache"].view(torch.uint8)[page, slot, h]
        codes[codes & 0x7f == 0] = 1
        codes &= 0x7f
        c["v_scale"][page, h, slot] = x
    else:
        assert x != x
        c["v_cache"].view(torch.uint8)[page, slot, h, d] = 0x7f


def check(c, got, glse, q, new, lens, bad, fp8, what):
    """Every row against 64 bits, but for the dimensions that the poisoned tokens make infinite or NaN in the rows
    that see them: there, what they add is asked for. c holds the values before poisoning."""
    got, at = got.float(), 0
    for b, n in enumerate(new):
        k, v = c["k"][0][b], c["v"][0][b]
        hist = lens[b] - n
        ref = tl.attend(q[at:at + n], k, v, [max(0, min(lens[b], hist + i + 1)) for i in range(n)])
        want = torch.zeros((n, q.shape[1], 128), device="cuda")  # what is added
        for b2, t, h, d, x in bad:
            if b2 == b:
                want[max(0, t - hist):, 8 * h:8 * h + 8, slice(None) if d is None else d] += x
        rows, odd = got[at:at + n], ~torch.isfinite(want)
        assert torch.equal(torch.isnan(rows[odd]), torch.isnan(want[odd])), f"{what} sequence {b}: NaN"
        inf = torch.isinf(want)
        assert torch.equal(rows[inf], want[inf]), f"{what} sequence {b}: infinities"
        tl.check_rows(torch.where(odd, ref[0].float(), rows), glse[at:at + n], ref, fp8, f"{what} sequence {b}")
        at += n


CASES = {
    "one prompt": ([100], [100], [(0, 77, 0, 5, NAN)]),
    "every token late": ([64], [64], [(0, 63, 0, 0, NAN), (0, 63, 1, 127, NAN)]),
    "first token": ([130], [130], [(0, 0, 0, 64, NAN)]),
    "behind a history": ([90, 3], [500, 260], [(0, 411, 0, 1, NAN), (0, 480, 0, 66, NAN), (1, 258, 1, 100, NAN)]),
    "several tiles and blocks": ([300, 40], [300, 300], [(0, 130, 0, 3, NAN), (0, 200, 1, 3, NAN), (0, 299, 0, 90, NAN),
                                                         (1, 262, 0, 0, NAN)]),
    "more new than keys": ([70], [40], [(0, 39, 0, 9, NAN)]),
    "a decode beside": ([1, 50], [200, 50], [(1, 30, 0, 2, NAN)]),
}


@pytest.mark.parametrize("tile", [32, 64])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(CASES))
def test_nan_in_one_dimension(name, kv, tile):
    new, lens, bad = CASES[name]
    c = tl.make_cache([lens], 2, kv, 81)
    q = tl.make_q((sum(new), 16, 128), 82)
    args = (c["tables"][0], tl.i32(tl.starts(new)), tl.i32(lens), c["k_scale"], c["v_scale"])
    for x in bad:
        poison(c, kv, *x)
    for ctas in (None, 3):
        got, glse, plan = hb.prefill(q, c["k_cache"], c["v_cache"], *args, num_ctas=ctas, tile_tokens=tile)
        assert hb.hpc_tile_read_error(plan) == 0
        check(c, got, glse, q, new, lens, bad, kv != "bf16", f"{name}, {ctas} CTAs")


@pytest.mark.parametrize("tile", [32, 64])
def test_infinities(tile):
    """Signs are kept; both signs in one dimension are NaN for the rows that see both; rows of one sequence
    leave the others alone."""
    new, lens = [120, 33], [200, 33]
    bad = [(0, 100, 0, 7, INF), (0, 150, 0, 7, -INF), (0, 199, 1, 8, -INF), (1, 20, 1, 127, INF), (1, 21, 0, None, -INF)]
    c = tl.make_cache([lens], 2, "bf16", 83)
    q = tl.make_q((153, 16, 128), 84)
    for x in bad:
        poison(c, "bf16", *x)
    got, glse, _ = hb.prefill(q, c["k_cache"], c["v_cache"], c["tables"][0], tl.i32([0, 120, 153]), tl.i32(lens), tile_tokens=tile)
    check(c, got, glse, q, new, lens, bad, False, "infinities")


@pytest.mark.parametrize("tile", [32, 64])
def test_scales_out_of_range(tile):
    """A scale that takes code x scale out of f16's range, an infinite and a NaN one: rows before their token
    do not know of them."""
    for x in (INF, NAN, 1e6, -1e6):
        c = tl.make_cache([[100]], 1, "e4m3", 85)
        q = tl.make_q((100, 8, 128), 86)
        poison(c, "e4m3", 0, 70, 0, None, x)
        got, glse, _ = hb.prefill(q, c["k_cache"], c["v_cache"], c["tables"][0], tl.i32([0, 100]), tl.i32([100]), c["k_scale"],
                                  c["v_scale"], tile_tokens=tile)
        ref = tl.attend(q, c["k"][0][0], c["v"][0][0], list(range(1, 101)))
        tl.check_rows(got[:70], glse[:70], tuple(r[:70] for r in ref), True, f"scale {x}")
        if abs(x) != 1e6:
            assert not torch.isfinite(got[70:].float()).any()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_among_many_prompts(kv):
    """Many prompts in one run of work, some with such values: captured and replayed, the same bits every time, and
    rows of tiles that hold none are bit for bit what they are without them."""
    rng = np.random.default_rng(3)
    new = [int(x) for x in rng.integers(1, 90, 40)]
    new[0] = 60
    c = tl.make_cache([new], 2, kv, 87)
    q = tl.make_q((sum(new), 16, 128), 88)
    st = tl.starts(new)
    args = (c["tables"][0], tl.i32(st), tl.i32(new), c["k_scale"], c["v_scale"])
    bad = [(0, 31, 1, 17, NAN), (20, new[20] - 1, 0, 99, NAN)]
    clean = c["v_cache"].clone()
    for x in bad:
        poison(c, kv, *x)
    for tile in (32, 64):
        out, _, _ = hb.prefill(q, c["k_cache"], clean, *args, num_ctas=4, tile_tokens=tile)
        got, glse = torch.empty_like(out), torch.empty((sum(new), 16), device="cuda")
        ws = torch.empty(hb.prefill_workspace_bytes(40, 4), dtype=torch.uint8, device="cuda")

        def call():
            hb.prefill(q, c["k_cache"], c["v_cache"], *args, num_ctas=4, tile_tokens=tile, out=got, out_lse=glse, workspace=ws)
        call()
        torch.cuda.synchronize()
        first = got.clone()
        check(c, got, glse, q, new, new, bad, kv != "bf16", "many prompts")
        for b in set(range(40)) - {0, 20}:
            assert torch.equal(got[st[b]:st[b + 1]], out[st[b]:st[b + 1]])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        for _ in range(3):
            got.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(got.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("tile", [32, 64])
def test_not_finite_for_other_reasons(tile):
    """NaN queries beside values of V that are not finite: their own rows are NaN, the others right."""
    c = tl.make_cache([[150]], 1, "bf16", 89)
    q = tl.make_q((100, 8, 128), 90)
    poison(c, "bf16", 0, 120, 0, 50, NAN)
    q[10, 3] = NAN
    got, glse, _ = hb.prefill(q, c["k_cache"], c["v_cache"], c["tables"][0], tl.i32([0, 100]), tl.i32([150]), tile_tokens=tile)
    assert torch.isnan(got[10, 3].float()).all()
    q[10, 3], got[10, 3] = 0.0, 0.0
    ref = tl.attend(q, c["k"][0][0], c["v"][0][0], [51 + i for i in range(100)])
    got[10, 3], glse[10, 3] = ref[0][10, 3].bfloat16(), ref[1][10, 3].float()
    tl.check_rows(got[:70], glse[:70], tuple(r[:70] for r in ref), False, "before the token")
    assert torch.isnan(got[70:, :, 50].float()).all() and torch.isfinite(got[70:, :, :50].float()).all()
