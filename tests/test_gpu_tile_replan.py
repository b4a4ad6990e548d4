"""Maps planned again into a plan's buffer with the sizes that the old plan's header has: other new tokens per
request, and a wider page table."""
import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb
import _tiles as tl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("tile", [32, 64])
def test_a_wider_table(tile, kv):
    """The old plan's table has two columns, the map in its buffer keys of eight: page ids are read from the
    table's rows alone, and the keys beyond them are not seen."""
    new, lens, wide = [30, 9], [120, 100], [500, 400]
    c = tl.make_cache([lens, [64]], 1, kv, 31)
    other = int(c["tables"][1][0, 0])
    # behind the table, ids of a page whose keys must not be seen
    behind = torch.full((2 * 2 + 64,), other, dtype=torch.int32, device="cuda")
    behind[:4] = c["tables"][0][:, :2].reshape(-1)
    table = behind[:4].view(2, 2)
    q = tl.make_q((39, 8, 128), 32)
    plan = hb.hpc_prefill_plan(tl.i32([0, 30, 39]), tl.i32(lens), 39, 1, 2, num_ctas=6, tile_tokens=tile)
    old = hb.TilePlanStruct.from_buffer_copy(plan.struct)
    hb.hpc_prefill_plan(tl.i32([0, 30, 39]), tl.i32(wide), 39, 1, 8, num_ctas=6, tile_tokens=tile, plan=plan)
    plan.struct = old
    so, sl = hb.prefill_split_buffers(plan)
    out, lse = torch.empty_like(q), torch.empty((39, 8), device="cuda")
    hb.hpc_prefill_attn(q, c["k_cache"], c["v_cache"], table, plan, so, sl, out, lse, c["k_scale"], c["v_scale"])
    hb.hpc_prefill_combine(plan, so, sl, out, lse)
    assert hb.hpc_tile_read_error(plan) == 4  # HPC_DEVERR_PAGE_OUT_OF_RANGE
    # slots 120..127 and 100..127 hold NaN in this cache: rows see them by the wider map, so only
    # the sums of whole tokens can be looked at: fill them first
    for b, n in enumerate(lens):
        page, at = int(table[b, 1]), n % 64
        for name in "kv":
            x = torch.randn((64 - at, 1, 128), device="cuda")
            if kv == "bf16":
                c[name + "_cache"][page, at:] = x.bfloat16()
                val = c[name + "_cache"][page, at:].double()
            else:
                c[name + "_cache"].view(torch.uint8)[page, at:] = (x * 60).to(torch.float8_e4m3fn).view(torch.uint8)
                c[name + "_scale"][page, :, at:] = 1 / 64
                val = c[name + "_cache"].view(torch.uint8)[page, at:].view(torch.float8_e4m3fn).double() / 64
            c[name][0][b] = torch.cat([c[name][0][b], val])
    hb.hpc_prefill_attn(q, c["k_cache"], c["v_cache"], table, plan, so, sl, out, lse, c["k_scale"], c["v_scale"])
    hb.hpc_prefill_combine(plan, so, sl, out, lse)
    at = 0
    for b, n in enumerate(new):
        ref = tl.attend(q[at:at + n], c["k"][0][b], c["v"][0][b], [128] * n)
        tl.check_rows(out[at:at + n], lse[at:at + n], ref, kv != "bf16", f"sequence {b}")
        at += n


@pytest.mark.parametrize("tile", [32, 64])
def test_other_new_tokens_per_request(tile):
    """Eight requests of one token and four of two have the same rows: the map says which it is of."""
    c = tl.make_cache([[200, 70]], 1, "bf16", 41)
    q = tl.make_q((8, 8, 128), 42)
    plan = hb.hpc_prefix_plan(tl.i32([0, 5, 8]), tl.i32([200, 70]), 8, 1, 4, num_ctas=8, tile_tokens=tile)
    old = hb.TilePlanStruct.from_buffer_copy(plan.struct)
    hb.hpc_prefix_plan(tl.i32([0, 1, 4]), tl.i32([200, 70]), 4, 1, 4, q_len=2, num_ctas=8, tile_tokens=tile, plan=plan)
    plan.struct = old
    po, pl = hb.prefix_split_buffers(plan)
    po.fill_(7.0), pl.fill_(7.0)
    hb.hpc_prefix_attn(q, c["k_cache"], c["v_cache"], c["tables"][0], plan, po, pl)
    assert hb.hpc_tile_read_error(plan) & 16 and bool((po == 7).all())
    own = torch.zeros(8, dtype=torch.int32, device="cuda")
    dplan = hb.hpc_decode_plan(own, 1)
    so, sl = hb.split_buffers(dplan)
    out, lse = torch.empty_like(q), torch.empty((8, 8), device="cuda")
    hb.hpc_prefix_combine(plan, po, pl, dplan, so, sl, out, lse)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
