"""Maps on another device than the call's tensors (here: in host memory) are refused before any launch."""
import types

import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb
import _tiles as tl

pytestmark = pytest.mark.gpu


def on_host(plan):
    """The plan with its map on the host: the checks have to find it, the struct still names device memory."""
    names = ("struct", "ref", "num_ctas", "split_capacity")
    return types.SimpleNamespace(buf=plan.buf.cpu(), **{n: getattr(plan, n) for n in names if hasattr(plan, n)})


def test_maps_elsewhere():
    c = tl.make_cache([[9, 20], [70]], 1, "bf16", 51)
    q = tl.make_q((2, 8, 128), 52)
    st, lens, own = tl.i32([0, 1, 2]), tl.i32([9, 20]), tl.i32([9, 20])
    table, ptable = c["tables"]
    plan = hb.hpc_prefill_plan(st, lens, 2, 1, table.shape[1])
    pplan = hb.hpc_prefix_plan(tl.i32([0, 2]), tl.i32([70]), 2, 1, ptable.shape[1])
    dplan = hb.hpc_decode_plan(own, 1)
    so, sl = hb.prefill_split_buffers(plan)
    po, pl = hb.prefix_split_buffers(pplan)
    do, dl = hb.split_buffers(dplan)
    out = torch.empty_like(q)
    calls = [lambda: hb.hpc_prefill_plan(st, lens, 2, 1, table.shape[1], plan=on_host(plan)),
             lambda: hb.hpc_prefix_plan(tl.i32([0, 2]), tl.i32([70]), 2, 1, ptable.shape[1], plan=on_host(pplan)),
             lambda: hb.hpc_prefill_attn(q, c["k_cache"], c["v_cache"], table, on_host(plan), so, sl, out),
             lambda: hb.hpc_prefill_combine(on_host(plan), so, sl, out),
             lambda: hb.hpc_prefix_attn(q, c["k_cache"], c["v_cache"], ptable, on_host(pplan), po, pl),
             lambda: hb.hpc_prefix_combine(on_host(pplan), po, pl, dplan, do, dl, out),
             lambda: hb.hpc_prefix_combine(pplan, po, pl, on_host(dplan), do, dl, out)]
    for i, call in enumerate(calls):
        with pytest.raises(hb.HpcError, match="tensors on"):
            call()
            pytest.fail(f"call {i} took a map in host memory")
