"""decode_shared_prefix beside the calls that it is made of: its plans handed on to them, its outputs given to it."""
import numpy as np
import pytest
import torch

import oracle
from load_balanced_paged_02_gb300 import binding as hb
import _tiles as tl

pytestmark = pytest.mark.gpu

OWN, PREFIXES, GROUPS = [20, 64, 0, 130, 5, 200], [300, 70], [0, 4, 6]


def case(kv, q_len, seed, hkv=2):
    c = tl.make_cache([OWN, PREFIXES], hkv, kv, seed)
    q = tl.make_q((6, 8 * hkv, 128) if q_len == 1 else (6, q_len, 8 * hkv, 128), seed)
    return c, (q, c["k_cache"], c["v_cache"], c["tables"][0], tl.i32(OWN), c["tables"][1], tl.i32(PREFIXES), tl.i32(GROUPS),
               c["k_scale"], c["v_scale"])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [1, 3])
def test_its_plans_serve_the_single_calls(q_len, kv):
    """The next layer runs on the maps of the one before, with buffers of its own."""
    c, args = case(kv, q_len, 61)
    q = args[0]
    out, lse, pplan, plan = hb.decode_shared_prefix(*args)
    assert np.array_equal(plan.buf.cpu().numpy(), oracle.plan(np.asarray(OWN, np.int32), 2, plan.num_ctas, 2))
    po, pl = hb.prefix_split_buffers(pplan)
    so, sl = hb.split_buffers(plan, q_len=q_len)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    hb.hpc_prefix_attn(q, c["k_cache"], c["v_cache"], args[5], pplan, po, pl, c["k_scale"], c["v_scale"])
    hb.hpc_decode_attn(q, c["k_cache"], c["v_cache"], args[3], args[4], plan, so, sl, c["k_scale"], c["v_scale"])
    hb.hpc_prefix_combine(pplan, po, pl, plan, so, sl, o2, l2)
    assert hb.hpc_decode_read_error(plan) == 0 and hb.hpc_tile_read_error(pplan) == 0
    # (hpc_decode_attn runs one token on the kernel that hpc_decode_attn_multi runs it on)
    assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("q_len", [1, 2])
def test_outputs_that_are_given(q_len):
    c, args = case("bf16", q_len, 71)
    out, lse, _, _ = hb.decode_shared_prefix(*args)
    ws = torch.empty(hb.decode_shared_prefix_workspace_bytes(2, 6, 2, q_len), dtype=torch.uint8, device="cuda")
    o2, l2 = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    got = hb.decode_shared_prefix(*args, workspace=ws, out=o2, out_lse=l2)
    assert got[0] is o2 and got[1] is l2 and torch.equal(o2, out) and torch.equal(l2, lse)
    for kw in (dict(out=o2.float()), dict(out=o2[:5]), dict(out_lse=l2[..., :8]), dict(out_lse=l2.double()), dict(out=o2.cpu())):
        with pytest.raises(hb.HpcError):
            hb.decode_shared_prefix(*args, workspace=ws, **kw)
