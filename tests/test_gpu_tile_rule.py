"""The tile size that the calls choose: by the average of query tokens per sequence, by cache type in prefill."""
import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb
import _tiles as tl

pytestmark = pytest.mark.gpu


def chosen(kv, new):
    c = tl.make_cache([new], 1, kv, 1)
    q = tl.make_q((sum(new), 8, 128), 2)
    return hb.prefill(q, c["k_cache"], c["v_cache"], c["tables"][0], tl.i32(tl.starts(new)), tl.i32(new), c["k_scale"],
                      c["v_scale"])[2].tile_tokens


def test_prompts():
    assert [chosen("bf16", [n, n]) for n in (63, 64, 96, 97)] == [32, 64, 64, 64]
    assert [chosen("e4m3", [n, n]) for n in (63, 64, 96, 97)] == [32, 32, 32, 64]
    assert chosen("bf16", [127, 0]) == 32 and chosen("bf16", [128, 0]) == 64
    plan = hb.hpc_prefill_plan(tl.i32([0, 64]), tl.i32([64]), 64, 1, 1)
    assert plan.tile_tokens == 64


def test_prefixes():
    got = [hb.hpc_prefix_plan(tl.i32([0, n]), tl.i32([64]), n, 1, 1).tile_tokens for n in (64, 96, 97, 200)]
    assert got == [32, 32, 64, 64]
    assert hb.hpc_prefix_plan(tl.i32([0, 25]), tl.i32([64]), 25, 1, 1, q_len=4).tile_tokens == 64
