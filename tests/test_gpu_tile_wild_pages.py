"""Values of V that are not finite beside page ids out of range: the hidden tokens stay hidden in rows that are
computed again, whole tiles and cut ones."""
import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb
import _tiles as tl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctas", [None, 5])
@pytest.mark.parametrize("tile", [32, 64])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_hidden_page_and_nan(kv, tile, ctas):
    n, L, t = 80, 400, 370
    c = tl.make_cache([[L]], 2, kv, 91)
    q = tl.make_q((n, 16, 128), 92)
    table = c["tables"][0].clone()
    page, slot = int(table[0, t // 64]), t % 64
    if kv == "bf16":
        c["v_cache"][page, slot, 1, 9] = float("nan")
    else:
        c["v_cache"].view(torch.uint8)[page, slot, 1, 9] = 0x7f
    table[0, 2] = c["pages"] + 3
    out, lse, plan = hb.prefill(q, c["k_cache"], c["v_cache"], table, tl.i32([0, n]), tl.i32([L]), c["k_scale"], c["v_scale"],
                                tile_tokens=tile, num_ctas=ctas)
    assert hb.hpc_tile_read_error(plan) == 4
    keep = torch.cat([torch.arange(0, 128), torch.arange(192, L)]).cuda()
    k, v = c["k"][0][0][keep], c["v"][0][0][keep]
    ref = tl.attend(q, k, v, [L - n + i + 1 - 64 for i in range(n)])
    first = t - (L - n)
    rows = out.float()
    assert torch.isnan(rows[first:, 8:, 9]).all()
    rows[first:, 8:, 9] = ref[0][first:, 8:, 9].float()
    tl.check_rows(rows, lse, ref, kv != "bf16", "hidden page")
