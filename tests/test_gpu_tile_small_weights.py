"""Many keys of very small weight beside a heavy one, e4m3 cache: their probabilities enter the second product as f16
numbers, and must count there as they do in the sum."""
import math

import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb
import _tiles as tl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tile", [32, 64])
@pytest.mark.parametrize("q0", [180.0, 204.0, 220.0])
def test_weights_far_below_the_largest(q0, tile):
    """One key of score q0 / sqrt(128) and 2^17 - 1 keys of score 0, V 0 and 1: the output is the small ones' part
    of the sum, N w / (1 + N w), w = exp(-q0 / sqrt(128)) (2^-23 to 2^-28).

    P is 2^5 w in f16, a multiple of 2^-24 (subnormal): off by half of that at most, 2^-25 / (2^5 w) relative to
    itself. V = 448 x (1 / 448), scale and product rounded to f16: 2^-10. The sums add 2^-13 (2048 pages, each added
    in float32 with 2^-24 of the sum so far), the output's rounding 2^-8. The LSE: 128 products of the score, of
    which one is not zero, and the sums, 2^-17 of the score in all (2^-17 x 180 > 2^-13 + 2^-19)."""
    n, pages = 1 << 17, 1 << 11
    kc = torch.zeros((pages, 64, 1, 128), dtype=torch.uint8, device="cuda")
    vc = torch.full((pages, 64, 1, 128), 0x7e, dtype=torch.uint8, device="cuda")  # 448
    ks = torch.full((pages, 1, 64), 1 / 448, device="cuda")
    vs = ks.clone()
    kc[0, 0, 0, 0], vc[0, 0] = 0x7e, 0
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = q0
    e4m3 = torch.float8_e4m3fn
    out, lse, _ = hb.prefill(q, kc.view(e4m3), vc.view(e4m3), torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages),
                             tl.i32([0, 1]), tl.i32([n]), ks, vs, num_ctas=1 if tile == 32 else 2, tile_tokens=tile)
    one = float(torch.tensor(1 / 448)) * 448
    w = math.exp(-q0 * one / math.sqrt(128))
    want = (n - 1) * w / (1 + (n - 1) * w) * one
    tol = want * (2.0 ** -25 / (32 * w) + 2.0 ** -10 + 2.0 ** -13 + 2.0 ** -8)
    assert (out.double() - want).abs().max().item() <= tol
    assert (lse.double() - (q0 * one / math.sqrt(128) + math.log1p((n - 1) * w))).abs().max().item() <= 2.0 ** -17 * q0
