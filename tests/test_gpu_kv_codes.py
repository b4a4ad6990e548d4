"""hpc_kv_write's e4m3 codes and scales bit for bit, over every pair of significands of a row's largest element and
of its other ones, at sizes on both sides of the kernel's two ways to divide."""
import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb

pytestmark = pytest.mark.gpu


def test_codes_and_scales_bit_for_bit():
    exponents = [-125, -110, -92, -91, -90, -73, -72, -71, -70, -20, 0, 1, 60, 107, 108, 109, 110, 127]
    j = torch.arange(128)
    rows = []
    for e in exponents:
        for d in range(10):  # elements 2^(1 + d) below the largest, one significand each, the signs mixed
            top = (1 + torch.arange(128, dtype=torch.float64) / 128) * 2.0 ** e
            x = (1 + ((j + d) % 128).double() / 128) * 2.0 ** (e - 1 - d) * (1 - 2 * (j % 2)).double()
            row = x.expand(128, 128).clone()
            row[:, 0] = top
            rows.append(row)
    x = torch.cat(rows).to(torch.bfloat16)
    T = x.shape[0]
    pages = -(-T // 64)
    kc, vc = (torch.zeros((pages, 64, 1, 128), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, 1, 64), device="cuda") for _ in range(2))
    k = x.cuda().view(T, 1, 128)
    hb.hpc_kv_write(k, -k, torch.arange(T, dtype=torch.int32, device="cuda"), kc, vc, ks, vs)
    torch.cuda.synchronize()
    scale = x.float().abs().amax(dim=1) / torch.tensor(448.0)
    for cache, scales, sign in ((kc, ks, 1.0), (vc, vs, -1.0)):
        assert torch.equal(scales.cpu().view(-1)[:T].view(torch.int32), scale.view(torch.int32))
        want = (sign * x.float() / scale.unsqueeze(1)).to(torch.float8_e4m3fn).view(torch.uint8)
        got = cache.cpu().view(torch.uint8).view(-1, 128)[:T]
        assert torch.equal(got, want)
