"""hpc_kv_compact, bit for bit."""
import numpy as np
import pytest
import torch

import _tiles
from load_balanced_paged_02_gb300 import binding as hb

pytestmark = pytest.mark.gpu


def bits(x):
    return x.view(torch.int32) if x.dtype == torch.float32 else x.view(torch.int16) if x.dtype == torch.bfloat16 else x.view(torch.uint8)


def make(lens, kept, hkv, kv, seed):
    c = _tiles.make_cache([lens, kept], hkv, kv, seed)
    rng = np.random.default_rng(seed)
    budget = max([1] + kept)
    keep = torch.full((len(lens), hkv, budget), -1, dtype=torch.int32)
    for b, (n, m) in enumerate(zip(lens, kept)):
        for h in range(hkv):
            keep[b, h, :m] = torch.from_numpy(np.sort(rng.permutation(n)[:m]).astype(np.int32))
    c["keep"], c["kept"] = keep.cuda(), _tiles.i32(kept)
    return c


def plain(c, lens, kept, names, table, new):
    want = {n: bits(c[n]).clone() for n in names}
    for b, m in enumerate(kept):
        for h in range(c["keep"].shape[1]):
            t = c["keep"][b, h, :m].long()
            j = torch.arange(m, device="cuda")
            src, dst = table[b].long()[t // 64], new[b].long()[j // 64]
            for n in names:
                if n.endswith("cache"):
                    want[n][dst, j % 64, h] = bits(c[n])[src, t % 64, h]
                else:
                    want[n][dst, h, j % 64] = bits(c[n])[src, h, t % 64]
    return want


def move(c, **kw):
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    hb.hpc_kv_compact(c["k_cache"], c["v_cache"], c["tables"][0], c["keep"], c["kept"], c["tables"][1], k_scale=c["k_scale"],
                      v_scale=c["v_scale"], error_word=word, **kw)
    return int(word.item())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens, kept, hkv", [
    ([37, 128, 300, 1000], [37, 100, 160, 160], 1),
    ([65, 1, 0, 64], [1, 1, 0, 63], 3),
    ([2000, 700], [1025, 513], 8),
    ([130], [129], 256),
    ([300 + i for i in range(70)], [70 + i for i in range(70)], 2),
])
def test_bit_for_bit(lens, kept, hkv, kv):
    c = make(lens, kept, hkv, kv, len(lens) + hkv)
    names = [n for n in ("k_cache", "v_cache", "k_scale", "v_scale") if c[n] is not None]
    want = plain(c, lens, kept, names, *c["tables"])
    w = torch.rand((len(lens), hkv, c["tables"][0].shape[1] * 64)).cuda()
    out = torch.full((len(lens), hkv, c["keep"].shape[2] + 3), 5.0).cuda()
    assert move(c, weights=w, weights_out=out) == 0
    for n in names:
        assert torch.equal(bits(c[n]), want[n]), n
    for b, m in enumerate(kept):
        assert torch.equal(out[b, :, :m], w[b].gather(1, c["keep"][b, :, :m].long()))
        assert (out[b, :, m:] == 5.0).all()


def test_all_kept_in_place():
    c = make([100, 300], [100, 80], 2, "bf16", 3)
    table = c["tables"][1].clone()
    table[0, :2] = c["tables"][0][0, :2]          # the first request's own pages
    names = ["k_cache", "v_cache"]
    want = plain(c, [100, 300], [100, 80], names, c["tables"][0], table)
    c["tables"][1] = table
    assert move(c) == 0
    for n in names:
        assert torch.equal(bits(c[n]), want[n])


def test_bad_tokens_pages_and_lengths():
    lens, kept = [300, 200, 90], [130, 100, 50]
    c = make(lens, kept, 2, "e4m3", 5)
    names = ["k_cache", "v_cache", "k_scale", "v_scale"]
    before = {n: bits(c[n]).clone() for n in names}
    good = plain(c, lens, kept, names, *c["tables"])
    # row (0, 1) names tokens that are not there, request 1's new page is out of the pool
    c["keep"][0, 1, 3] = -1
    c["keep"][0, 1, 4] = 1 << 30
    table = c["tables"][1].clone()
    page = int(table[1, 1])
    table[1, 1] = c["pages"] + 5
    p0 = int(table[0, 0])
    c["tables"][1] = table
    assert move(c) == 4
    for n in names:
        w = good[n]
        if n.endswith("cache"):
            w[p0, 3:5, 1] = before[n][p0, 3:5, 1]
        else:
            w[p0, 1, 3:5] = before[n][p0, 1, 3:5]
        w[page] = before[n][page]
        assert torch.equal(bits(c[n]), w), n
    # lengths that are negative or longer than a row
    c = make(lens, kept, 2, "bf16", 6)
    names = names[:2]
    good = plain(c, lens, [0, 100, 50], names, *c["tables"])
    c["kept"] = _tiles.i32([-3, 100, 50])
    assert move(c) == 1
    for n in names:
        assert torch.equal(bits(c[n]), good[n])
    c = make([300], [130], 2, "bf16", 6)
    good = plain(c, [300], [130], names, *c["tables"])
    c["kept"] = _tiles.i32([100000])
    assert move(c) == 4
    for n in names:
        assert torch.equal(bits(c[n]), good[n])


def test_graph_and_stream():
    lens, kept = [500, 300], [200, 64]
    c = make(lens, kept, 4, "bf16", 9)
    names = ["k_cache", "v_cache"]
    k0, v0 = c["k_cache"].clone(), c["v_cache"].clone()
    want = plain(c, lens, kept, names, *c["tables"])
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    args = (c["k_cache"], c["v_cache"], c["tables"][0], c["keep"], c["kept"], c["tables"][1])
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        hb.hpc_kv_compact(*args, stream=s)
    for _ in range(2):
        c["k_cache"].copy_(k0)
        c["v_cache"].copy_(v0)
        g.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(bits(c[n]), want[n])


def test_far_pages():
    """Pages whose rows lie beyond 2^31 elements (and 2^32 bytes) of the cache, read and written; weights in rows as far apart."""
    pages, hkv, lens, kept = 140000, 2, [300, 70], [130, 65]
    c = make(lens, kept, hkv, "bf16", 61)
    k, v = (torch.zeros((pages, 64, hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    far = [torch.where(t >= 0, pages - 1 - t, t).contiguous() for t in c["tables"]]
    for b, n in enumerate(lens):
        for j in range(-(-n // 64)):
            k[far[0][b, j]] = c["k_cache"][c["tables"][0][b, j]]
            v[far[0][b, j]] = c["v_cache"][c["tables"][0][b, j]]
    w = torch.empty((2, hkv, 700_000_000), device="cuda")
    near = torch.rand((2, hkv, 320), device="cuda")
    w[:, :, :320] = near
    out = torch.empty((2, hkv, 700_000_000), device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    hb.hpc_kv_compact(k, v, far[0], c["keep"], c["kept"], far[1], weights=w, weights_out=out, error_word=word)
    assert int(word.item()) == 0
    for b, m in enumerate(kept):
        j = torch.arange(m, device="cuda")
        for h in range(hkv):
            t = c["keep"][b, h, :m].long()
            old, new = c["tables"][0][b].long()[t // 64], far[1][b].long()[j // 64]
            assert torch.equal(k[new, j % 64, h], c["k_cache"][old, t % 64, h])
            assert torch.equal(v[new, j % 64, h], c["v_cache"][old, t % 64, h])
            assert torch.equal(out[b, h, :m], near[b, h, t])
