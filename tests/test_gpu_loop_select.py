"""hpc_kv_select against a sort of each row."""
import pytest
import torch

import _loop
import _tiles
from load_balanced_paged_02_gb300 import binding as hb

pytestmark = pytest.mark.gpu


def run(w, lens, budget, first, recent, **kw):
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = torch.full((len(lens), w.shape[1], budget), 77, dtype=torch.int32, device="cuda")
    kl = torch.full((len(lens),), 77, dtype=torch.int32, device="cuda")
    hb.hpc_kv_select(w, _tiles.i32(lens), budget, first, recent, keep=keep, keep_lens=kl, error_word=word, **kw)
    return keep.cpu(), kl.cpu(), int(word.item())


def check(w, lens, budget, first, recent):
    keep, kl, word = run(w, lens, budget, first, recent)
    want, wl = _loop.select(w, lens, budget, first, recent)
    assert torch.equal(kl, wl) and torch.equal(keep, want)
    return word


def weights(B, hkv, width, seed, kind):
    gen = torch.Generator().manual_seed(seed)
    x = torch.exp(2.0 * torch.randn((B, hkv, width), generator=gen))
    if kind == "ties":
        x = torch.round(x)
    elif kind == "equal":
        x = torch.full_like(x, 0.25)
    elif kind == "signs":
        x = torch.randn((B, hkv, width), generator=gen)
        x[torch.rand(x.shape, generator=gen) < 0.2] = 0.0
        x[torch.rand(x.shape, generator=gen) < 0.2] = -0.0
    elif kind == "wild":
        pick = torch.randint(0, 8, x.shape, generator=gen)
        for k, v in enumerate((float("nan"), float("inf"), -float("inf"), 1e-45, -1e-45, 3e38)):
            x[pick == k] = v
    elif kind == "close":  # they differ in their last bits alone
        x = (torch.full_like(x, 1.0).view(torch.int32) + torch.randint(0, 900, x.shape, generator=gen, dtype=torch.int32)).view(torch.float32)
    return x.cuda()


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "signs", "wild", "close"])
@pytest.mark.parametrize("lens, budget, first, recent", [
    ([37, 128, 300, 1000], 160, 4, 32),
    ([1, 0, 2, 64, 65], 1, 0, 0),
    ([5, 6, 7], 6, 0, 6),                 # the recent ones fill the budget
    ([5, 6, 7, 90], 6, 6, 0),
    ([100, 99, 98], 98, 50, 47),
    ([3000, 2049, 2048, 31], 2047, 1, 0),
    ([4096, 33, 1024], 1, 1, 0),
])
def test_against_a_sort(lens, budget, first, recent, kind):
    assert check(weights(len(lens), 1 + budget % 3, max(lens) + 3, budget, kind), lens, budget, first, recent) == 0


@pytest.mark.parametrize("kind", ["plain", "ties", "equal"])
@pytest.mark.parametrize("B, hkv, n, budget", [
    (1, 1, 70000, 5000), (1, 8, 262147, 16384), (3, 8, 40001, 2048), (40, 8, 9000, 1000), (200, 2, 700, 64),
    (1, 1, 150000, 149999), (2, 1, 131072, 1),
])
def test_long_rows(B, hkv, n, budget, kind):
    """Clusters of every size, and parts that no longer fit a CTA's shared memory."""
    lens = [max(1, n - 97 * b) for b in range(B)]
    assert check(weights(B, hkv, n, n, kind), lens, budget, min(4, budget), max(0, min(30, budget - 4))) == 0


def test_rows_longer_than_shared_memory():
    w = weights(160, 2, 40000, 3, "ties")  # one CTA per row
    assert check(w, [40000 - 11 * b for b in range(160)], 3000, 16, 100) == 0


def test_bad_lengths():
    w = weights(3, 2, 200, 5, "plain")
    keep, kl, word = run(w, [-4, 5000, 120], 100, 2, 10)
    want, wl = _loop.select(w, [-4, 5000, 120], 100, 2, 10)
    assert word == 5 and torch.equal(kl, wl) and torch.equal(keep, want)


def test_streams_and_graphs():
    lens = [3000, 500]
    w = weights(2, 4, 3000, 8, "plain")
    want, wl = _loop.select(w, lens, 256, 4, 64)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep, kl = hb.hpc_kv_select(w, _tiles.i32(lens), 256, 4, 64, stream=s)
    s.synchronize()
    assert torch.equal(keep.cpu(), want) and torch.equal(kl.cpu(), wl)
    sl = _tiles.i32(lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hb.hpc_kv_select(w, sl, 256, 4, 64, keep=keep, keep_lens=kl)
    w2 = weights(2, 4, 3000, 9, "ties")
    w.copy_(w2)
    sl.copy_(_tiles.i32([100, 2999]))
    g.replay()
    torch.cuda.synchronize()
    want, wl = _loop.select(w2, [100, 2999], 256, 4, 64)
    assert torch.equal(keep.cpu(), want) and torch.equal(kl.cpu(), wl)


@pytest.mark.parametrize("B, hkv, n, budget", [(1, 1, 60000, 55000), (2, 8, 30000, 20000), (20, 8, 20000, 18000), (200, 1, 11000, 10800)])
@pytest.mark.parametrize("kind", ["plain", "ties", "wild"])
def test_more_stay_than_a_list_holds(B, hkv, n, budget, kind):
    lens = [n - 13 * b for b in range(B)]
    assert check(weights(B, hkv, n, n + 1, kind), lens, budget, 4, 30) == 0


@pytest.mark.parametrize("B, n", [(1, 50000), (3, 300), (170, 9000)])
@pytest.mark.parametrize("share", [0.3, 0.7, 0.95])
def test_down_to_infinities_and_undefined_values(B, n, share):
    """The budget reaches -infinity, or NaN of either sign."""
    w = weights(B, 2, n, 17, "plain").cpu()
    gen = torch.Generator().manual_seed(18)
    pick = torch.rand(w.shape, generator=gen)
    bits = w.view(torch.int32)
    bits[pick < 0.9] = 0x7fc00000
    bits[pick < 0.6] = 0x7f800001
    bits[pick < 0.5] = -0x00000001  # 0xffffffff
    bits[pick < 0.4] = -0x007fffff  # 0xff800001
    w[pick < 0.3] = -float("inf")
    assert torch.isnan(w).float().mean() > 0.5
    assert check(w.cuda(), [n - b for b in range(B)], int(share * n), 2, 5) == 0


@pytest.mark.parametrize("lens", [[70000, 100, 9000], [0, 70000], [5000, 4200, 4097, 1, 8000, 4096, 70000, 30000]])
def test_short_rows_beside_long_ones(lens):
    """Clusters of which a row uses all CTAs, some, or one; and rows that need none."""
    for budget, first, recent in ((64, 4, 32), (4096, 0, 0), (1, 0, 1), (100, 50, 50)):
        assert check(weights(len(lens), 2, 70001, budget, "ties"), lens, budget, first, recent) == 0


def test_rows_far_apart():
    """Rows that begin beyond 2^31 elements of the weights, at the longest distance that the call takes."""
    far = torch.empty((3, 1, 1 << 30), device="cuda")
    near = weights(3, 1, 5000, 21, "ties")
    far[:, :, :5000] = near
    lens = [5000, 160, 4097]
    keep, kl, word = run(far, lens, 160, 4, 32)
    want, wl = _loop.select(near, lens, 160, 4, 32)
    assert word == 0 and torch.equal(kl, wl) and torch.equal(keep, want)
