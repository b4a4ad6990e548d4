"""hpc_attn_weights against its definition in 64 bits."""
import math

import pytest
import torch

import _loop
import _tiles
from load_balanced_paged_02_gb300 import binding as hb

pytestmark = pytest.mark.gpu


def case(new, lens, hkv, kv, seed, scale=1.0, spread=False):
    c = _tiles.make_cache([[max(0, n) for n in lens]], hkv, kv, seed, scale=scale, spread=spread)
    starts = _tiles.starts(new)
    q = _tiles.make_q((starts[-1], 8 * hkv, 128), seed, scale=scale)
    lse = _loop.row_lse(q, starts, c["k"][0], lens)
    width = c["tables"][0].shape[1] * 64 + 5  # rows longer than the table's
    gen = torch.Generator().manual_seed(seed + 7)
    old = torch.rand((len(lens), hkv, width), generator=gen).cuda()
    return c, starts, q, lse, old


def run(c, starts, q, lse, w, lens, **kw):
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    hb.hpc_attn_weights(q, c["k_cache"], c["tables"][0], _tiles.i32(lens), lse, w, q_starts=_tiles.i32(starts), k_scale=c["k_scale"],
                        error_word=word, **{k: v for k, v in kw.items()})
    return int(word.item())


def check(got, want, bound, old, what=""):
    touched = bound > 0
    assert torch.equal(got[~touched], old[~touched]), f"{what}: weights that are not the call's have changed"
    off = ((got.double() - want).abs() / bound)[touched]
    assert torch.isfinite(got[touched]).all(), what
    assert off.numel() == 0 or off.max().item() <= 1.0, f"{what}: off by {off.max().item():.2f} bounds"


CASES = [
    # (rows of each sequence, lengths, counts, window)
    ([1, 1, 1, 1], [37, 128, 300, 1000], None, 0),
    ([1], [1], None, 0),
    ([1, 1, 1], [0, 65, 64], None, 0),
    ([4, 4, 4], [129, 4, 700], [1, 3, 4], 0),
    ([8, 8], [8, 1025], [0, 9], 0),                       # none counted; more than there are
    ([5, 0, 2, 7], [3, 50, 2, 600], None, 0),             # rows that see nothing; a sequence without rows
    ([100, 33, 1, 64], [100, 500, 129, 64], None, 0),     # whole prompts and pieces
    ([100, 33, 1, 64], [300, 500, 129, 64], None, 32),
    ([70, 17, 16, 15], [128, 1000, 257, 40], None, 16),
    ([90, 200], [90, 1500], [50, 120], 65),
    ([130], [1153], None, 0),                             # more rows than one pass takes
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("k", range(len(CASES)))
def test_against_definition(k, kv):
    new, lens, counts, window = CASES[k]
    hkv = 1 + k % 3
    c, starts, q, lse, old = case(new, lens, hkv, kv, 100 + k, spread=k % 2 == 1)
    for decay in (1.0, 0.0, 0.625):
        w = old.clone()
        if decay == 0.0:
            w.fill_(float("nan"))  # nothing is read
        before = w.clone()
        assert run(c, starts, q, lse, w, lens, counts=None if counts is None else _tiles.i32(counts), window=window, decay=decay) == 0
        want, bound = _loop.attn_weights(q, starts, lse, c["k"][0], lens, old, counts, window, decay, kv == "e4m3")
        if decay == 0.0:
            touched = bound > 0
            assert torch.isnan(w[~touched]).all()
            check(torch.where(touched, w, old), want, bound, old, f"decay {decay}")
        else:
            check(w, want, bound, before, f"decay {decay}")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_batch_shapes(kv):
    """q [B, Hq, 128] and [B, q_len, Hq, 128] without starts: the same rows, the same weights."""
    for q_len in (1, 3, 8):
        lens = [200, 64, 9, 1500, 77]
        c, starts, q, lse, old = case([q_len] * 5, lens, 2, kv, 40 + q_len)
        w0, w1 = old.clone(), old.clone()
        run(c, starts, q, lse, w0, lens)
        shape = (5, 16, 128) if q_len == 1 else (5, q_len, 16, 128)
        hb.hpc_attn_weights(q.view(shape), c["k_cache"], c["tables"][0], _tiles.i32(lens), lse.view(shape[:-1]), w1, k_scale=c["k_scale"])
        assert torch.equal(w0, w1)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_weights_of_a_row_sum_to_one(kv):
    """Every row hands out a weight of one per query head: 8 per KV head and row."""
    lens, new = [777, 130, 64], [3, 130, 1]
    c, starts, q, lse, old = case(new, lens, 2, kv, 9)
    w = torch.zeros_like(old)
    run(c, starts, q, lse, w, lens, decay=0.0)
    total = w.double().sum(-1)
    want = torch.tensor([[8.0 * n] * 2 for n in new], device="cuda", dtype=torch.float64)
    # every weight is relatively off by at most the bound on its scores (lse rounds at 2^-24 of itself too)
    assert ((total - want).abs() / want).max().item() < 2e-4


def test_batch_composition_changes_no_bit():
    lens, new = [777, 130, 64, 2000, 33], [3, 60, 1, 40, 8]
    c, starts, q, lse, old = case(new, lens, 2, "bf16", 11)
    all_w = old.clone()
    run(c, starts, q, lse, all_w, lens)
    for b in range(5):
        w = old[b:b + 1].clone()
        rows = slice(starts[b], starts[b + 1])
        hb.hpc_attn_weights(q[rows].contiguous(), c["k_cache"], c["tables"][0][b:b + 1], _tiles.i32(lens[b:b + 1]), lse[rows].contiguous(), w,
                            q_starts=_tiles.i32([0, new[b]]))
        assert torch.equal(w[0], all_w[b])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_bad_pages_starts_and_lengths(kv):
    lens, new = [300, 200, 150, 90], [4, 3, 2, 1]
    c, starts, q, lse, old = case(new, lens, 1, kv, 21)
    keys = c["k"][0]
    table = c["tables"][0].clone()
    table[0, 2] = c["pages"]           # tokens 128 .. 191 of the first
    table[1, 0] = -7
    broken = dict(c, tables=[table])
    w = old.clone()
    assert run(broken, starts, q, lse, w, lens) == 4
    want, bound = _loop.attn_weights(q, starts, lse, keys, lens, old, fp8=kv == "e4m3")
    for b, t0, t1 in ((0, 128, 192), (1, 0, 64)):
        want[b, :, t0:t1] = old[b, :, t0:t1].double()
    check(w, want, bound, old)
    # a sequence whose starts decrease or leave the rows is passed over
    w = old.clone()
    assert run(c, [0, 4, 2, 9, 99], q, lse, w, lens) == 16
    assert torch.equal(w[1], old[1]) and torch.equal(w[3], old[3])
    assert not torch.equal(w[0], old[0])
    # lengths below zero and beyond the table
    w = old.clone()
    assert run(c, starts, q, lse, w, [-5, 1 << 30, 150, 90]) == 5
    assert torch.equal(w[0], old[0]) and not torch.equal(w[2], old[2])


def test_infinite_and_undefined_values_stay_with_their_token():
    lens, new = [200], [3]
    c, starts, q, lse, old = case(new, lens, 1, "bf16", 31)
    clean = old.clone()
    run(c, starts, q, lse, clean, lens)
    page, slot = int(c["tables"][0][0, 1]), 7
    for value in (float("nan"), float("inf")):
        dirty = dict(c, k_cache=c["k_cache"].clone())
        dirty["k_cache"][page, slot] = value
        w = old.clone()
        run(dirty, starts, q, lse, w, lens)
        same = torch.ones(old.shape[2], dtype=torch.bool, device="cuda")
        same[64 + slot] = False
        assert torch.equal(w[0, 0, same], clean[0, 0, same])
    # a row of -inf has no weight, one of NaN spoils what it sees
    l2 = lse.clone()
    l2[1, 3] = -math.inf
    w = old.clone()
    run(c, starts, q, l2, w, lens)
    want, bound = _loop.attn_weights(q, starts, l2, c["k"][0], lens, old)
    check(w, want, bound, old)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_large_and_small_scores(kv):
    """Peaked rows: scores of some hundreds, weights from one down to nothing."""
    lens, new = [400, 130], [2, 20]
    c, starts, q, lse, old = case(new, lens, 1, kv, 33, scale=4.0)
    w = old.clone()
    run(c, starts, q, lse, w, lens)
    want, bound = _loop.attn_weights(q, starts, lse, c["k"][0], lens, old, fp8=kv == "e4m3")
    check(w, want, bound, old)


def test_far_pages():
    """Pages whose rows lie beyond 2^31 elements (and 2^32 bytes) of the cache."""
    pages, hkv = 140000, 2
    k = torch.zeros((pages, 64, hkv, 128), dtype=torch.bfloat16, device="cuda")
    lens, new = [300, 70], [2, 1]
    c, starts, q, lse, old = case(new, lens, hkv, "bf16", 51)
    table = c["tables"][0]
    far = torch.where(table >= 0, pages - 1 - table, table)
    for b in range(2):
        for j in range(-(-lens[b] // 64)):
            k[far[b, j]] = c["k_cache"][table[b, j]]
    w0, w1 = old.clone(), old.clone()
    run(c, starts, q, lse, w0, lens)
    run(dict(c, k_cache=k, tables=[far.contiguous()]), starts, q, lse, w1, lens)
    assert torch.equal(w0, w1)


def test_many_sequences_and_heads():
    """More sequences than a block has threads; and the most KV heads."""
    lens = [1 + (7 * i) % 200 for i in range(1100)]
    new = [1 + i % 3 for i in range(1100)]
    c, starts, q, lse, old = case(new, lens, 1, "bf16", 61)
    w = old.clone()
    assert run(c, starts, q, lse, w, lens) == 0
    want, bound = _loop.attn_weights(q, starts, lse, c["k"][0], lens, old)
    check(w, want, bound, old)
    lens, new = [100, 33], [1, 2]
    c, starts, q, lse, old = case(new, lens, 256, "e4m3", 62)
    w = old.clone()
    assert run(c, starts, q, lse, w, lens) == 0
    want, bound = _loop.attn_weights(q, starts, lse, c["k"][0], lens, old, fp8=True)
    check(w, want, bound, old)


def test_streams_and_graphs():
    """Two streams at once, and a captured call replayed on new inputs."""
    lens, new = [900, 130, 64], [3, 60, 1]
    c, starts, q, lse, old = case(new, lens, 2, "bf16", 71)
    want, bound = _loop.attn_weights(q, starts, lse, c["k"][0], lens, old)
    table, sl, qs = c["tables"][0], _tiles.i32(lens), _tiles.i32(starts)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [old.clone() for _ in range(2)]
    torch.cuda.synchronize()
    for s, w in zip(streams, outs):
        hb.hpc_attn_weights(q, c["k_cache"], table, sl, lse, w, q_starts=qs, stream=s)
    torch.cuda.synchronize()
    for w in outs:
        check(w, want, bound, old)
    w = old.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hb.hpc_attn_weights(q, c["k_cache"], table, sl, lse, w, q_starts=qs)
    w.copy_(old)
    g.replay()
    check(w, want, bound, old)
    lens2 = [500, 70, 63]  # other lengths, the same buffers
    lse2 = _loop.row_lse(q, starts, [k[:n] for k, n in zip(c["k"][0], lens2)], lens2)
    sl.copy_(_tiles.i32(lens2))
    lse.copy_(lse2)
    w.copy_(old)
    g.replay()
    torch.cuda.synchronize()
    want, bound = _loop.attn_weights(q, starts, lse2, c["k"][0], lens2, old)
    check(w, want, bound, old)
