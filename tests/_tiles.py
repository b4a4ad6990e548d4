"""Helpers for the tests of prompt attention, shared-prefix decode and the cache
write / read calls: small paged batches with poisoned unused slots, plain
implementations in 64 bits, and the tolerances that the kernels' roundings give."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE, DIM, GROUP = 64, 128, 8
E4M3_MAX = 448.0
INF = float("inf")


def make_cache(lens_lists, hkv, kv, seed, device="cuda", scale=1.0, spread=False):
    """K and V for lists of lengths, in one shuffled pool whose unused slots hold NaN (NaN codes and
    NaN scales for e4m3). Returns a dict with caches, scales, one page table per list (unused entries
    -1) and the exact values k[list][row], v[...] in float64, [tokens, hkv, 128]."""
    gen = torch.Generator(device="cpu").manual_seed(seed)
    rng = np.random.default_rng(seed)
    counts = [[-(-n // PAGE) for n in lens] for lens in lens_lists]
    pages = sum(sum(c) for c in counts) + 2
    perm = rng.permutation(pages)
    c = dict(pages=pages, tables=[], k=[], v=[])
    raw = {}
    for name in "kv":
        x = torch.full((pages, PAGE, hkv, DIM), float("nan"), dtype=torch.float32)
        raw[name] = x
    at = 0
    where = []
    for lens, cnt in zip(lens_lists, counts):
        table = torch.full((max(1, len(lens)), max([1] + cnt)), -1, dtype=torch.int32)
        spots = []
        for b, (n, m) in enumerate(zip(lens, cnt)):
            mine = perm[at:at + m]
            at += m
            table[b, :m] = torch.from_numpy(mine.astype(np.int32))
            t = np.arange(n)
            spots.append((torch.from_numpy(mine[t // PAGE].astype(np.int64)), torch.from_numpy(t % PAGE)))
            for name in "kv":
                val = torch.randn((n, hkv, DIM), generator=gen) * scale
                if spread:  # tokens of very different sizes
                    val = val * torch.exp(torch.randn((n, hkv, 1), generator=gen) * 1.5)
                raw[name][spots[-1]] = val.to(torch.bfloat16).float()
        c["tables"].append(table.to(device))
        where.append(spots)
    for name in "kv":
        x = raw[name]
        if kv == "bf16":
            cache, sc = x.to(torch.bfloat16), None
            value = cache.double()
        else:
            amax = x.abs().amax(dim=-1)
            step = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
            cache = (x / step.unsqueeze(-1)).to(torch.float8_e4m3fn)
            value = cache.to(torch.float32).double() * step.double().unsqueeze(-1)
            sc = step.permute(0, 2, 1).contiguous()
        c[name + "_cache"] = cache.to(device)
        c[name + "_scale"] = None if sc is None else sc.to(device)
        c[name] = [[value[s].to(device) for s in spots] for spots in where]
    return c


def make_q(shape, seed, device="cuda", scale=1.0):
    gen = torch.Generator(device="cpu").manual_seed(seed + 1)
    return (torch.randn(shape, generator=gen) * scale).to(torch.bfloat16).to(device)


def attend(q, k, v, visible):
    """q [n, hq, 128], k / v [t, hkv, 128] in float64; row i sees the first visible[i] tokens. Returns out,
    lse, the values' weighted mean sizes sum w |v|, each row's bound on the score's products, the
    largest sum_d |q_d k_d| / sqrt(128) among the tokens it sees, and sum |v| over the tokens it sees."""
    n, hq, _ = q.shape
    t, hkv, _ = k.shape
    if t == 0:
        z = torch.zeros((n, hq, DIM), dtype=torch.float64, device=q.device)
        s = torch.zeros((n, hq), dtype=torch.float64, device=q.device)
        return z, s - INF, z, s, z
    qg = q.double().view(n, hkv, GROUP, DIM)
    s = torch.einsum("nhgd,thd->nhgt", qg, k) / math.sqrt(DIM)
    size = torch.einsum("nhgd,thd->nhgt", qg.abs(), k.abs()) / math.sqrt(DIM)
    hidden = torch.arange(t, device=q.device) >= torch.as_tensor(visible, device=q.device).view(n, 1, 1, 1)
    s = s.masked_fill(hidden, -INF)
    size = size.masked_fill(hidden, 0.0).amax(dim=-1)
    lse = torch.logsumexp(s, dim=-1)
    w = torch.where(torch.isfinite(lse).unsqueeze(-1), torch.exp(s - torch.where(torch.isfinite(lse), lse, 0.0).unsqueeze(-1)), 0.0)
    out = torch.einsum("nhgt,thd->nhgd", w, v)
    absv = torch.einsum("nhgt,thd->nhgd", w, v.abs())
    seen = torch.einsum("nt,thd->nhd", (~hidden.view(n, t)).double(), v.abs()).repeat_interleave(GROUP, dim=1)
    return (out.reshape(n, hq, DIM), lse.reshape(n, hq), absv.reshape(n, hq, DIM), size.reshape(n, hq), seen)


def check_rows(got, got_lse, ref, fp8, what=""):
    """got (bf16) and got_lse (float32) against attend()'s answer.

    A row's score is a float32 sum of 128 products: off by at most es = 128 * 2^-23 * sum |q_d k_d| /
    sqrt(128). On an e4m3 cache the query is split into two e4m3 numbers, which leaves at most 2^-17 of
    the row's largest element per product: less than es, counted by doubling it. exp2 and the sums add 2^-20.
    So a probability is off by 2 es + 2^-20 relative to the row's sum. Probabilities enter the second
    product rounded to bf16 (2^-8), or to f16 (2^-11) with V rounded to f16 twice (scale and product,
    2^-11 each, and 2^-25 per element for results under f16's normal range). A probability below 2^-14 of
    the reference is under f16's normal range too: off by at most 2^-25 whatever its size, so a token adds
    2^-25 |v| / l, and l >= 1, for the key that set the reference counts as 1. The output is rounded to
    bf16 (2^-8)."""
    out, lse, absv, size, seen = ref
    assert torch.equal(torch.isfinite(lse), torch.isfinite(got_lse)), f"{what}: rows that see nothing differ"
    assert torch.isfinite(got.float()).all(), f"{what}: non-finite outputs"
    es = (2 if fp8 else 1) * 128 * 2.0 ** -23 * size
    p_err = 2 * es.unsqueeze(-1) + 2.0 ** -20
    prod = 3 * 2.0 ** -11 if fp8 else 2.0 ** -8
    tol = (p_err + prod) * absv * 1.01 + (2.0 ** -24 + 2.0 ** -25 * seen if fp8 else 0.0)
    tol = tol + 2.0 ** -8 * (out.abs() + tol) + 1e-30
    err = (got.double() - out).abs()
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: output off by {worst:.2f} tolerances (max abs {err.max().item():.3g})"
    fin = torch.isfinite(lse)
    if fin.any():
        lt = es + 2.0 ** -19 + lse.abs() * 2.0 ** -22
        lw = ((got_lse.double() - lse).abs()[fin] / lt[fin]).max().item()
        assert lw <= 1.0, f"{what}: LSE off by {lw:.2f} tolerances"


def i32(values, device="cuda"):
    return torch.tensor(list(values), dtype=torch.int32, device=device)


def starts(counts):
    return [0] + list(np.cumsum(counts).astype(int).tolist()) if len(counts) else [0]


def tile_map(mode, q_starts, lens, num_tokens, hkv, workers, min_blocks, T, q_len=1, max_len=1 << 30):
    """The words of a tile map from its definition: every (head, sequence, tile, unit) in order, cut
    into equal runs."""
    S = len(lens)
    seqs, units_before, tiles_before = [], [0], 0
    walk = []  # of one head: (sequence, tile, block, or -1 twice for the fixed cost)
    err = 0
    for s in range(S):
        a, b, L = q_starts[s] * q_len, q_starts[s + 1] * q_len, lens[s]
        if L < 0:
            err |= 1
            L = 0
        if L > max_len:
            err |= 4
            L = max_len
        if a < 0 or b < a or b > num_tokens:
            err |= 16
            a, n = 0, 0
        else:
            n = b - a
        a = a if n or (q_starts[s] * q_len >= 0 and b >= a) else 0
        seqs.append([a, n, L, tiles_before])
        tiles = 0
        if n > 0 and (mode == 0 or L > 0):
            tiles = -(-n // T)
            for i in range(tiles):
                end = L if mode == 1 else max(0, L - n + min(n, T * (i + 1)))
                blocks = max(1, -(-end // 128)) if mode == 0 else -(-end // 128)
                walk += [(s, i, -1)] * 2 + [(s, i, blk) for blk in range(blocks)]
        tiles_before += tiles
        units_before.append(len(walk))
    per_head, total = len(walk), len(walk) * hkv
    bucket = max(-(-total // workers), min_blocks, 1)
    words = [per_head & 0xffffffff, per_head >> 32, bucket & 0xffffffff, bucket >> 32, -(-total // bucket), S, hkv,
             workers, num_tokens, mode, tiles_before, q_len, err, T, 0, 0]
    for j in range(workers + 1):
        g = j * bucket
        if g >= total:
            words += [hkv, 0, 0, 0, 0, 0, 0, 0]
        else:
            s, i, blk = walk[g % per_head]
            h = g // per_head
            words += [h, s, i, max(blk, 0)] + seqs[s]
    for x in seqs:
        words += x
    for u in units_before:
        words += [u & 0xffffffff, u >> 32]
    return np.asarray(words, dtype=np.int64).astype(np.int32)
