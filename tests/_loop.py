"""Helpers for the tests of the decode loop's operators between two attention steps: plain
implementations in 64 bits and the tolerances that the kernels' roundings give."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE, DIM, GROUP = 64, 128, 8


def attn_weights(q, q_starts, lse, keys, lens, old, counts=None, window=0, decay=1.0, fp8=False):
    """weights [B, hkv, tokens] (float64) after a call, and the bound on each one's error. keys[b] holds the exact
    keys [tokens, hkv, 128] of request b in float64; rows and lengths as the call takes them.

    The bound: a score is a float32 sum of 128 products, off by at most es = 128 * 2^-23 * sum |q_d k_d| / sqrt(128); on
    an e4m3 cache the query is split into two e4m3 numbers, which leaves at most 2^-17 of the row's largest element per
    product, counted by doubling es and adding 2^-17 max |q| sum |k_d| / sqrt(128). In the exponent, the factors
    (log2(e) / sqrt(128), its product with scales, lse * log2(e)) and the result are each rounded: 2^-22 of |score| +
    |lse| covers four roundings of 2^-24. exp2 is off by 2^-22, the float32 sum of m numbers that are not negative by
    at most m * 2^-24 of itself; the old value takes two roundings."""
    w = old.double().clone()
    bound = torch.zeros_like(w)
    for b, total in enumerate(lens):
        first, n = q_starts[b], q_starts[b + 1] - q_starts[b]
        if n <= 0:
            continue
        total = max(0, total)
        hi = n if counts is None else max(0, min(n, counts[b]))
        lo = max(0, hi - window) if window else 0
        hkv = w.shape[1]
        got = torch.zeros((hkv, total), dtype=torch.float64, device=w.device)
        err = torch.zeros_like(got)
        for i0 in range(lo, hi, 32):
            i1 = min(hi, i0 + 32)
            r = torch.arange(i0, i1, device=w.device)
            qd = q[first + i0:first + i1].double().view(i1 - i0, hkv, GROUP, DIM)
            l = lse[first + i0:first + i1].double().view(i1 - i0, hkv, GROUP, 1)
            s = torch.einsum("rhgd,thd->rhgt", qd, keys[b][:total]) / math.sqrt(DIM)
            es = 128 * 2.0 ** -23 * torch.einsum("rhgd,thd->rhgt", qd.abs(), keys[b][:total].abs()) / math.sqrt(DIM)
            if fp8:
                es = 2 * es + 2.0 ** -17 * torch.einsum("rhg,th->rhgt", qd.abs().amax(-1), keys[b][:total].abs().sum(-1)) / math.sqrt(DIM)
            seen = torch.arange(total, device=w.device).view(1, 1, 1, -1) <= (total - n + r).view(-1, 1, 1, 1)
            use = seen & (l != -math.inf)
            e = torch.where(use, torch.exp(s - l), 0.0)
            rel = es + 2.0 ** -22 * (s.abs() + l.abs()) + 2.0 ** -22
            got += e.sum(dim=(0, 2))
            err += torch.where(use, e * torch.expm1(rel), 0.0).sum(dim=(0, 2))
        older = max(0, total - n)
        bound[b, :, :total] = 1.01 * (err + (GROUP * (hi - lo) + 2) * 2.0 ** -24 * got) + 1e-37
        if decay:
            bound[b, :, :older] += 2.0 ** -22 * (decay * w[b, :, :older]).abs()
            got[:, :older] += decay * w[b, :, :older]
        w[b, :, :total] = got
    return w, bound


def row_lse(q, q_starts, keys, lens):
    """The attention call's log-sum-exps in float32: -inf for a row that sees nothing."""
    rows, hq = q.shape[0], q.shape[1]
    lse = torch.full((rows, hq), float("nan"), device=q.device)
    for b, total in enumerate(lens):
        first, n = q_starts[b], q_starts[b + 1] - q_starts[b]
        total = max(0, total)
        for i in range(max(0, n)):
            seen = max(0, total - n + i + 1)
            qd = q[first + i].double().view(-1, GROUP, DIM)
            s = torch.einsum("hgd,thd->hgt", qd, keys[b][:seen]) / math.sqrt(DIM)
            lse[first + i] = torch.logsumexp(s, dim=-1).reshape(-1).float() if seen else -math.inf
    return lse


def select(weights, lens, budget, first, recent):
    """keep [B, hkv, budget] and its lengths, by a sort of each row."""
    w = weights.double().cpu().numpy()
    B, hkv, stride = w.shape
    keep = np.full((B, hkv, budget), -1, dtype=np.int32)
    kept = []
    for b, total in enumerate(lens):
        total = min(max(0, total), stride)
        kept.append(min(total, budget))
        for h in range(hkv):
            if total <= budget:
                keep[b, h, :total] = np.arange(total)
                continue
            row = np.where(np.isnan(w[b, h]), -np.inf, w[b, h])
            nan = np.isnan(w[b, h])
            mid = np.arange(first, total - recent)
            # NaN behind everything, -inf included
            chosen = mid[np.lexsort((mid, -row[mid], nan[mid]))][:budget - first - recent]
            keep[b, h] = np.sort(np.concatenate((np.arange(first), chosen, np.arange(total - recent, total))))
    return torch.from_numpy(keep), torch.tensor(kept, dtype=torch.int32)


def verify(target, draft, drafted, accept, sample, counts=None):
    """num_accepted and tokens, request by request in 64 bits."""
    p = target.double().cpu().numpy()
    q = None if draft is None else draft.double().cpu().numpy()
    d = drafted.cpu().numpy()
    u, us = accept.double().cpu().numpy(), sample.double().cpu().numpy()
    B, n, V = d.shape[0], d.shape[1], p.shape[2]

    def clean(x):
        return np.where((x > 0) & (x < 2.0 ** 64), x, 0.0)

    accepted, tokens = [], []
    for b in range(B):
        c = n if counts is None else max(0, min(n, int(counts[b])))
        r, out = 0, []
        while r < c:
            t = int(d[b, r])
            if not 0 <= t < V:
                break
            qq = 1.0 if q is None else q[b, r, t]
            if not u[b, r] * qq < p[b, r, t]:
                break
            out.append(t)
            r += 1
        rest = p[b, r].copy()
        if r < c:
            if q is not None:
                with np.errstate(invalid="ignore"):
                    rest = rest - q[b, r]
            elif 0 <= d[b, r] < V:
                rest[d[b, r]] = 0.0
        rest = clean(rest)
        if rest.sum() == 0:
            rest = clean(p[b, r])
        sums = np.cumsum(rest)
        if sums[-1] == 0:
            out.append(-1)
        else:
            over = np.nonzero((sums > us[b] * sums[-1]) & (rest > 0))[0]
            out.append(int(over[0]) if len(over) else int(np.nonzero(rest > 0)[0][-1]))
        accepted.append(r)
        tokens.append(out + [-1] * (n + 1 - len(out)))
    return torch.tensor(accepted, dtype=torch.int32), torch.tensor(tokens, dtype=torch.int32)
