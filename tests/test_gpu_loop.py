"""The operators between two attention steps as a decode loop runs them: prompts, weights of their last queries, eviction,
decode over what is left, drafted tokens verified and only the accepted rows counted; then the same captured into
a graph; and tensors that are not where the others are."""
import math

import pytest
import torch

import _loop
import _tiles
import load_balanced_paged_02_gb300 as hpc

pytestmark = pytest.mark.gpu

BUDGET, FIRST, RECENT, WINDOW = 160, 4, 32, 16


def kept_rows(values, keep, m):
    """values [tokens, hkv, 128] -> the kept tokens of each head, [m, hkv, 128]."""
    return torch.stack([values[keep[h, :m].long(), h] for h in range(values.shape[1])], dim=1)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_loop(kv):
    hkv, fp8 = 2, kv == "e4m3"
    lens = [700, 129, 300, 64]
    drafts = 3
    kept_len = [min(n, BUDGET) for n in lens]
    grown = [m + drafts + 1 for m in kept_len]
    c = _tiles.make_cache([lens, grown], hkv, kv, 5)
    table, new_table = c["tables"]
    B = len(lens)

    # the prompts, and what their last queries looked at
    starts = _tiles.starts(lens)
    q = _tiles.make_q((starts[-1], 8 * hkv, 128), 6)
    qs, sl = _tiles.i32(starts), _tiles.i32(lens)
    out, lse, _ = hpc.prefill(q, c["k_cache"], c["v_cache"], table, qs, sl, c["k_scale"], c["v_scale"])
    weights = torch.full((B, hkv, table.shape[1] * 64), float("nan"), device="cuda")
    hpc.hpc_attn_weights(q, c["k_cache"], table, sl, lse, weights, q_starts=qs, k_scale=c["k_scale"], window=WINDOW, decay=0.0)
    want, bound = _loop.attn_weights(q, starts, lse, c["k"][0], lens, torch.zeros_like(weights), None, WINDOW, 0.0, fp8)
    for b, n in enumerate(lens):
        assert ((weights[b, :, :n].double() - want[b, :, :n]).abs() <= bound[b, :, :n]).all()

    # what stays, and where it goes
    keep, kept = hpc.hpc_kv_select(weights, sl, BUDGET, FIRST, RECENT)
    want_keep, want_kept = _loop.select(weights, lens, BUDGET, FIRST, RECENT)
    assert torch.equal(keep.cpu(), want_keep) and kept.tolist() == kept_len
    new_weights = torch.full((B, hkv, new_table.shape[1] * 64), float("nan"), device="cuda")
    hpc.hpc_kv_compact(c["k_cache"], c["v_cache"], table, keep, kept, new_table, k_scale=c["k_scale"], v_scale=c["v_scale"],
                       weights=weights, weights_out=new_weights)
    for b, m in enumerate(kept_len):
        assert torch.equal(new_weights[b, :, :m], weights[b].gather(1, keep[b, :, :m].long()))

    # a step of drafted tokens behind the kept ones (their keys and values were in the new pages' later slots)
    qd = _tiles.make_q((B, drafts + 1, 8 * hkv, 128), 7)
    steps = _tiles.i32(grown)
    od, ld, _ = hpc.decode(qd, c["k_cache"], c["v_cache"], new_table, steps, c["k_scale"], c["v_scale"])
    keys = []
    for b, m in enumerate(kept_len):
        k = torch.cat([kept_rows(c["k"][0][b], keep[b], m), c["k"][1][b][m:]])
        v = torch.cat([kept_rows(c["v"][0][b], keep[b], m), c["v"][1][b][m:]])
        keys.append(k)
        ref = _tiles.attend(qd[b], k, v, [m + 1 + i for i in range(drafts + 1)])
        assert (od[b].double() - ref[0]).abs().max().item() <= (6e-2 if fp8 else 2e-2)
        assert (ld[b].double() - ref[1]).abs().max().item() <= 1e-3

    # verification, and the weights of the rows that count
    gen = torch.Generator(device="cuda").manual_seed(8)
    target = torch.softmax(2 * torch.randn((B, drafts + 1, 5000), generator=gen, device="cuda"), -1)
    draft = torch.softmax(2 * torch.randn((B, drafts, 5000), generator=gen, device="cuda") + target[:, :drafts].log(), -1)
    drafted = draft.argmax(-1).to(torch.int32)
    accept, sample = torch.rand((B, drafts), generator=gen, device="cuda"), torch.rand(B, generator=gen, device="cuda")
    left = torch.empty_like(steps)
    accepted, tokens = hpc.hpc_verify_drafts(target, drafted, accept, sample, draft_probs=draft, seq_lens=steps, kept_lens=left)
    wa, wt = _loop.verify(target, draft, drafted, accept, sample)
    assert torch.equal(accepted.cpu(), wa) and torch.equal(tokens.cpu(), wt)
    assert torch.equal(left, steps - drafts + accepted)
    before = new_weights.clone()
    counts = accepted + 1
    hpc.hpc_attn_weights(qd, c["k_cache"], new_table, steps, ld, new_weights, k_scale=c["k_scale"], counts=counts)
    rows = [b * (drafts + 1) for b in range(B + 1)]
    want, bound = _loop.attn_weights(qd.view(-1, 8 * hkv, 128), rows, ld.view(-1, 8 * hkv), keys, grown,
                                     torch.nan_to_num(before), counts.tolist(), 0, 1.0, fp8)
    for b, n in enumerate(grown):
        assert ((new_weights[b, :, :n].double() - want[b, :, :n]).abs() <= bound[b, :, :n]).all()
        # each counted row hands out a weight of one per query head
        given = new_weights[b, :, :n].double().sum(-1) - torch.nan_to_num(before)[b, :, :kept_len[b]].double().sum(-1)
        assert ((given - 8 * int(counts[b])).abs() <= 1e-3 * 8 * (drafts + 1)).all()


def test_a_captured_loop():
    """Weights, selection and compaction in one graph: replayed on other lengths, queries and old weights, it does what
    the calls do one by one."""
    hkv = 2
    lens = [700, 129, 300, 64]
    B, starts = 4, [0, 1, 2, 3, 4]
    c = _tiles.make_cache([lens, [BUDGET] * B], hkv, "bf16", 15)
    table, new_table = c["tables"]
    k0, v0 = c["k_cache"].clone(), c["v_cache"].clone()
    q, sl = _tiles.make_q((B, 8 * hkv, 128), 16), _tiles.i32(lens)
    lse = _loop.row_lse(q, starts, c["k"][0], lens)
    weights = torch.rand((B, hkv, table.shape[1] * 64), device="cuda")
    moved = torch.zeros((B, hkv, new_table.shape[1] * 64), device="cuda")
    keep = torch.empty((B, hkv, BUDGET), dtype=torch.int32, device="cuda")
    kept = torch.empty(B, dtype=torch.int32, device="cuda")

    def loop():
        hpc.hpc_attn_weights(q, c["k_cache"], table, sl, lse, weights, decay=0.5)
        hpc.hpc_kv_select(weights, sl, BUDGET, FIRST, RECENT, keep=keep, keep_lens=kept)
        hpc.hpc_kv_compact(c["k_cache"], c["v_cache"], table, keep, kept, new_table, weights=weights, weights_out=moved)

    w0 = weights.clone()
    g = torch.cuda.CUDAGraph()
    loop()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        loop()
    for lens2, seed in ((lens, 17), ([650, 100, 30, 1], 18)):
        w1 = torch.rand(w0.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
        q2 = _tiles.make_q(q.shape, seed)
        lse2 = _loop.row_lse(q2, starts, [k[:n] for k, n in zip(c["k"][0], lens2)], lens2)
        got = []
        for run in (loop, g.replay):
            c["k_cache"].copy_(k0)
            c["v_cache"].copy_(v0)
            moved.zero_()
            keep.fill_(77)
            weights.copy_(w1)
            q.copy_(q2)
            lse.copy_(lse2)
            sl.copy_(_tiles.i32(lens2))
            run()
            torch.cuda.synchronize()
            got.append([x.clone() for x in (weights, keep, kept, moved, c["k_cache"].view(torch.int16), c["v_cache"].view(torch.int16))])
        for x, y in zip(*got):
            assert torch.equal(x, y)
        want, _ = _loop.select(got[0][0], lens2, BUDGET, FIRST, RECENT)
        assert torch.equal(got[0][1].cpu(), want)


def test_tensors_elsewhere():
    """Any one tensor on the host is refused before a launch."""
    c = _tiles.make_cache([[300, 70], [100, 70]], 1, "bf16", 25)
    q, sl = _tiles.make_q((2, 8, 128), 26), _tiles.i32([300, 70])
    lse = torch.zeros((2, 8), device="cuda")
    w = torch.zeros((2, 1, c["tables"][0].shape[1] * 64), device="cuda")
    keep, kept = hpc.hpc_kv_select(w, sl, 100)
    out = torch.zeros((2, 1, 128), device="cuda")
    p = torch.rand((2, 3, 50), device="cuda")
    d = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    u, us = torch.rand((2, 2), device="cuda"), torch.rand(2, device="cuda")
    calls = [
        (hpc.hpc_attn_weights, [q, c["k_cache"], c["tables"][0], sl, lse, w], dict(q_starts=_tiles.i32([0, 1, 2]), counts=_tiles.i32([1, 1]))),
        (hpc.hpc_kv_select, [w, sl, 100], dict(keep=keep, keep_lens=kept)),
        (hpc.hpc_kv_compact, [c["k_cache"], c["v_cache"], c["tables"][0], keep, kept, c["tables"][1]], dict(weights=w, weights_out=out)),
        (hpc.hpc_verify_drafts, [p, d, u, us], dict(draft_probs=p[:, :2].contiguous(), draft_counts=_tiles.i32([2, 2]), seq_lens=sl,
                                                    kept_lens=sl.clone())),
    ]
    for call, args, kw in calls:
        call(*args, **kw)
        for i, x in enumerate(args):
            if isinstance(x, torch.Tensor):
                with pytest.raises(hpc.HpcError, match="tensors on|CUDA device"):
                    call(*args[:i], x.cpu(), *args[i + 1:], **kw)
        for n, x in kw.items():
            with pytest.raises(hpc.HpcError, match="tensors on"):
                call(*args, **dict(kw, **{n: x.cpu()}))
    torch.cuda.synchronize()


def test_another_stream_than_the_current_one():
    """Outputs allocated by a call belong to the call's stream, also where that is not the current one."""
    w = torch.rand((3, 2, 2000), device="cuda")
    lens = [2000, 900, 10]
    sl = _tiles.i32(lens)
    want, kept = _loop.select(w, lens, 300, 2, 20)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        keep, kl = hpc.hpc_kv_select(w, sl, 300, 2, 20, stream=s)
        junk = [torch.full((3, 2, 300), 9, dtype=torch.int32, device="cuda") for _ in range(4)]  # on the current stream
        s.synchronize()
        assert torch.equal(keep.cpu(), want) and torch.equal(kl.cpu(), kept)
        del junk


def test_limits():
    """The most drafts, and a request whose rows' log-sum-exps are all -inf."""
    B, n, V = 3, 31, 300
    gen = torch.Generator(device="cuda").manual_seed(31)
    p = torch.softmax(torch.randn((B, n + 1, V), generator=gen, device="cuda"), -1)
    drafted = torch.randint(0, V, (B, n), generator=gen, device="cuda", dtype=torch.int32)
    u, us = torch.zeros((B, n), device="cuda"), torch.rand(B, generator=gen, device="cuda")
    acc, tok = hpc.hpc_verify_drafts(p, drafted, u, us, draft_probs=p[:, :n].contiguous())
    wa, wt = _loop.verify(p, p[:, :n], drafted, u, us)
    assert torch.equal(acc.cpu(), wa) and torch.equal(tok.cpu(), wt) and acc.tolist() == [n] * B
    c = _tiles.make_cache([[200]], 1, "bf16", 35)
    q = _tiles.make_q((2, 8, 128), 36)
    w = torch.ones((1, 1, 256), device="cuda")
    hpc.hpc_attn_weights(q, c["k_cache"], c["tables"][0], _tiles.i32([200]), torch.full((2, 8), -math.inf, device="cuda"), w,
                         q_starts=_tiles.i32([0, 2]), decay=0.25)
    assert (w[0, 0, :198] == 0.25).all() and (w[0, 0, 198:200] == 0).all() and (w[0, 0, 200:] == 1).all()


def test_calls_at_once():
    """The operators on two streams, over and over, beside one another: each gives what it gives alone."""
    def problem(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        lens = [3000 - 700 * seed, 129, 2000, 40 + seed]
        c = _tiles.make_cache([lens], 2, "bf16", seed)
        q = _tiles.make_q((4, 16, 128), seed + 9)
        lse = 3.0 + torch.rand((4, 16), generator=gen, device="cuda")
        width = c["tables"][0].shape[1] * 64
        p = torch.softmax(2.0 * torch.randn((4, 3, 9001), generator=gen, device="cuda"), -1)
        d = torch.randint(0, 9001, (4, 2), generator=gen, device="cuda", dtype=torch.int32)
        u, us = torch.rand((4, 2), generator=gen, device="cuda"), torch.rand(4, generator=gen, device="cuda")
        sl, w = _tiles.i32(lens), torch.empty((4, 2, width), device="cuda")

        def run(stream):
            w.zero_()
            hpc.hpc_attn_weights(q, c["k_cache"], c["tables"][0], sl, lse, w, stream=stream)
            keep, kl = hpc.hpc_kv_select(w, sl, 500, 4, 32, stream=stream)
            acc, tok = hpc.hpc_verify_drafts(p, d, u, us, stream=stream)
            return [w.clone(), keep, kl, acc, tok]
        return run
    runs = [problem(0), problem(1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    want = []
    for run, s in zip(runs, streams):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            want.append(run(s))
        torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for _ in range(3):
            for run, s in zip(runs, streams):
                with torch.cuda.stream(s):
                    got.append(run(s))
        torch.cuda.synchronize()
        for i, g in enumerate(got):
            assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
