"""What the decode loop's operators between two attention steps are measured on: the attention weight
that cached tokens received (`hpc_attn_weights`), the choice of the tokens that stay (`hpc_kv_select`),
their move into new pages (`hpc_kv_compact`), and the verification of drafted tokens
(`hpc_verify_drafts`).

`run` computes each operator in its plain form, from elementary torch operations in 32 bits (64 where the
place of a border counts), or, with `own` set, by the calls that a user makes of the library. `exact` gives
the same outputs from the operators' definitions in 64 bits.

Lengths are texts: "37,128" lists values, "512x4" repeats one, "lu:LO:HI:N:SEED" draws N values
log-uniformly from [LO, HI]; the parts are joined by commas.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE, DIM, GROUP = 64, 128, 8
E4M3_MAX = 448.0


def lengths(text):
    """The list of lengths that a text stands for."""
    got = []
    for part in text.split(","):
        if part.startswith("lu:"):
            lo, hi, n, seed = (int(x) for x in part[3:].split(":"))
            r = random.Random(seed)
            got += [min(hi, max(lo, int(math.exp(r.uniform(math.log(lo), math.log(hi)))))) for _ in range(n)]
        elif "x" in part:
            value, n = part.split("x")
            got += [int(value)] * int(n)
        else:
            got.append(int(part))
    return got


# ---------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of the smallest batch, one KV head: launches and latency
        dict(name="weights of four short requests", op="weights", hkv=1, kv="bf16", new="1x4", lens="37,128,300,1000", window=0, decay=1.0,
             counted=False),
        # the weights of one decode step of a mixed batch at the full head shape: K is read once
        dict(name="weights of a decode step", op="weights", hkv=8, kv="bf16", new="1x64", lens="lu:128:65536:64:3", window=0, decay=1.0,
             counted=False),
        # four drafted tokens each over a quantised cache, only the accepted rows counted, older weight fading
        dict(name="weights of accepted rows", op="weights", hkv=8, kv="e4m3", new="4x48", lens="lu:512:65536:48:4", window=0, decay=0.96875,
             counted=True),
        # the last 32 queries of the prompts' last pieces look back over the whole prompts
        dict(name="weights of prompt windows", op="weights", hkv=8, kv="bf16", new="512x7,100,33,501", lens="lu:2048:32768:10:5", window=32,
             decay=0.0, counted=False),
        # four short requests, two of which are within their budget
        dict(name="select in short requests", op="select", hkv=1, lens="37,128,300,1000", budget=160, first=4, recent=32),
        # a mixed batch brought down to 2048 tokens per head
        dict(name="select in a mixed batch", op="select", hkv=8, lens="lu:128:65536:64:3", budget=2048, first=4, recent=256),
        # one very long document: few rows, many tokens
        dict(name="select in one long request", op="select", hkv=8, lens="262144", budget=16384, first=16, recent=1024),
        # the kept tokens of four short requests into new pages
        dict(name="compact short requests", op="compact", hkv=1, kv="bf16", lens="37,128,300,1000", budget=160, moved=True),
        # a mixed batch moved into the pages that it keeps, its weights with it
        dict(name="compact a mixed batch", op="compact", hkv=8, kv="bf16", lens="lu:1024:16384:64:6", budget=2048, moved=True),
        # the same on a quantised cache, longer budget
        dict(name="compact a quantised batch", op="compact", hkv=8, kv="e4m3", lens="lu:4096:32768:32:7", budget=4096, moved=True),
        # one conversation with three drafted tokens
        dict(name="verify one request", op="verify", batch=1, drafts=3, vocab=32000, type="f32", given=True),
        # a full batch with five drafted tokens each
        dict(name="verify a full batch", op="verify", batch=256, drafts=5, vocab=131072, type="f32", given=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _text(values):
    return ",".join(str(v) for v in values)


def draw(rng):
    op = rng.choice(["weights", "weights", "weights", "select", "compact", "verify"])
    hkv, kv = rng.choice([1, 2, 3, 4, 8]), rng.choice(["bf16", "e4m3"])
    if op == "verify":
        batch, drafts = _log(rng, 1, 128), rng.choice([0, 1, 2, 3, 5, 7])
        return dict(op=op, batch=batch, drafts=drafts, vocab=_log(rng, 1000, 131072), type=rng.choice(["f32", "f32", "bf16"]),
                    given=rng.random() < 0.75)
    if op == "weights":
        budget = 4000000  # tokens x rows over all requests: under the largest listed case's
        new, lens = [], []
        kind = rng.choice(["decode", "drafts", "window"])
        window = 0 if kind != "window" else _log(rng, 4, 100)
        rows = dict(decode=1, drafts=rng.choice([2, 3, 5, 8]), window=0)[kind]
        for _ in range(_log(rng, 1, 64)):
            total = _log(rng, 1, 40000)
            n = rows if rows else _log(rng, 1, min(total, 512))
            seen = min(n, window) if window else n
            if seen * total <= budget:
                budget -= seen * total
                new.append(n)
                lens.append(total)
        if not new:
            new, lens = [3], [97]
        return dict(op=op, hkv=hkv, kv=kv, new=_text(new), lens=_text(lens), window=window, decay=rng.choice([0.0, 1.0, 1.0, 0.875]),
                    counted=kind == "drafts")
    lens = [_log(rng, 1, 32768 if op == "select" else 12000) for _ in range(_log(rng, 1, 48))]
    budget = _log(rng, 64, 4096)
    if op == "select":
        first, recent = rng.choice([0, 1, 4, 30]), rng.randrange(0, 34)
        return dict(op=op, hkv=hkv, lens=_text(lens), budget=budget, first=first, recent=recent)
    return dict(op=op, hkv=hkv, kv=kv, lens=_text(lens), budget=budget, moved=rng.random() < 0.5)


# ---------------------------------------------------------------------------- the inputs

def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _cache(pages, hkv, kv, gen):
    """One paged cache [pages, 64, hkv, 128] and its scales [pages, hkv, 64] (None for bf16)."""
    if kv == "bf16":
        return _normal((pages, PAGE, hkv, DIM), gen), None
    x = torch.randn((pages, PAGE, hkv, DIM), generator=gen, device="cuda", dtype=torch.float32)
    scale = x.abs().amax(dim=-1) / E4M3_MAX
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale.permute(0, 2, 1).contiguous()


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    got = [0]
    for n in counts:
        got.append(got[-1] + n)
    return got


def _tables(lists_of_lens, rng):
    """One page table for each list of lengths, all from one shuffled pool; and the pool's size."""
    need = [[-(-n // PAGE) for n in lens] for lens in lists_of_lens]
    pages = list(range(sum(sum(x) for x in need) + 3))
    rng.shuffle(pages)
    tables, at = [], 0
    for counts in need:
        table = torch.full((len(counts), max(1, max(counts))), -1, dtype=torch.int32)
        for b, n in enumerate(counts):
            table[b, :n] = torch.tensor(pages[at:at + n], dtype=torch.int32)
            at += n
        tables.append(table.to("cuda"))
    return tables, len(pages)


def _received(shape, gen):
    """Weights as cached tokens collect them: a few large ones, most small, a tenth never looked at."""
    x = torch.exp(2.0 * torch.randn(shape, generator=gen, device="cuda") - 6.0)
    return torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.1, 0.0, x)


def _spans(case):
    """The counted rows [lo, hi) of each sequence; an accepted count takes the place of all rows where the case says so."""
    spans = []
    for b, n in enumerate(lengths(case["new"])):
        hi = 1 + (b * 7 + 3) % n if case["counted"] else n
        spans.append((max(0, hi - case["window"]) if case["window"] else 0, hi))
    return spans


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    s = dict(op=case["op"])
    if case["op"] == "verify":
        batch, drafts, vocab = case["batch"], case["drafts"], case["vocab"]
        kind = torch.float32 if case["type"] == "f32" else torch.bfloat16
        # what the target knows and the draft roughly does
        logits = torch.randn((batch, drafts + 1, vocab), generator=gen, device="cuda").mul_(3.0)
        target = torch.softmax(logits, dim=-1)
        logits = logits[:, :drafts]
        logits.add_(torch.randn((batch, drafts, vocab), generator=gen, device="cuda"), alpha=0.7)
        draft = torch.softmax(logits, dim=-1)
        del logits
        u = torch.rand((batch, drafts, 1), generator=gen, device="cuda", dtype=torch.float64)
        tokens = torch.empty((batch, drafts), dtype=torch.int64, device="cuda")
        for b in range(batch):  # drawn from the draft
            c = torch.cumsum(draft[b].double(), dim=-1)
            tokens[b] = torch.searchsorted(c, u[b] * c[:, -1:], right=True).squeeze(-1).clamp_(max=vocab - 1)
        s.update(target=target.to(kind), draft=draft.to(kind) if case["given"] else None, drafted=tokens.to(torch.int32),
                 accept=torch.rand((batch, drafts), generator=gen, device="cuda"),
                 sample=torch.rand((batch,), generator=gen, device="cuda"))
        return s
    lens, hkv = lengths(case["lens"]), case["hkv"]
    s.update(host_lens=lens, seq_lens=_i32(lens))
    width = -(-max(lens) // PAGE) * PAGE
    if case["op"] == "select":
        s.update(weights=_received((len(lens), hkv, width), gen), budget=case["budget"], first=case["first"], recent=case["recent"])
        return s
    if case["op"] == "compact":
        kept = [min(n, case["budget"]) for n in lens]
        tables, pool = _tables([lens, kept], rng)
        s.update(page_table=tables[0], new_table=tables[1], host_kept=kept, kept=_i32(kept))
        keep = torch.full((len(lens), hkv, case["budget"]), -1, dtype=torch.int32, device="cuda")
        for b, (n, m) in enumerate(zip(lens, kept)):
            some = torch.rand((hkv, n), generator=gen, device="cuda").argsort(dim=-1)[:, :m]
            keep[b, :, :m] = some.sort(dim=-1).values.to(torch.int32)
        s["keep"] = keep
        s["weights"] = _received((len(lens), hkv, width), gen) if case["moved"] else None
        s["new_weights"] = torch.zeros((len(lens), hkv, tables[1].shape[1] * PAGE), device="cuda") if case["moved"] else None
        s["k_cache"], s["k_scale"] = _cache(pool, hkv, case["kv"], gen)
        s["v_cache"], s["v_scale"] = _cache(pool, hkv, case["kv"], gen)
        return s
    tables, pool = _tables([lens], rng)
    new, spans = lengths(case["new"]), _spans(case)
    s.update(page_table=tables[0], host_new=new, q_starts=_i32(_starts(new)), host_spans=spans, window=case["window"], decay=case["decay"],
             counts=_i32([hi for _, hi in spans]) if case["counted"] else None)
    s["k_cache"], s["k_scale"] = _cache(pool, hkv, case["kv"], gen)
    s["q"] = _normal((sum(new), GROUP * hkv, DIM), gen)
    s["old"] = _received((len(lens), hkv, tables[0].shape[1] * PAGE), gen)
    s["weights"] = s["old"].clone()
    # the attention call's log-sum-exps (of the rows that count; no other is looked at)
    s["lse"] = torch.zeros((sum(new), GROUP * hkv), device="cuda")
    at = 0
    for b, (n, total, (lo, hi)) in enumerate(zip(new, lens, spans)):
        scores = _scores(s, b, at, n, total, lo, hi)
        s["lse"][at + lo:at + hi] = torch.logsumexp(scores, dim=-1).permute(2, 0, 1).reshape(hi - lo, hkv * GROUP)
        at += n
    return s


# ---------------------------------------------------------------------------- the plain forms

def _keys(s, b, total):
    """The keys of a request in 32 bits, [total, hkv, 128]."""
    pages = s["page_table"][b, :-(-total // PAGE)].long()
    if s["k_scale"] is None:
        x = s["k_cache"][pages].float()
    else:
        x = s["k_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * s["k_scale"][pages].transpose(1, 2).unsqueeze(-1)
    return x.flatten(0, 1)[:total]


def _scores(s, b, at, n, total, lo, hi):
    """Scores of the counted rows of one sequence with all its keys, -inf where a row does not see the token:
    [hkv, 8, rows, total]."""
    k = _keys(s, b, total).permute(1, 2, 0)
    hkv = k.shape[0]
    q = s["q"][at + lo:at + hi].float().view(hi - lo, hkv, GROUP, DIM).permute(1, 2, 0, 3)
    scores = torch.matmul(q.reshape(hkv, -1, DIM) / math.sqrt(DIM), k).view(hkv, GROUP, hi - lo, total)
    last = torch.arange(lo, hi, device="cuda").unsqueeze(1) + (total - n)
    return scores.masked_fill_(torch.arange(total, device="cuda") > last, -math.inf)


def _weights(s):
    w = s["weights"]
    at = 0
    for b, (n, total, (lo, hi)) in enumerate(zip(s["host_new"], s["host_lens"], s["host_spans"])):
        scores = _scores(s, b, at, n, total, lo, hi)
        hkv = scores.shape[0]
        lse = s["lse"][at + lo:at + hi].view(hi - lo, hkv, GROUP, 1).permute(1, 2, 0, 3)
        # a row that sees nothing has the lse -inf, and no weight
        got = torch.where(lse > -math.inf, scores.sub_(lse).exp_(), 0.0).sum(dim=(1, 2))
        older = max(0, total - n)
        if s["decay"] != 0.0:
            got[:, :older] += s["decay"] * w[b, :, :older]
        w[b, :, :total] = got
        at += n
    return w


def _select(s):
    w, budget, first, recent = s["weights"], s["budget"], s["first"], s["recent"]
    keep = torch.full((w.shape[0], w.shape[1], budget), -1, dtype=torch.int32, device="cuda")
    for b, total in enumerate(s["host_lens"]):
        if total <= budget:
            keep[b, :, :total] = torch.arange(total, dtype=torch.int32, device="cuda")
            continue
        order = torch.sort(w[b, :, first:total - recent], dim=-1, descending=True, stable=True).indices + first
        chosen = torch.zeros((w.shape[1], total), dtype=torch.bool, device="cuda")
        chosen[:, :first] = True
        chosen[:, total - recent:] = True
        chosen.scatter_(1, order[:, :budget - first - recent], True)
        keep[b] = chosen.nonzero()[:, 1].view(w.shape[1], budget).to(torch.int32)
    return keep, s["seq_lens"].clamp(max=budget)


def _compact(s):
    pairs = ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]))
    for b, m in enumerate(s["host_kept"]):
        t = s["keep"][b, :, :m].long()                                       # [hkv, m]
        h = torch.arange(t.shape[0], device="cuda").unsqueeze(1)
        j = torch.arange(m, device="cuda").unsqueeze(0)
        src, dst = s["page_table"][b][t // PAGE].long(), s["new_table"][b][j // PAGE].long()
        for cache, scale in pairs:
            x = cache if scale is None else cache.view(torch.uint8)
            x[dst, j % PAGE, h] = x[src, t % PAGE, h]
            if scale is not None:
                scale[dst, h, j % PAGE] = scale[src, h, t % PAGE]
        if s["weights"] is not None:
            s["new_weights"][b, :, :m] = s["weights"][b].gather(1, t)


def _verify(s):
    p, q, drafted = s["target"], s["draft"], s["drafted"].long()
    batch, drafts = drafted.shape
    p_at = p[:, :drafts].gather(2, drafted.unsqueeze(-1)).squeeze(-1).double()
    q_at = torch.ones_like(p_at) if q is None else q.gather(2, drafted.unsqueeze(-1)).squeeze(-1).double()
    accepted = (s["accept"].double() * q_at < p_at).to(torch.int32).cumprod(dim=1).sum(dim=1)
    rows = torch.arange(batch, device="cuda")
    rest = p[rows, accepted].double()
    if drafts:
        refused = accepted < drafts
        at = accepted.clamp(max=drafts - 1)
        if q is None:
            rest[rows, drafted[rows, at]] *= (~refused).double()
        else:
            rest = (rest - q[rows, at].double() * refused.unsqueeze(1)).clamp_(min=0.0)
    sums = torch.cumsum(rest, dim=-1)
    token = torch.searchsorted(sums, s["sample"].double().unsqueeze(1) * sums[:, -1:], right=True).squeeze(1)
    out = torch.full((batch, drafts + 1), -1, dtype=torch.int64, device="cuda")
    place = torch.arange(drafts, device="cuda")
    out[:, :drafts] = torch.where(place < accepted.unsqueeze(1), drafted, -1)
    out[rows, accepted] = token
    return accepted.to(torch.int32), out.to(torch.int32)


def run(s):
    if own:
        import load_balanced_paged_02_gb300 as hpc
    if s["op"] == "weights":
        if own:
            hpc.hpc_attn_weights(s["q"], s["k_cache"], s["page_table"], s["seq_lens"], s["lse"], s["weights"], q_starts=s["q_starts"],
                                 k_scale=s["k_scale"], counts=s["counts"], window=s["window"], decay=s["decay"])
            return dict(weights=s["weights"])
        return dict(weights=_weights(s))
    if s["op"] == "select":
        if own:
            keep, kept = hpc.hpc_kv_select(s["weights"], s["seq_lens"], s["budget"], num_first=s["first"], num_recent=s["recent"])
        else:
            keep, kept = _select(s)
        return dict(keep=keep, kept=kept)
    if s["op"] == "compact":
        if own:
            hpc.hpc_kv_compact(s["k_cache"], s["v_cache"], s["page_table"], s["keep"], s["kept"], s["new_table"], k_scale=s["k_scale"],
                               v_scale=s["v_scale"], weights=s["weights"], weights_out=s["new_weights"])
        else:
            _compact(s)
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"], weights=s["new_weights"])
    if own:
        accepted, tokens = hpc.hpc_verify_drafts(s["target"], s["drafted"], s["accept"], s["sample"], draft_probs=s["draft"])
    else:
        accepted, tokens = _verify(s)
    return dict(accepted=accepted, tokens=tokens)


# ---------------------------------------------------------------------------- work, and the same in 64 bits

def work(case):
    if case["op"] == "verify":
        # a row of each, and the drafted tokens' entries
        size = 4 if case["type"] == "f32" else 2
        rows = 2 if case["given"] and case["drafts"] else 1
        return dict(bytes=case["batch"] * (case["vocab"] * size * rows + case["drafts"] * (2 * size + 12) + 8),
                    flops=case["batch"] * case["vocab"] * 2 * rows)
    hkv, lens = case["hkv"], lengths(case["lens"])
    if case["op"] == "weights":
        row = DIM * 2 if case["kv"] == "bf16" else DIM + 4
        kept = 4 if case["decay"] == 0.0 else 8
        spans = _spans(case)
        pairs = sum((hi - lo) * n for n, (lo, hi) in zip(lens, spans))
        return dict(bytes=hkv * (sum(lens) * (row + kept) + sum(hi - lo for lo, hi in spans) * GROUP * (2 * DIM + 4)),
                    flops=2 * DIM * GROUP * hkv * pairs)
    kept = sum(min(n, case["budget"]) for n in lens)
    if case["op"] == "select":
        return dict(bytes=4 * hkv * (sum(lens) + case["budget"] * len(lens)), flops=hkv * sum(lens))
    row = 2 * DIM * 2 if case["kv"] == "bf16" else 2 * DIM + 8
    return dict(bytes=hkv * kept * (2 * row + 4 + (8 if case["moved"] else 0)), flops=hkv * kept)


def _exact_weights(case, s):
    w = s["old"].double()
    at = 0
    for b, (n, total, (lo, hi)) in enumerate(zip(lengths(case["new"]), lengths(case["lens"]), _spans(case))):
        t = torch.arange(total, device="cuda")
        page, slot = s["page_table"][b].long()[t // PAGE], t % PAGE
        for h in range(case["hkv"]):
            if s["k_scale"] is None:
                k = s["k_cache"][page, slot, h].double()
            else:
                k = s["k_cache"].view(torch.uint8)[page, slot, h].view(torch.float8_e4m3fn).double() * s["k_scale"][page, h, slot].double().unsqueeze(-1)
            got = torch.zeros(total, dtype=torch.float64, device="cuda")
            for i in range(lo, hi):
                seen = max(0, total - n + i + 1)
                q = s["q"][at + i, GROUP * h:GROUP * (h + 1)].double()
                lse = s["lse"][at + i, GROUP * h:GROUP * (h + 1)].double()
                e = torch.exp((q @ k[:seen].T) / math.sqrt(DIM) - lse.unsqueeze(1))
                got[:seen] += e[lse > -math.inf].sum(dim=0)
            old = torch.where(t < total - n, w[b, h, :total] * case["decay"], 0.0) if case["decay"] else 0.0
            w[b, h, :total] = got + old
        at += n
    return w


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "weights":
        return dict(weights=_exact_weights(case, s))
    if case["op"] == "select":
        w = s["weights"].double().cpu().numpy()
        budget, first, recent = case["budget"], case["first"], case["recent"]
        keep = torch.full((w.shape[0], w.shape[1], budget), -1, dtype=torch.int64)
        kept = []
        for b, total in enumerate(lengths(case["lens"])):
            kept.append(min(total, budget))
            for h in range(w.shape[1]):
                if total <= budget:
                    keep[b, h, :total] = torch.arange(total)
                    continue
                # larger weights first, of equal ones the earlier token
                middle = np.arange(first, total - recent)
                chosen = middle[np.lexsort((middle, -w[b, h, first:total - recent]))][:budget - first - recent]
                both = np.concatenate((np.arange(first), chosen, np.arange(total - recent, total)))
                keep[b, h] = torch.from_numpy(np.sort(both))
        return dict(keep=keep.to("cuda"), kept=torch.tensor(kept, device="cuda"))
    if case["op"] == "compact":
        old = {n: s[n].clone() if s[n] is not None else None for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
        got = {n: x.double() if x is not None else None for n, x in old.items()}
        got["weights"] = s["new_weights"].double() if case["moved"] else None
        for b, m in enumerate(s["host_kept"]):
            j = torch.arange(m, device="cuda")
            to, slot = s["new_table"][b].long()[j // PAGE], j % PAGE
            for h in range(case["hkv"]):
                t = s["keep"][b, h, :m].long()
                page, at = s["page_table"][b].long()[t // PAGE], t % PAGE
                for n in ("k", "v"):
                    cache = old[n + "_cache"]
                    if old[n + "_scale"] is not None:
                        got[n + "_scale"][to, h, slot] = old[n + "_scale"][page, h, at].double()
                        got[n + "_cache"][to, slot, h] = cache.view(torch.uint8)[page, at, h].view(cache.dtype).double()
                    else:
                        got[n + "_cache"][to, slot, h] = cache[page, at, h].double()
                if case["moved"]:
                    got["weights"][b, h, :m] = s["weights"][b, h][t].double()
        return got
    accepted, tokens = [], []
    drafts = case["drafts"]
    for b in range(case["batch"]):
        out, r = [], 0
        drafted, u = s["drafted"][b].tolist(), s["accept"][b].tolist()
        while r < drafts:
            p = float(s["target"][b, r, drafted[r]])
            q = float(s["draft"][b, r, drafted[r]]) if case["given"] else 1.0
            if not u[r] * q < p:
                break
            out.append(drafted[r])
            r += 1
        rest = s["target"][b, r].double()
        if r < drafts and case["given"]:
            rest = torch.clamp(rest - s["draft"][b, r].double(), min=0.0)
        elif r < drafts:
            rest[drafted[r]] = 0.0
        sums = rest.cumsum(0)
        above = sums > float(s["sample"][b]) * float(sums[-1])
        out.append(int(above.to(torch.uint8).argmax()))
        accepted.append(r)
        tokens.append(out + [-1] * (drafts + 1 - len(out)))
    return dict(accepted=torch.tensor(accepted, device="cuda"), tokens=torch.tensor(tokens, device="cuda"))
