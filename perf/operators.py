"""What the prompt-side operators of the library are measured on: attention over packed prompts
(`prefill`), decode for batches that share long prefixes (`decode_shared_prefix`), and the paged
cache written and read back on its own (`hpc_kv_write`, `hpc_kv_read`).

`run` computes each operator in its plain form, from elementary torch operations in 32 bits, or,
with `own` set, by the calls that a user makes of the library. `exact` gives the same outputs from
the operators' definitions in 64 bits.

Lengths are texts: "37,128" lists values, "512x4" repeats one, "lu:LO:HI:N:SEED" draws N values
log-uniformly from [LO, HI]; the parts are joined by commas.
"""
import math
import random

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
        # four short prompts of the smallest batch, one KV head: a step whose time is launches and latency
        dict(name="prefill four short prompts", op="prefill", hkv=1, kv="bf16", new="37,128,300,1000", lens="37,128,300,1000"),
        # one document of 8192 tokens at the full head shape: the tensor cores' case
        dict(name="prefill one long prompt", op="prefill", hkv=8, kv="bf16", new="8192", lens="8192"),
        # a packed batch of prompts of very different lengths
        dict(name="prefill packed prompts", op="prefill", hkv=8, kv="bf16", new="lu:100:6000:12:5", lens="lu:100:6000:12:5"),
        # one engine step on a quantised cache: 512-token pieces of four long prompts beside 28 requests that
        # decode one token each
        dict(name="prefill pieces and decode", op="prefill", hkv=8, kv="e4m3", new="512x3,501,1x28", lens="lu:4096:32768:4:7,lu:512:16384:28:8"),
        # eight requests of a small model behind one system prompt
        dict(name="prefix small batch", op="prefix", hkv=1, kv="bf16", q_len=1, groups="8", prefixes="1000", lens="37x3,128,129,300,1,0"),
        # 64 conversations behind a long system prompt
        dict(name="prefix of 8192 tokens", op="prefix", hkv=8, kv="bf16", q_len=1, groups="64", prefixes="8192", lens="lu:32:2048:64:3"),
        # many questions about one very long document, quantised cache
        dict(name="prefix of 65536 tokens", op="prefix", hkv=8, kv="e4m3", q_len=1, groups="128", prefixes="65536", lens="lu:16:1024:128:4"),
        # several prefixes in one batch, requests without company among them, four new tokens each to verify
        dict(name="prefixes of four groups", op="prefix", hkv=8, kv="bf16", q_len=4, groups="16,5,1,42", prefixes="4096,1000,20000,333", lens="lu:64:4096:64:6"),
        # one decode step's keys and values, sliced out of the projection's output, into a quantised cache
        dict(name="write 64 tokens", op="write", hkv=8, kv="e4m3", tokens=64, padded=3),
        # a prompt's keys and values into a quantised cache
        dict(name="write 8192 tokens", op="write", hkv=8, kv="e4m3", tokens=8192, padded=0),
        # four short requests copied out of a paged cache
        dict(name="read four short requests", op="read", hkv=1, kv="bf16", lens="37,128,300,1000", first="0,64,5,131"),
        # a batch's history brought back from a quantised cache to bf16
        dict(name="read a long batch", op="read", hkv=8, kv="e4m3", lens="lu:512:32768:24:9", first="0x24"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _text(values):
    return ",".join(str(v) for v in values)


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefix", "prefix", "write", "read"])
    hkv, kv = rng.choice([1, 2, 3, 4, 8]), rng.choice(["bf16", "e4m3"])
    if op == "prefill":
        budget = 64 * 8192 * 8192 // (8 * hkv)  # of (new tokens x length), the largest listed case's
        new, lens = [], []
        for _ in range(_log(rng, 1, 24)):
            total = _log(rng, 1, 8192)
            n = total if rng.random() < 0.5 else _log(rng, 1, min(total, 700))
            if n * total <= budget:
                budget -= n * total
                new.append(n)
                lens.append(total)
        if not new:
            new, lens = [33], [97]
        return dict(op=op, hkv=hkv, kv=kv, new=_text(new), lens=_text(lens))
    if op == "prefix":
        groups = [_log(rng, 1, 64) for _ in range(rng.choice([1, 1, 2, 3]))]
        hi = _log(rng, 16, 1500)
        return dict(op=op, hkv=hkv, kv=kv, q_len=rng.choice([1, 1, 1, 2, 3, 6]), groups=_text(groups),
                    prefixes=_text([_log(rng, 1, 24000) for _ in groups]),
                    lens="lu:8:%d:%d:%d" % (hi, sum(groups), rng.randrange(1 << 20)))
    if op == "write":
        tokens = _log(rng, 1, 8192)
        return dict(op=op, hkv=hkv, kv=kv, tokens=tokens, padded=rng.randrange(0, max(1, tokens // 8)))
    lens = [_log(rng, 1, 20000) for _ in range(_log(rng, 1, 24))]
    return dict(op=op, hkv=hkv, kv=kv, lens=_text(lens), first=_text([rng.randrange(0, 300) for _ in lens]))


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    hkv, kv = case["hkv"], case["kv"]
    s = dict(op=case["op"])
    if case["op"] == "write":
        tokens = case["tokens"]
        pool = -(-tokens // PAGE) + 3
        slots = rng.sample(range(pool * PAGE), tokens)
        for t in rng.sample(range(tokens), case["padded"]):
            slots[t] = -1
        live = [t for t in range(tokens) if slots[t] >= 0]
        qkv = _normal((tokens, (GROUP + 2) * hkv, DIM), gen)
        s.update(k=qkv[:, GROUP * hkv:(GROUP + 1) * hkv], v=qkv[:, (GROUP + 1) * hkv:], slots=_i32(slots),
                 live=torch.tensor(live, device="cuda"), live_slots=torch.tensor([slots[t] for t in live], device="cuda"))
        s["k_cache"], s["k_scale"] = _cache(pool, hkv, kv, gen)
        s["v_cache"], s["v_scale"] = _cache(pool, hkv, kv, gen)
        return s
    lens = lengths(case["lens"])
    lists = [lens]
    if case["op"] == "prefix":
        s["host_groups"], s["host_prefixes"] = lengths(case["groups"]), lengths(case["prefixes"])
        lists.append(s["host_prefixes"])
        s.update(group_starts=_i32(_starts(s["host_groups"])), prefix_lens=_i32(s["host_prefixes"]))
    if case["op"] == "read":
        first = lengths(case["first"])
        lists = [[n + f for n, f in zip(lens, first)]]
        s.update(first=_i32(first), host_first=first, out_starts=_i32(_starts(lens)))
    tables, pool = _tables(lists, rng)
    s.update(host_lens=lens, seq_lens=_i32(lens), page_table=tables[0])
    s["k_cache"], s["k_scale"] = _cache(pool, hkv, kv, gen)
    s["v_cache"], s["v_scale"] = _cache(pool, hkv, kv, gen)
    if case["op"] == "prefill":
        s["host_new"] = lengths(case["new"])
        s.update(q=_normal((sum(s["host_new"]), GROUP * hkv, DIM), gen), q_starts=_i32(_starts(s["host_new"])))
    if case["op"] == "prefix":
        s["prefix_table"] = tables[1]
        q_len = case["q_len"]
        shape = (len(lens), GROUP * hkv, DIM) if q_len == 1 else (len(lens), q_len, GROUP * hkv, DIM)
        s["q"] = _normal(shape, gen)
    return s


# ---------------------------------------------------------------------------- the plain forms

def _values(cache, scale, pages):
    """The values of some pages of a cache in 32 bits, [..., 64 x pages, hkv, 128]."""
    x = cache.view(torch.uint8)[pages].view(cache.dtype) if scale is not None else cache[pages]
    x = x.float()
    if scale is not None:
        x = x * scale[pages].transpose(-1, -2).unsqueeze(-1)
    return x.flatten(-4, -3)


def _table_rows(table, lens):
    return table[:, :max(1, -(-max(lens) // PAGE))].clamp(min=0).long()


def _prefill(s):
    """Each sequence on its own: scores of its new tokens with all its keys, causal softmax, values."""
    hkv = s["k_cache"].shape[2]
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    at = 0
    for b, (n, total) in enumerate(zip(s["host_new"], s["host_lens"])):
        pages = s["page_table"][b, :-(-total // PAGE)].long()
        k = _values(s["k_cache"], s["k_scale"], pages)[:total].permute(1, 2, 0)          # [hkv, 128, total]
        v = _values(s["v_cache"], s["v_scale"], pages)[:total].permute(1, 0, 2)          # [hkv, total, 128]
        q = s["q"][at:at + n].float().view(n, hkv, GROUP, DIM).permute(1, 2, 0, 3)        # [hkv, 8, n, 128]
        scores = torch.matmul(q.reshape(hkv, GROUP * n, DIM) / math.sqrt(DIM), k).view(hkv, GROUP, n, total)
        row = torch.arange(n, device="cuda").unsqueeze(1) + (total - n)
        scores.masked_fill_(torch.arange(total, device="cuda") > row, -math.inf)
        top = scores.amax(dim=-1, keepdim=True)
        p = scores.sub_(top).exp_()
        sums = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p.view(hkv, GROUP * n, total), v).view(hkv, GROUP, n, DIM) / sums
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, hkv * GROUP, DIM).to(torch.bfloat16)
        lse[at:at + n] = (top + sums.log()).squeeze(-1).permute(2, 0, 1).reshape(n, hkv * GROUP)
        at += n
    return out, lse


def _prefix(s):
    """Each group's queries with the prefix's keys as one product, with the padded suffixes as another, one softmax
    over both."""
    q = s["q"] if s["q"].dim() == 4 else s["q"].unsqueeze(1)
    batch, q_len, hq, _ = q.shape
    hkv = hq // GROUP
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    b0 = 0
    for g, (count, plen) in enumerate(zip(s["host_groups"], s["host_prefixes"])):
        b1 = b0 + count
        qg = q[b0:b1].float().view(count, q_len, hkv, GROUP, DIM).permute(2, 0, 1, 3, 4) / math.sqrt(DIM)
        pages = s["prefix_table"][g, :-(-plen // PAGE)].long()
        kp = _values(s["k_cache"], s["k_scale"], pages)[:plen].permute(1, 2, 0)
        vp = _values(s["v_cache"], s["v_scale"], pages)[:plen].permute(1, 0, 2)
        rows = _table_rows(s["page_table"][b0:b1], s["host_lens"][b0:b1])
        ks = _values(s["k_cache"], s["k_scale"], rows).permute(2, 0, 3, 1)                # [hkv, count, 128, padded]
        vs = _values(s["v_cache"], s["v_scale"], rows).permute(2, 0, 1, 3)                # [hkv, count, padded, 128]
        padded = ks.shape[-1]
        sp = torch.matmul(qg.reshape(hkv, -1, DIM), kp).view(hkv, count, q_len * GROUP, plen)
        ss = torch.matmul(qg.reshape(hkv, count, q_len * GROUP, DIM), ks)
        last = s["seq_lens"][b0:b1].view(-1, 1, 1) - q_len + torch.arange(q_len, device="cuda").view(1, -1, 1)
        hidden = torch.arange(padded, device="cuda").view(1, 1, -1) > last                # [count, q_len, padded]
        ss.view(hkv, count, q_len, GROUP, padded).masked_fill_(hidden.unsqueeze(2), -math.inf)
        # slots behind a request's last token hold what other requests left there
        behind = torch.arange(padded, device="cuda").view(1, -1) >= s["seq_lens"][b0:b1].view(-1, 1)
        vs = vs.masked_fill(behind.view(1, count, padded, 1), 0.0)
        top = torch.maximum(sp.amax(dim=-1, keepdim=True), ss.amax(dim=-1, keepdim=True))
        sp, ss = sp.sub_(top).exp_(), ss.sub_(top).exp_()
        sums = sp.sum(dim=-1, keepdim=True) + ss.sum(dim=-1, keepdim=True)
        o = torch.matmul(sp.view(hkv, -1, plen), vp).view(hkv, count, q_len * GROUP, DIM) + torch.matmul(ss, vs)
        o = (o / sums).view(hkv, count, q_len, GROUP, DIM).permute(1, 2, 0, 3, 4)
        out[b0:b1] = o.reshape(count, q_len, hq, DIM).to(torch.bfloat16)
        lse[b0:b1] = (top + sums.log()).view(hkv, count, q_len, GROUP).permute(1, 2, 0, 3).reshape(count, q_len, hq)
        b0 = b1
    return out.view(s["q"].shape), lse.view(s["q"].shape[:-1])


def _write(s):
    page, slot = s["live_slots"] // PAGE, s["live_slots"] % PAGE
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x[s["live"]]
        if scale is None:
            cache[page, slot] = x
            continue
        x = x.float()
        step = x.abs().amax(dim=-1) / E4M3_MAX
        step = torch.where(step > 0, step, torch.ones_like(step))
        codes = (x / step.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        cache.view(torch.uint8)[page, slot] = codes.view(torch.uint8)
        scale.transpose(1, 2)[page, slot] = step


def _read(s):
    """Every row's page and slot, then one gather."""
    lens = torch.diff(s["out_starts"])
    row = torch.arange(sum(s["host_lens"]), device="cuda")
    b = torch.repeat_interleave(torch.arange(len(s["host_lens"]), device="cuda"), lens, output_size=row.numel())
    t = row - s["out_starts"][b] + s["first"][b]
    page, slot = s["page_table"][b, t // PAGE].long(), t % PAGE
    got = []
    for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        if scale is None:
            got.append(cache[page, slot])
        else:
            codes = cache.view(torch.uint8)[page, slot].view(cache.dtype)
            got.append((codes.float() * scale.transpose(1, 2)[page, slot].unsqueeze(-1)).to(torch.bfloat16))
    return tuple(got)


def run(s):
    if s["op"] == "prefill":
        if own:
            import load_balanced_paged_02_gb300 as hpc
            out, lse, _ = hpc.prefill(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["q_starts"],
                                      s["seq_lens"], s["k_scale"], s["v_scale"])
        else:
            out, lse = _prefill(s)
        return dict(out=out, lse=lse)
    if s["op"] == "prefix":
        if own:
            import load_balanced_paged_02_gb300 as hpc
            out, lse, _, _ = hpc.decode_shared_prefix(
                s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"], s["prefix_table"],
                s["prefix_lens"], s["group_starts"], s["k_scale"], s["v_scale"])
        else:
            out, lse = _prefix(s)
        return dict(out=out, lse=lse)
    if s["op"] == "write":
        if own:
            import load_balanced_paged_02_gb300 as hpc
            hpc.hpc_kv_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        else:
            _write(s)
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if own:
        import load_balanced_paged_02_gb300 as hpc
        rows = sum(s["host_lens"])
        k = torch.empty((rows,) + s["k_cache"].shape[2:], dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        hpc.hpc_kv_read(s["k_cache"], s["v_cache"], s["page_table"], s["out_starts"], k, v, s["k_scale"],
                        s["v_scale"], first=s["first"])
    else:
        k, v = _read(s)
    return dict(k=k, v=v)


# ---------------------------------------------------------------------------- work, and the same in 64 bits

def work(case):
    hkv = case["hkv"]
    row = 2 * DIM * 2 if case["kv"] == "bf16" else 2 * DIM + 8  # K and V of one token and head, with their scales
    wide = 2 * DIM * 2
    if case["op"] == "prefill":
        new, lens = lengths(case["new"]), lengths(case["lens"])
        pairs = sum(n * total - n * (n - 1) // 2 for n, total in zip(new, lens))
        return dict(bytes=hkv * (sum(lens) * row + sum(new) * GROUP * (2 * 2 * DIM + 4)),
                    flops=4 * DIM * GROUP * hkv * pairs)
    if case["op"] == "prefix":
        groups, prefixes, lens, q_len = lengths(case["groups"]), lengths(case["prefixes"]), lengths(case["lens"]), case["q_len"]
        pairs = q_len * (sum(n * p for n, p in zip(groups, prefixes)) + sum(lens))
        return dict(bytes=hkv * ((sum(prefixes) + sum(lens)) * row + len(lens) * q_len * GROUP * (2 * 2 * DIM + 4)),
                    flops=4 * DIM * GROUP * hkv * pairs)
    rows = case["tokens"] - case["padded"] if case["op"] == "write" else sum(lengths(case["lens"]))
    return dict(bytes=rows * hkv * (row + wide) + 4 * rows, flops=4 * rows * hkv * DIM)


def _exact_rows(q, k, v, visible):
    """Attention of q [n, hq, 128] over k, v [t, hkv, 128], all in 64 bits, row i seeing the first visible[i] tokens."""
    n, hq, _ = q.shape
    hkv = k.shape[1]
    out = torch.zeros((n, hq, DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i0 in range(0, n, 1024):
        i1 = min(n, i0 + 1024)
        most = int(max(visible[i0:i1]))
        seen = torch.tensor(visible[i0:i1], device="cuda")
        for h in range(hkv):
            x = q[i0:i1, GROUP * h:GROUP * (h + 1)].reshape(-1, DIM)
            z = (x @ k[:most, h].T) / math.sqrt(DIM)
            z = z.view(i1 - i0, GROUP, most)
            z = torch.where(torch.arange(most, device="cuda") < seen.view(-1, 1, 1), z, -math.inf)
            w = torch.logsumexp(z, dim=-1)
            some = torch.isfinite(w).unsqueeze(-1)
            weights = torch.where(some, torch.exp(z - torch.where(some, w.unsqueeze(-1), 0.0)), 0.0)
            out[i0:i1, GROUP * h:GROUP * (h + 1)] = (weights.view(-1, most) @ v[:most, h]).view(i1 - i0, GROUP, DIM)
            lse[i0:i1, GROUP * h:GROUP * (h + 1)] = w
    return out, lse


def _exact_tokens(cache, scale, pages, count):
    """The first `count` tokens of a list of pages in 64 bits, [count, hkv, 128]."""
    t = torch.arange(count, device="cuda")
    page, slot = pages.long()[t // PAGE], t % PAGE
    x = cache.double()[page, slot] if scale is None else cache.view(torch.uint8)[page, slot].view(cache.dtype).double()
    return x if scale is None else x * scale.double()[page, :, slot].unsqueeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefill":
        out, lse, at = [], [], 0
        for b, (n, total) in enumerate(zip(lengths(case["new"]), lengths(case["lens"]))):
            k = _exact_tokens(s["k_cache"], s["k_scale"], s["page_table"][b], total)
            v = _exact_tokens(s["v_cache"], s["v_scale"], s["page_table"][b], total)
            o, w = _exact_rows(s["q"][at:at + n].double(), k, v, [total - n + i + 1 for i in range(n)])
            out.append(o)
            lse.append(w)
            at += n
        return dict(out=torch.cat(out), lse=torch.cat(lse))
    if case["op"] == "prefix":
        out, lse, b = [], [], 0
        lens, q_len = lengths(case["lens"]), case["q_len"]
        for g, (count, plen) in enumerate(zip(lengths(case["groups"]), lengths(case["prefixes"]))):
            kp = _exact_tokens(s["k_cache"], s["k_scale"], s["prefix_table"][g], plen)
            vp = _exact_tokens(s["v_cache"], s["v_scale"], s["prefix_table"][g], plen)
            for _ in range(count):
                k = torch.cat([kp, _exact_tokens(s["k_cache"], s["k_scale"], s["page_table"][b], lens[b])])
                v = torch.cat([vp, _exact_tokens(s["v_cache"], s["v_scale"], s["page_table"][b], lens[b])])
                o, w = _exact_rows(s["q"][b].double().view(q_len, -1, DIM), k, v,
                                   [plen + max(0, lens[b] - q_len + i + 1) for i in range(q_len)])
                out.append(o)
                lse.append(w)
                b += 1
        return dict(out=torch.stack(out).view(s["q"].shape), lse=torch.stack(lse).view(s["q"].shape[:-1]))
    if case["op"] == "write":
        got = {}
        for x, name in ((s["k"], "k"), (s["v"], "v")):
            cache, scale = s[name + "_cache"], s[name + "_scale"]
            if scale is None:
                full = cache.double()
                full[s["live_slots"] // PAGE, s["live_slots"] % PAGE] = x[s["live"]].double()
                got[name + "_cache"], got[name + "_scale"] = full, None
            else:  # the codes are roundings of a rounded quotient: compared with the plain form's alone
                steps = scale.double().transpose(1, 2).contiguous()
                top = x[s["live"]].double().abs().amax(dim=-1)
                steps[s["live_slots"] // PAGE, s["live_slots"] % PAGE] = torch.where(top > 0, top / E4M3_MAX, 1.0)
                got[name + "_cache"], got[name + "_scale"] = None, steps.transpose(1, 2).contiguous()
        return got
    k, v = [], []
    for b, (n, first) in enumerate(zip(lengths(case["lens"]), lengths(case["first"]))):
        k.append(_exact_tokens(s["k_cache"], s["k_scale"], s["page_table"][b], first + n)[first:])
        v.append(_exact_tokens(s["v_cache"], s["v_scale"], s["page_table"][b], first + n)[first:])
    return dict(k=torch.cat(k), v=torch.cat(v))
