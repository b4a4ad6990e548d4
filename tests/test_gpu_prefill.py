"""Prompt attention over packed sequences (hpc_prefill_*) against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb
import _tiles as tl

pytestmark = pytest.mark.gpu


def case(new, lens, hkv, kv, seed, **kw):
    """A packed batch; lens are the keys of each sequence (its new tokens among them)."""
    c = tl.make_cache([[max(0, n) for n in lens]], hkv, kv, seed, **kw)
    T = sum(new)
    c.update(new=list(new), lens=list(lens), hkv=hkv, kv=kv, q=tl.make_q((T, 8 * hkv, tl.DIM), seed), table=c["tables"][0],
             q_starts=tl.i32(tl.starts(new)), seq_lens=tl.i32(lens))
    return c


def run(c, **kw):
    out, lse, plan = hb.prefill(c["q"], c["k_cache"], c["v_cache"], c["table"], c["q_starts"], c["seq_lens"], c["k_scale"],
                                c["v_scale"], **kw)
    torch.cuda.synchronize()
    return out, lse, plan


def reference(c, b):
    n, L = c["new"][b], max(0, c["lens"][b])
    s = sum(c["new"][:b])
    return tl.attend(c["q"][s:s + n], c["k"][0][b], c["v"][0][b], [max(0, min(L, L - n + i + 1)) for i in range(n)])


def check(c, out, lse, what=""):
    s = 0
    for b, n in enumerate(c["new"]):
        tl.check_rows(out[s:s + n], lse[s:s + n], reference(c, b), c["kv"] != "bf16", f"{what} sequence {b} ({n} of {c['lens'][b]})")
        s += n


# new tokens and keys: one token, a page less one, exactly, more one; tiles of 16, 32, 64 tokens and their
# neighbours; pieces behind a history; sequences without new tokens or keys; more new tokens than keys
BATCHES = {
    "one token": ([1], [1]),
    "small": ([16, 17, 1, 0, 31], [16, 17, 64, 65, 31]),
    "pages": ([63, 64, 65, 127, 128, 129], [63, 64, 65, 127, 128, 129]),
    "tiles": ([15, 32, 33, 48, 49, 64, 80, 97], [15, 32, 133, 48, 300, 64, 128, 97]),
    "pieces": ([5, 40, 1, 100], [700, 640, 513, 1001]),
    "decode": ([1] * 9, [1, 63, 64, 65, 128, 129, 1000, 2, 500]),
    "gaps": ([0, 0, 70, 0, 3, 0], [0, 90, 70, 0, 200, 64]),
    "more new than keys": ([40, 10, 3, 70], [33, 0, 2, 5]),
    "long": ([700], [2000]),
}


@pytest.mark.parametrize("tile", [32, 64])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(BATCHES))
def test_batches(name, kv, tile):
    new, lens = BATCHES[name]
    c = case(new, lens, 2, kv, seed=len(name) + 7)
    for ctas in (None, 7, 300):
        out, lse, plan = run(c, num_ctas=ctas, tile_tokens=tile)
        check(c, out, lse, f"{name}, {ctas} CTAs")
        assert hb.hpc_tile_read_error(plan) == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_heads_and_one_worker(kv, hkv):
    c = case([37, 128, 90], [37, 300, 90], hkv, kv, seed=hkv)
    for ctas, tile, m in ((1, 0, 1), (2, 64, 1), (152, 0, 3), (5, 32, 4)):
        out, lse, _ = run(c, num_ctas=ctas, tile_tokens=tile, min_blocks_per_cta=m)
        check(c, out, lse, f"{ctas} CTAs, tile {tile}, floor {m}")


@pytest.mark.parametrize("tile", [32, 64])
def test_random_maps_bit_for_bit(tile):
    rng = np.random.default_rng(5)
    for rep in range(60):
        S = int(rng.integers(1, 40))
        new = [int(x) if rng.random() > 0.2 else 0 for x in np.exp(rng.uniform(0, np.log(400), S))]
        lens = [int(n + rng.integers(0, 500)) if rng.random() > 0.1 else int(rng.integers(0, 60)) for n in new]
        hkv, ctas, m = int(rng.integers(1, 9)), int(rng.integers(2, 200)), int(rng.integers(0, 4))
        T = sum(new) + 3
        plan = hb.hpc_prefill_plan(tl.i32(tl.starts(new)), tl.i32(lens), T, hkv, 40, num_ctas=ctas, min_blocks_per_cta=m,
                                   tile_tokens=tile)
        workers = ctas // (tile // 32)
        want = tl.tile_map(0, tl.starts(new), lens, T, hkv, workers, m, tile)
        assert np.array_equal(plan.words().cpu().numpy()[:len(want)], want), f"map {rep}"


def test_plan_of_many_sequences():
    rng = np.random.default_rng(6)
    new = rng.integers(0, 4, 5000).tolist()
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 300, 5000))]
    plan = hb.hpc_prefill_plan(tl.i32(tl.starts(new)), tl.i32(lens), sum(new), 2, 8, num_ctas=152, tile_tokens=32)
    want = tl.tile_map(0, tl.starts(new), lens, sum(new), 2, 152, 1, 32)
    assert np.array_equal(plan.words().cpu().numpy()[:len(want)], want)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_rows_of_no_sequence_keep_their_bits(kv):
    """Rows before the first start, behind the last one, and of passed-over sequences are left as they were."""
    c = case([9, 50, 20], [9, 80, 20], 1, kv, seed=3)
    T = 100
    q = torch.full((T, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[4:83] = c["q"]
    out = torch.full((T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 8), 5.0, device="cuda")
    for tile in (32, 64):
        out.fill_(7.0), lse.fill_(5.0)
        hb.prefill(q, c["k_cache"], c["v_cache"], c["table"], tl.i32([4, 13, 63, 83]), c["seq_lens"], c["k_scale"], c["v_scale"],
                   out=out, out_lse=lse, num_ctas=9, tile_tokens=tile)
        check(c, out[4:83], lse[4:83])
        assert (out[:4] == 7).all() and (out[83:] == 7).all() and (lse[:4] == 5).all() and (lse[83:] == 5).all()


def test_no_tokens():
    c = case([4], [4], 1, "bf16", seed=1)
    out, lse, _ = hb.prefill(c["q"][:0], c["k_cache"], c["v_cache"], c["table"], tl.i32([0, 0]), c["seq_lens"])
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("tile", [32, 64])
def test_scores_that_grow(kv, tile):
    """Each block's scores far above the last's, so the reference maximum moves in every block; rows
    whose weight sits on one key; very negative scores."""
    c = case([96, 40], [900, 700], 1, kv, seed=11)
    for b in range(2):
        L = c["lens"][b]
        ramp = torch.linspace(0.0, 6.0, L, device="cuda").to(torch.bfloat16)
        c["q"].copy_(c["q"].abs())
        pages = c["table"][b][torch.arange(L, device="cuda") // 64].long()
        slot = torch.arange(L, device="cuda") % 64
        k = (torch.ones((L, 1, 128), device="cuda") * ramp.view(L, 1, 1)).to(torch.bfloat16)
        if kv == "bf16":
            c["k_cache"][pages, slot] = k
            c["k"][0][b] = k.double()
        else:
            hb.hpc_kv_write(k, c["v"][0][b].to(torch.bfloat16).contiguous(), (pages * 64 + slot).int(), c["k_cache"], c["v_cache"],
                            c["k_scale"], c["v_scale"])
            for n in "kv":
                codes = c[n + "_cache"].view(torch.uint8)[pages, slot].view(torch.float8_e4m3fn).double()
                c[n][0][b] = codes * c[n + "_scale"].double()[pages, :, slot].unsqueeze(-1)
    for ctas in (None, 3):
        out, lse, _ = run(c, num_ctas=ctas, tile_tokens=tile)
        check(c, out, lse, "growing")
    c["q"].neg_()
    out, lse, _ = run(c, tile_tokens=tile)
    check(c, out, lse, "falling")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_sizes_that_vary(kv):
    """Tokens of K and V whose sizes differ by orders of magnitude, small and large queries."""
    for qs, cs in ((1.0, 1.0), (8.0, 1.0), (0.01, 20.0), (1.0, 1e-3)):
        c = case([50, 130], [400, 130], 2, kv, seed=21, spread=True, scale=cs)
        c["q"].mul_(qs)
        out, lse, _ = run(c)
        check(c, out, lse, f"query {qs}, cache {cs}")


@pytest.mark.parametrize("tile", [32, 64])
def test_keys_that_are_not_seen(tile):
    """Infinities and NaN in keys behind a row's limit reach neither its maximum nor its sum."""
    c = case([100], [100], 1, "bf16", seed=31)
    t = 77
    page, slot = int(c["table"][0][t // 64]), t % 64
    for bad in (float("nan"), float("inf"), torch.finfo(torch.bfloat16).min):
        c["k_cache"][page, slot] = bad
        out, lse, _ = run(c, tile_tokens=tile)
        ref = reference(c, 0)
        tl.check_rows(out[:t], lse[:t], tuple(x[:t] for x in ref), False, f"rows before a key of {bad}")


def test_pages_out_of_range():
    """A bad page id hides its 64 tokens and is reported; so do keys beyond the table's row."""
    c = case([30], [300], 1, "bf16", seed=41)
    for tile in (32, 64):
        for bad in (-5, c["pages"], 2147483647):
            table = c["table"].clone()
            table[0, 1] = bad
            out, lse, plan = hb.prefill(c["q"], c["k_cache"], c["v_cache"], table, c["q_starts"], c["seq_lens"], tile_tokens=tile)
            keep = torch.cat([torch.arange(0, 64), torch.arange(128, 300)]).cuda()
            k, v = c["k"][0][0][keep], c["v"][0][0][keep]
            ref = tl.attend(c["q"], k, v, [300 - 30 + i + 1 - 64 for i in range(30)])
            tl.check_rows(out, lse, ref, False, f"page {bad}")
            assert hb.hpc_tile_read_error(plan) == 4
        short = c["table"][:, :2].contiguous()
        out, lse, plan = hb.prefill(c["q"], c["k_cache"], c["v_cache"], short, c["q_starts"], c["seq_lens"], tile_tokens=tile)
        assert hb.hpc_tile_read_error(plan) == 4
        ref = tl.attend(c["q"], c["k"][0][0][:128], c["v"][0][0][:128], [128 - 30 + i + 1 for i in range(30)])
        tl.check_rows(out, lse, ref, False, "keys beyond the table")


def test_bad_starts_and_lengths():
    c = case([10, 20], [10, 64], 1, "bf16", seed=51)
    plan = hb.hpc_prefill_plan(tl.i32([0, 10, 30]), tl.i32([10, -4]), 30, 1, c["table"].shape[1])
    assert hb.hpc_tile_read_error(plan) == 1
    for st in ([0, 10, 31], [0, 40, 30], [-1, 10, 30], [5, 3, 30]):
        out = torch.full_like(c["q"], 3.0)
        out2, lse, plan = hb.prefill(c["q"], c["k_cache"], c["v_cache"], c["table"], tl.i32(st), c["seq_lens"], out=out)
        assert hb.hpc_tile_read_error(plan) & 16
        want = tl.tile_map(0, st, c["lens"], 30, 1, plan.struct.num_workers, 1, plan.tile_tokens)
        assert np.array_equal(plan.words().cpu().numpy()[:16], want[:16])
        for b in range(2):  # a sequence whose starts are right is computed all the same
            a, e = st[b], st[b + 1]
            if 0 <= a <= e <= 30 and e - a == c["new"][b]:
                ref = tl.attend(c["q"][a:e], c["k"][0][b], c["v"][0][b],
                                [max(0, c["lens"][b] - (e - a) + i + 1) for i in range(e - a)])
                tl.check_rows(out2[a:e], lse[a:e], ref, False, f"starts {st}, sequence {b}")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_three_calls_and_one_agree(kv):
    c = case([300, 40], [420, 333], 2, kv, seed=61)
    out, lse, plan = run(c, num_ctas=20)
    p = hb.hpc_prefill_plan(c["q_starts"], c["seq_lens"], c["q"].shape[0], 2, c["table"].shape[1], num_ctas=20)
    so, sl = hb.prefill_split_buffers(p)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    for _ in range(2):  # one map serves every layer
        hb.hpc_prefill_attn(c["q"], c["k_cache"], c["v_cache"], c["table"], p, so, sl, o2, l2, c["k_scale"], c["v_scale"])
        hb.hpc_prefill_combine(p, so, sl, o2, l2)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    hb.hpc_prefill_attn(c["q"], c["k_cache"], c["v_cache"], c["table"], p, so, sl, o2, None, c["k_scale"], c["v_scale"])
    hb.hpc_prefill_combine(p, so, sl, o2)
    assert torch.equal(o2, out)
    # the same call again gives the same bits
    again, lagain, _ = run(c, num_ctas=20)
    assert torch.equal(again, out) and torch.equal(lagain, lse)


def test_graph_streams_and_two_calls_at_once():
    """Captured and replayed with new inputs; on another stream; two calls in flight with their own workspaces."""
    a, b = case([200, 3], [300, 90], 2, "bf16", seed=71), case([90], [500], 1, "e4m3", seed=72)
    run(a), run(b)
    ws = torch.empty(hb.prefill_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(a["q"]), torch.empty(a["q"].shape[:2], device="cuda")
    q = a["q"].clone()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        hb.prefill(q, a["k_cache"], a["v_cache"], a["table"], a["q_starts"], a["seq_lens"], out=out, out_lse=lse, workspace=ws)
    for seed in (1, 2):
        a["q"] = tl.make_q(tuple(q.shape), seed)
        q.copy_(a["q"])
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(a, out, lse, "replayed")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for c, st in ((a, s1), (b, s2)):
            got.append((c, hb.prefill(c["q"], c["k_cache"], c["v_cache"], c["table"], c["q_starts"], c["seq_lens"], c["k_scale"],
                                      c["v_scale"], stream=st)))
    torch.cuda.synchronize()
    for c, (o, l, _) in got[-4:]:
        check(c, o, l, "two streams")


def test_offsets_past_31_bits():
    """Pages at the end of a cache of more than 2^31 elements."""
    hkv, pages = 8, 33000
    cache = torch.zeros((pages, 64, hkv, 128), dtype=torch.bfloat16, device="cuda")
    assert cache.numel() > 2 ** 31
    vcache = torch.zeros_like(cache)
    gen = torch.Generator(device="cuda").manual_seed(1)
    used = torch.tensor([pages - 1, pages - 2, 5], device="cuda")
    cache[used] = torch.randn((3, 64, hkv, 128), generator=gen, device="cuda").to(torch.bfloat16)
    vcache[used] = torch.randn((3, 64, hkv, 128), generator=gen, device="cuda").to(torch.bfloat16)
    q = tl.make_q((20, 64, 128), 3)
    for tile in (32, 64):
        out, lse, _ = hb.prefill(q, cache, vcache, used.int().view(1, 3), tl.i32([0, 20]), tl.i32([150]), tile_tokens=tile)
        k, v = cache[used].double().flatten(0, 1)[:150], vcache[used].double().flatten(0, 1)[:150]
        tl.check_rows(out, lse, tl.attend(q, k, v, [150 - 20 + i + 1 for i in range(20)]), False, "far pages")
    del cache, vcache


def test_binding_refusals():
    c = case([9], [9], 1, "bf16", seed=81)
    good = dict(q=c["q"], k=c["k_cache"], v=c["v_cache"], t=c["table"], s=c["q_starts"], l=c["seq_lens"])

    def call(**kw):
        a = dict(good, **kw)
        return hb.prefill(a["q"], a["k"], a["v"], a["t"], a["s"], a["l"])
    call()
    for kw in (dict(q=c["q"].float()), dict(q=c["q"].transpose(0, 1)), dict(s=c["q_starts"].long()), dict(s=c["q_starts"][:1]),
               dict(t=c["table"].cpu()), dict(t=torch.cat([c["table"]] * 2)), dict(v=c["v_cache"][:1]), dict(l=c["seq_lens"].float()),
               dict(k=c["k_cache"].float()), dict(k=c["k_cache"].to(torch.float8_e4m3fn), v=c["v_cache"].to(torch.float8_e4m3fn))):
        with pytest.raises(hb.HpcError):
            call(**kw)
    with pytest.raises(hb.HpcError):
        hb.prefill(*[good[n] for n in "qkvtsl"], out=torch.empty((9, 8, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(hb.HpcError):
        hb.prefill(*[good[n] for n in "qkvtsl"], num_pages=c["pages"] + 1)
    with pytest.raises(hb.HpcError):
        hb.prefill(*[good[n] for n in "qkvtsl"], workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_another_map_in_the_plans_buffer():
    """A map planned for other sizes into the same buffer: the old plan's calls compute nothing and say so."""
    for tile in (32, 64):
        c = case([40, 3], [200, 3], 1, "bf16", 91)
        plan = hb.hpc_prefill_plan(c["q_starts"], c["seq_lens"], 43, 1, c["table"].shape[1], num_ctas=8, tile_tokens=tile)
        old = hb.TilePlanStruct.from_buffer_copy(plan.struct)
        hb.hpc_prefill_plan(tl.i32([0, 43]), tl.i32([200]), 43, 1, c["table"].shape[1], num_ctas=8, tile_tokens=tile, plan=plan)
        plan.struct = old
        so, sl = hb.prefill_split_buffers(plan)
        out = torch.full_like(c["q"], 7.0)
        lse = torch.full((43, 8), 7.0, device="cuda")
        hb.hpc_prefill_attn(c["q"], c["k_cache"], c["v_cache"], c["table"], plan, so, sl, out, lse)
        hb.hpc_prefill_combine(plan, so, sl, out, lse)
        assert hb.hpc_tile_read_error(plan) & 16  # HPC_DEVERR_BAD_DESCRIPTOR
        assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


@pytest.mark.parametrize("tile", [32, 64])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("growth", ["steady", "late page", "steps", "falling", "beyond exp2"])
def test_references_that_move(growth, kv, tile):
    """The reference maximum moves in the first page of a block, in its second, in every block, never,
    and by more than float32's exponents hold."""
    n, hkv = 520, 2
    c = case([90, 1], [n, n - 64], hkv, kv, 97)
    t = torch.arange(n, dtype=torch.float64)
    size = {"steady": t / n * 40.0, "late page": torch.where(t % 128 >= 100, 30.0 + t / 16.0, 0.0), "steps": (t // 64) * 12.0,
            "falling": 60.0 - t / n * 60.0, "beyond exp2": (t // 128) * 150.0}[growth]
    sign = torch.where(torch.arange(128) % 3 == 0, -1.0, 1.0).double()
    for b in range(2):
        m = c["lens"][b]
        gen = torch.Generator().manual_seed(b)
        k = size[:m, None, None] * sign / np.sqrt(128.0) + 0.1 * torch.randn((m, hkv, 128), generator=gen, dtype=torch.float64)
        v = torch.randn((m, hkv, 128), generator=gen, dtype=torch.float64)
        pages = c["table"][b].cpu().long()
        at = torch.arange(m)
        slots = (pages[at // 64] * 64 + at % 64).int().cuda()
        hb.hpc_kv_write(k.bfloat16().cuda(), v.bfloat16().cuda(), slots, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"])
        torch.cuda.synchronize()
        for name in "kv":
            page, off = slots.long() // 64, slots.long() % 64
            x = c[name + "_cache"][page, off].float().double()
            if kv == "e4m3":
                x = x * c[name + "_scale"].double()[page, :, off].unsqueeze(-1)
            c[name][0][b] = x
    q = (sign.float() + 0.05 * torch.randn((91, 8 * hkv, 128), generator=torch.Generator().manual_seed(9)))
    c["q"] = q.bfloat16().cuda()
    for ctas in (None, 8):
        out, lse, _ = run(c, tile_tokens=tile, num_ctas=ctas)
        check(c, out, lse, growth)


@pytest.mark.parametrize("tile", [32, 64])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_queries_of_every_size(kv, tile):
    """Query rows from 1e-30 to 1e4, rows whose elements span 2^40, rows of zeros; then rows with an
    infinity or a NaN, which leave the others bit for bit as they were."""
    c = case([70, 33], [200, 333], 1, kv, seed=131)
    gen = torch.Generator().manual_seed(7)
    rows = torch.tensor([1e-30, 1e-10, 1e-4, 1.0, 30.0, 1e4]).repeat(200)[:103 * 8].view(103, 8, 1)
    spans = torch.exp2(-40.0 * torch.rand((103, 8, 128), generator=gen)) * (torch.arange(103) % 5 == 0).view(103, 1, 1)
    q = torch.randn((103, 8, 128), generator=gen) * rows
    q = torch.where(spans > 0, torch.sign(q) * spans * 4.0, q)
    q[11] = 0.0
    c["q"] = q.bfloat16().cuda()
    for ctas in (None, 5):
        out, lse, _ = run(c, tile_tokens=tile, num_ctas=ctas)
        check(c, out, lse, "sizes")
        kept = c["q"]
        c["q"] = kept.clone()
        bad = [(3, 1, 5, float("inf")), (40, 7, 0, float("nan")), (69, 0, 127, -float("inf")), (100, 3, 64, float("nan"))]
        for t, h, d, x in bad:
            c["q"][t, h, d] = x
        out2, lse2, _ = run(c, tile_tokens=tile, num_ctas=ctas)
        same = torch.ones((103, 8), dtype=torch.bool, device="cuda")
        for t, h, d, x in bad:
            same[t, h] = False
            assert not torch.isfinite(out2[t, h].float()).all()
        assert torch.equal(out[same], out2[same]) and torch.equal(lse[same], lse2[same])
        c["q"] = kept
