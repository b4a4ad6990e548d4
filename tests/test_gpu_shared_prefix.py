"""Decode for batches whose groups share prefixes (hpc_prefix_*, hpc_decode_shared_prefix) against a
plain 64-bit implementation, and a run of the operators together."""
import numpy as np
import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb
import _tiles as tl

pytestmark = pytest.mark.gpu


def case(groups, prefixes, lens, hkv, kv, q_len, seed, first=0, batch=None):
    """groups: requests of each group, from request `first` on; lens: tokens behind the prefix."""
    B = len(lens) if batch is None else batch
    c = tl.make_cache([lens, prefixes], hkv, kv, seed)
    shape = (B, 8 * hkv, tl.DIM) if q_len == 1 else (B, q_len, 8 * hkv, tl.DIM)
    st = [first + x for x in tl.starts(groups)]
    c.update(starts=st, prefixes=list(prefixes), lens=list(lens), hkv=hkv, kv=kv, q_len=q_len, q=tl.make_q(shape, seed),
             table=c["tables"][0], ptable=c["tables"][1], seq_lens=tl.i32(lens), plens=tl.i32(prefixes), gstarts=tl.i32(st))
    return c


def run(c, **kw):
    out, lse, pplan, plan = hb.decode_shared_prefix(c["q"], c["k_cache"], c["v_cache"], c["table"], c["seq_lens"], c["ptable"],
                                                    c["plens"], c["gstarts"], c["k_scale"], c["v_scale"], **kw)
    torch.cuda.synchronize()
    return out, lse, pplan, plan


def check(c, out, lse, what=""):
    Q, hq = c["q_len"], 8 * c["hkv"]
    for b, n in enumerate(c["lens"]):
        k, v, p = c["k"][0][b], c["v"][0][b], 0
        for g in range(len(c["prefixes"])):
            if c["starts"][g] <= b < c["starts"][g + 1]:
                p = c["prefixes"][g]
                k, v = torch.cat([c["k"][1][g], k]), torch.cat([c["v"][1][g], v])
        ref = tl.attend(c["q"][b].reshape(Q, hq, 128), k, v, [p + max(0, n - Q + i + 1) for i in range(Q)])
        tl.check_rows(out[b].reshape(Q, hq, 128), lse[b].reshape(Q, hq), ref, c["kv"] != "bf16", f"{what} request {b}")


BATCHES = {
    "one request": ([1], [1], [1], 0),
    "one group": ([8], [1000], [37, 37, 37, 128, 129, 300, 1, 0], 0),
    "tiles": ([17, 33, 65], [64, 129, 200], [int(x) for x in np.random.default_rng(3).integers(0, 90, 115)], 0),
    "empty groups": ([0, 3, 0, 2, 0], [70, 128, 0, 500, 64], [5, 0, 64, 65, 9], 0),
    "no prefix": ([4], [0], [5, 0, 64, 100], 0),
    "requests outside": ([2, 3], [300, 65], [9, 10, 11, 12, 0, 14, 15, 130], 2),
}


@pytest.mark.parametrize("tile", [32, 64])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(BATCHES))
def test_batches(name, kv, tile):
    groups, prefixes, lens, first = BATCHES[name]
    for q_len in (1, 3):
        c = case(groups, prefixes, lens, 2, kv, q_len, seed=len(name), first=first)
        for ctas in (None, 6, 300):
            out, lse, pplan, plan = run(c, prefix_num_ctas=ctas, tile_tokens=tile)
            check(c, out, lse, f"{name}, {ctas} CTAs, {q_len} new")
            assert hb.hpc_tile_read_error(pplan) == 0 and hb.hpc_decode_read_error(plan) == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [1, 2, 4, 8])
def test_long_prefix_many_pieces(kv, q_len):
    c = case([20], [5000], [int(x) for x in np.random.default_rng(1).integers(0, 200, 20)], 1, kv, q_len, seed=q_len)
    for tile in (32, 64):
        out, lse, _, _ = run(c, tile_tokens=tile)
        check(c, out, lse, f"{q_len} new, tile {tile}")


def test_equals_decode_over_the_whole_sequence():
    """With a prefix of whole pages, a request's own page table behind it names the same tokens: plain
    decode gives the same rows, up to the rounding of the outputs and of P."""
    c = case([6, 3], [256, 640], [30, 64, 1, 100, 65, 128, 9, 10, 500], 2, "bf16", 1, seed=9)
    out, lse, _, _ = run(c)
    rows, full = [], []
    for b, n in enumerate(c["lens"]):
        g = 0 if b < 6 else 1
        pages = torch.cat([c["ptable"][g][:c["prefixes"][g] // 64], c["table"][b][:-(-n // 64)]])
        rows.append(pages)
        full.append(c["prefixes"][g] + n)
    table = torch.full((9, max(len(r) for r in rows)), -1, dtype=torch.int32, device="cuda")
    for b, r in enumerate(rows):
        table[b, :len(r)] = r
    o2, l2, _ = hb.decode(c["q"], c["k_cache"], c["v_cache"], table, tl.i32(full))
    check(c, o2, l2, "plain decode")
    check(c, out, lse, "shared prefix")


@pytest.mark.parametrize("tile", [32, 64])
def test_random_maps_bit_for_bit(tile):
    rng = np.random.default_rng(8)
    for rep in range(40):
        G = int(rng.integers(1, 12))
        groups = [int(x) if rng.random() > 0.2 else 0 for x in np.exp(rng.uniform(0, np.log(80), G))]
        plens = [int(x) if rng.random() > 0.15 else 0 for x in np.exp(rng.uniform(0, np.log(3000), G))]
        q_len, hkv, ctas, m = int(rng.integers(1, 9)), int(rng.integers(1, 9)), int(rng.integers(2, 200)), int(rng.integers(0, 4))
        B = max(1, sum(groups))
        plan = hb.hpc_prefix_plan(tl.i32(tl.starts(groups)), tl.i32(plens), B, hkv, 60, q_len=q_len, num_ctas=ctas,
                                  min_blocks_per_cta=m, tile_tokens=tile)
        want = tl.tile_map(1, tl.starts(groups), plens, B * q_len, hkv, ctas // (tile // 32), m, tile, q_len=q_len)
        assert np.array_equal(plan.words().cpu().numpy()[:len(want)], want), f"map {rep}"


def test_three_calls_graph_and_streams():
    c = case([5, 9], [500, 130], [20] * 14, 2, "bf16", 1, seed=4)
    out, lse, _, _ = run(c)
    pp = hb.hpc_prefix_plan(c["gstarts"], c["plens"], 14, 2, c["ptable"].shape[1])
    plan = hb.hpc_decode_plan(c["seq_lens"], 2)
    po, pl = hb.prefix_split_buffers(pp)
    so, sl = hb.split_buffers(plan)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    hb.hpc_prefix_attn(c["q"], c["k_cache"], c["v_cache"], c["ptable"], pp, po, pl)
    hb.hpc_decode_attn(c["q"], c["k_cache"], c["v_cache"], c["table"], c["seq_lens"], plan, so, sl)
    hb.hpc_prefix_combine(pp, po, pl, plan, so, sl, o2, l2)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    need = hb.decode_shared_prefix_workspace_bytes(2, 14, 2)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        o3, l3, _, _ = run_in(c, ws)
    o3.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o3, out) and torch.equal(l3, lse)
    d = case([3], [1000], [7, 8, 9], 1, "e4m3", 2, seed=5)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(x, hb.decode_shared_prefix(x["q"], x["k_cache"], x["v_cache"], x["table"], x["seq_lens"], x["ptable"], x["plens"],
                                       x["gstarts"], x["k_scale"], x["v_scale"], stream=st)) for _ in range(8) for x, st in ((c, s1), (d, s2))]
    torch.cuda.synchronize()
    for x, r in got[-4:]:
        check(x, r[0], r[1], "two streams")


def run_in(c, ws):
    return hb.decode_shared_prefix(c["q"], c["k_cache"], c["v_cache"], c["table"], c["seq_lens"], c["ptable"], c["plens"],
                                   c["gstarts"], c["k_scale"], c["v_scale"], workspace=ws)


def test_bad_inputs_are_reported():
    c = case([4], [300], [10, 11, 12, 13], 1, "bf16", 1, seed=6)
    table = c["ptable"].clone()
    table[0, 2] = c["pages"] + 9
    out, lse, pplan, _ = hb.decode_shared_prefix(c["q"], c["k_cache"], c["v_cache"], c["table"], c["seq_lens"], table, c["plens"],
                                                 c["gstarts"])
    assert hb.hpc_tile_read_error(pplan) == 4
    keep = torch.cat([torch.arange(0, 128), torch.arange(192, 300)]).cuda()
    for b in range(4):
        k, v = torch.cat([c["k"][1][0][keep], c["k"][0][b]]), torch.cat([c["v"][1][0][keep], c["v"][0][b]])
        tl.check_rows(out[b:b + 1], lse[b:b + 1], tl.attend(c["q"][b:b + 1], k, v, [len(k)]), False, "a page left out")
    for st, pl, want in (([0, 5], [300], 16), ([3, 1], [300], 16), ([0, 4], [-1], 1), ([0, 4], [100000], 4)):
        _, _, pplan, _ = hb.decode_shared_prefix(c["q"], c["k_cache"], c["v_cache"], c["table"], c["seq_lens"], c["ptable"], tl.i32(pl),
                                                 tl.i32(st))
        assert hb.hpc_tile_read_error(pplan) & want, (st, pl)
    for kw in (dict(q=c["q"].half()), dict(plens=c["plens"].long()), dict(gstarts=c["gstarts"][:1]), dict(ptable=c["ptable"][:, 0]),
               dict(seq_lens=c["seq_lens"][:2])):
        with pytest.raises(hb.HpcError):
            run(dict(c, **kw))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_the_operators_together(kv):
    """A system prompt written to the cache and computed, its pages then shared by a batch whose own tokens
    are written behind it; the batch's rows equal those of whole prompts; the cache read back."""
    hkv, P, own = 2, 192, [40, 1, 90]
    gen = torch.Generator(device="cuda").manual_seed(3)
    pages = 3 + 6
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    kc, vc = (torch.zeros((pages, 64, hkv, 128), dtype=dtype, device="cuda") for _ in range(2))
    ks = vs = None
    if kv != "bf16":
        ks, vs = (torch.zeros((pages, hkv, 64), device="cuda") for _ in range(2))
    total = P + sum(own)
    qkv = torch.randn((total, 12 * hkv - 4, 128), generator=gen, device="cuda").to(torch.bfloat16)[:, :10 * hkv]
    k, v, q = qkv[:, 8 * hkv:9 * hkv], qkv[:, 9 * hkv:], qkv[:, :8 * hkv].contiguous()
    prefix = torch.tensor([[7, 0, 3]], dtype=torch.int32, device="cuda")
    table = torch.tensor([[1, -1], [4, -1], [8, 2]], dtype=torch.int32, device="cuda")
    slots = [int(prefix[0, t // 64]) * 64 + t % 64 for t in range(P)]
    for b, n in enumerate(own):
        slots += [int(table[b, t // 64]) * 64 + t % 64 for t in range(n)]
    hb.hpc_kv_write(k, v, tl.i32(slots), kc, vc, ks, vs)
    # the system prompt alone
    po, pl, _ = hb.prefill(q[:P], kc, vc, prefix, tl.i32([0, P]), tl.i32([P]), ks, vs)
    # each request whole: its own tokens behind the prefix, as a piece
    whole = torch.cat([prefix.expand(3, 3), table], dim=1).contiguous()
    st = tl.starts(own)
    wo, wl, _ = hb.prefill(q[P:], kc, vc, whole, tl.i32(st), tl.i32([P + n for n in own]), ks, vs)
    # the same last tokens as a decode step behind the shared prefix
    last = torch.tensor([P + e - 1 for e in st[1:]], device="cuda")
    do, dl, _, _ = hb.decode_shared_prefix(q[last], kc, vc, table, tl.i32(own), prefix, tl.i32([P]), tl.i32([0, 3]), ks, vs)
    torch.cuda.synchronize()
    # values from the cache, read back
    rows = total
    kr, vr = (torch.empty((rows, hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    both = torch.full((4, 3), -1, dtype=torch.int32, device="cuda")
    both[0], both[1:, :2] = prefix[0], table
    hb.hpc_kv_read(kc, vc, both, tl.i32(tl.starts([P] + own)), kr, vr, ks, vs)
    if kv == "bf16":
        assert torch.equal(kr, k) and torch.equal(vr, v)
    at = torch.tensor(slots, device="cuda")

    def exact(cache, sc):
        x = cache.view(torch.uint8)[at // 64, at % 64].view(cache.dtype).double() if sc is not None else cache[at // 64, at % 64].double()
        return x if sc is None else x * sc.double()[at // 64, :, at % 64].unsqueeze(-1)
    ke, ve = exact(kc, ks), exact(vc, vs)
    assert ((kr.double() - ke).abs() <= 2.0 ** -8 * ke.abs()).all() and ((vr.double() - ve).abs() <= 2.0 ** -8 * ve.abs()).all()
    fp8 = kv != "bf16"
    tl.check_rows(po, pl, tl.attend(q[:P], ke[:P], ve[:P], list(range(1, P + 1))), fp8, "system prompt")
    for b, n in enumerate(own):
        rowsb = torch.cat([torch.arange(P), torch.arange(P + st[b], P + st[b + 1])]).cuda()
        ref = tl.attend(q[P + st[b]:P + st[b + 1]], ke[rowsb], ve[rowsb], [P + i + 1 for i in range(n)])
        tl.check_rows(wo[st[b]:st[b + 1]], wl[st[b]:st[b + 1]], ref, fp8, f"request {b}")
        tl.check_rows(do[b:b + 1], dl[b:b + 1], tuple(x[-1:] for x in ref), fp8, f"decode {b}")


def test_another_map_in_the_plans_buffer():
    """A prefix map planned for other groups into the same buffer: the old plan's call computes nothing and
    says so, and the merge takes the requests' own tokens alone."""
    for tile in (32, 64):
        c = case([5, 3], [200, 70], [9, 64, 1, 130, 20, 7, 65, 3], 1, "bf16", 1, 171)
        pplan = hb.hpc_prefix_plan(c["gstarts"], c["plens"], 8, 1, c["ptable"].shape[1], num_ctas=8, tile_tokens=tile)
        old = hb.TilePlanStruct.from_buffer_copy(pplan.struct)
        hb.hpc_prefix_plan(tl.i32([0, 8]), tl.i32([70]), 8, 1, c["ptable"].shape[1], num_ctas=8, tile_tokens=tile, plan=pplan)
        pplan.struct = old
        po, pl = hb.prefix_split_buffers(pplan)
        po.fill_(float("nan"))
        hb.hpc_prefix_attn(c["q"], c["k_cache"], c["v_cache"], c["ptable"], pplan, po, pl)
        assert hb.hpc_tile_read_error(pplan) & 16  # HPC_DEVERR_BAD_DESCRIPTOR
        plan = hb.hpc_decode_plan(c["seq_lens"], 1)
        so, sl = hb.split_buffers(plan)
        hb.hpc_decode_attn(c["q"], c["k_cache"], c["v_cache"], c["table"], c["seq_lens"], plan, so, sl)
        out, lse = torch.empty_like(c["q"]), torch.empty((8, 8), device="cuda")
        hb.hpc_prefix_combine(pplan, po, pl, plan, so, sl, out, lse)
        for b in range(8):
            n = c["lens"][b]
            tl.check_rows(out[b:b + 1], lse[b:b + 1], tl.attend(c["q"][b:b + 1], c["k"][0][b], c["v"][0][b], [n]), False, f"request {b}")


def test_the_largest_batch():
    """As many requests as the planners take (their length sums no longer fit the default shared memory)."""
    B = 16384
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 4, B)]
    c = case([B - 5, 3], [70, 129], lens, 1, "bf16", 1, 181, first=1)
    out, lse, pplan, plan = run(c)
    assert hb.hpc_tile_read_error(pplan) == 0
    for b in [0, 1, 2, 31, 32, 33, 4095, 8191, 12288, B - 5, B - 4, B - 3, B - 2, B - 1] + [int(x) for x in rng.integers(0, B, 40)]:
        k, v, n = c["k"][0][b], c["v"][0][b], c["lens"][b]
        p = 0
        for g in range(2):
            if c["starts"][g] <= b < c["starts"][g + 1]:
                p = c["prefixes"][g]
                k, v = torch.cat([c["k"][1][g], k]), torch.cat([c["v"][1][g], v])
        tl.check_rows(out[b:b + 1], lse[b:b + 1], tl.attend(c["q"][b:b + 1], k, v, [p + n]), False, f"request {b}")
