"""hpc_kv_write and hpc_kv_read against elementary operations."""
import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb
import _tiles as tl

pytestmark = pytest.mark.gpu


def pool(pages, hkv, kv):
    """Caches full of marks (code 0x55, scale -3; 0x5555 for bf16)."""
    n = (pages, 64, hkv, 128)
    if kv == "bf16":
        c = [torch.full(n, 0x5555, dtype=torch.int16, device="cuda").view(torch.bfloat16) for _ in range(2)]
        return c + [None, None]
    c = [torch.full(n, 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    return c + [torch.full((pages, hkv, 64), -3.0, device="cuda") for _ in range(2)]


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.uint8)


def quantised(x):
    """Codes and scales of rows x [T, hkv, 128] (bf16), from the rule, in float64 and rounded once to
    float32 where the rule has a float32."""
    amax = x.double().abs().amax(dim=-1)
    scale = (amax / 448.0).float()
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    q = (x.double() / scale.double().unsqueeze(-1))
    return q, scale


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("tokens", [1, 2, 63, 500])
def test_write(tokens, hkv, kv):
    gen = torch.Generator(device="cuda").manual_seed(tokens * 10 + hkv)
    pages = tokens // 64 + 3
    # strides: K and V as parts of a wider row, and with an odd number of heads between tokens
    wide = torch.randn((tokens, 10 * hkv + 1, 128), generator=gen, device="cuda")
    wide *= torch.exp(3 * torch.randn((tokens, 10 * hkv + 1, 1), generator=gen, device="cuda"))
    if tokens > 2:
        wide[1] = 0.0          # rows of zeros
        wide[2, :, 5:] = 0.0   # and nearly
    wide = wide.to(torch.bfloat16)
    k, v = wide[:, 8 * hkv:9 * hkv], wide[:, 9 * hkv:10 * hkv]
    slots = torch.randperm(pages * 64, generator=gen, device="cuda")[:tokens].int()
    if tokens > 10:
        slots[::7] = -1
    kc, vc, ks, vs = pool(pages, hkv, kv)
    before = [t.clone() if t is not None else None for t in (kc, vc, ks, vs)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    hb.hpc_kv_write(k, v, slots, kc, vc, ks, vs, error_word=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    live = slots >= 0
    page, slot = slots[live].long() // 64, slots[live].long() % 64
    for x, cache, scale, old, old_scale in ((k, kc, ks, before[0], before[2]), (v, vc, vs, before[1], before[3])):
        touched = torch.zeros((pages, 64), dtype=torch.bool, device="cuda")
        touched[page, slot] = True
        assert torch.equal(bits(cache)[~touched], bits(old)[~touched]), "a slot that was not named changed"
        if kv == "bf16":
            assert torch.equal(bits(cache[page, slot]), bits(x[live].contiguous()))
            continue
        q, want = quantised(x[live])
        assert torch.equal(scale.transpose(1, 2)[page, slot], want)
        got = bits(cache)[page, slot].view(torch.float8_e4m3fn).double()
        nearest = q.clamp(-448, 448).to(torch.float32).to(torch.float8_e4m3fn).double()
        # a code is the nearest value of the type to the quotient; the quotient's own rounding to float32 may
        # decide a tie only (2^-24 of it)
        wrong = got != nearest
        assert ((got - q).abs()[wrong] <= (nearest - q).abs()[wrong] + 2.0 ** -23 * q.abs()[wrong]).all()
        assert wrong.float().mean() < 1e-3
        assert torch.equal(scale.transpose(1, 2)[~touched], old_scale.transpose(1, 2)[~touched])


def test_write_extremes():
    """Values at the ends of bf16: the scale stays finite and every code a number; NaN stays NaN."""
    big, tiny = torch.finfo(torch.bfloat16).max, 1e-38
    rows = torch.zeros((6, 1, 128), device="cuda")
    rows[0], rows[1], rows[2, 0, 3] = big, tiny, -big
    rows[3, 0, :2] = torch.tensor([9.2e-41, -9.2e-41], device="cuda")
    rows[4], rows[5, 0, 7] = 448.0, float("nan")
    rows = rows.to(torch.bfloat16)
    kc, vc, ks, vs = pool(1, 1, "e4m3")
    hb.hpc_kv_write(rows, rows, tl.i32(range(6)), kc, vc, ks, vs)
    torch.cuda.synchronize()
    val = kc[0, :6].float() * ks[0, 0, :6].view(6, 1, 1)
    assert torch.isfinite(ks[0, 0, :6]).all() and torch.isfinite(kc[0, :5].float()).all()
    x = rows[:5].double()
    step = torch.where(x.abs().amax(dim=-1, keepdim=True) > 0, x.abs().amax(dim=-1, keepdim=True) / 448, 1.0)
    # half a step of the type (2^-4 of the value, 2^-10 of the scale where it is subnormal), and float32's own ends
    assert ((val[:5].double() - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * step + 2e-45 * 448).all()
    assert torch.isnan(kc[0, 5, 0, 7].float()) and torch.equal(bits(kc[0, :6]), bits(vc[0, :6]))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_write_slots_out_of_range(kv):
    kc, vc, ks, vs = pool(2, 1, kv)
    old = bits(kc).clone()
    k = torch.ones((3, 1, 128), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    hb.hpc_kv_write(k, k, tl.i32([128, 2147483647, 5]), kc, vc, ks, vs, error_word=err)
    torch.cuda.synchronize()
    assert err.item() == 4
    changed = (bits(kc) != old).flatten(2).any(dim=2)
    assert changed.sum() == 1 and changed[0, 5]
    # num_pages below the cache's: the pages past it are not written
    hb.hpc_kv_write(k[:1], k[:1], tl.i32([70]), kc, vc, ks, vs, num_pages=1, error_word=err)
    torch.cuda.synchronize()
    assert ((bits(kc) != old).flatten(2).any(dim=2).sum() == 1)
    hb.hpc_kv_write(k[:0], k[:0], tl.i32([]), kc, vc, ks, vs)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("lens,first", [([1], [0]), ([37, 0, 128, 300, 0, 65], [0, 5, 64, 131, 0, 1]), ([700, 900], [63, 1])])
def test_read(lens, first, hkv, kv):
    c = tl.make_cache([[n + f for n, f in zip(lens, first)]], hkv, kv, seed=sum(lens))
    rows = sum(lens) + 4
    starts = [2] + [2 + x for x in tl.starts(lens)[1:]]
    for use_first in (True, False):
        k, v = (torch.full((rows, hkv, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        hb.hpc_kv_read(c["k_cache"], c["v_cache"], c["tables"][0], tl.i32(starts), k, v, c["k_scale"], c["v_scale"],
                       first=tl.i32(first) if use_first else None, error_word=err)
        torch.cuda.synchronize()
        assert err.item() == 0
        for got, exact, cache, scale in ((k, c["k"], c["k_cache"], c["k_scale"]), (v, c["v"], c["v_cache"], c["v_scale"])):
            want = torch.cat([exact[0][b][(f if use_first else 0):][:n] for b, (n, f) in enumerate(zip(lens, first))])
            mine = got[2:2 + sum(lens)]
            assert (got[:2] == 9).all() and (got[2 + sum(lens):] == 9).all(), "rows of no request changed"
            if kv == "bf16":
                assert torch.equal(mine.double(), want)
            else:  # code x scale: rounded to float32, then to bf16
                assert torch.equal(mine, want.float().to(torch.bfloat16))


def test_read_many_requests_and_bad_pages():
    """More requests than the kernel keeps starts of; bad page ids and tokens beyond the table read as zeros."""
    n = 3000
    lens = [(b * 7) % 5 for b in range(n)]
    c = tl.make_cache([lens], 1, "bf16", seed=2)
    k, v = (torch.empty((sum(lens), 1, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    hb.hpc_kv_read(c["k_cache"], c["v_cache"], c["tables"][0], tl.i32(tl.starts(lens)), k, v)
    torch.cuda.synchronize()
    assert torch.equal(k.double(), torch.cat(c["k"][0])) and torch.equal(v.double(), torch.cat(c["v"][0]))
    c = tl.make_cache([[130]], 2, "e4m3", seed=3)
    table = c["tables"][0].clone()
    table[0, 1] = c["pages"]
    k, v = (torch.full((200, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    hb.hpc_kv_read(c["k_cache"], c["v_cache"], table, tl.i32([0, 200]), k, v, c["k_scale"], c["v_scale"], error_word=err)
    torch.cuda.synchronize()
    assert err.item() == 4 and (k[64:128] == 0).all() and (k[192:] == 0).all()
    assert torch.equal(k[:64], c["k"][0][0][:64].float().to(torch.bfloat16))
    hb.hpc_kv_read(c["k_cache"], c["v_cache"], table, tl.i32([0, 10]), k, v, c["k_scale"], c["v_scale"], first=tl.i32([-3]), error_word=err)
    torch.cuda.synchronize()
    assert (k[:3] == 0).all() and torch.equal(k[3:10], c["k"][0][0][:7].float().to(torch.bfloat16))


def test_round_trip_far_pages_graph_and_refusals():
    hkv, pages = 8, 33000
    kc, vc = (torch.zeros((pages, 64, hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    k, v = (torch.randn((130, hkv, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    table = tl.i32([pages - 1, 7, pages - 2]).view(1, 3)
    slots = tl.i32([int(table[0, t // 64]) * 64 + t % 64 for t in range(130)])
    out = [torch.empty_like(k) for _ in range(2)]
    st = tl.i32([0, 130])
    hb.hpc_kv_write(k, v, slots, kc, vc)
    hb.hpc_kv_read(kc, vc, table, st, out[0], out[1])
    torch.cuda.synchronize()
    assert torch.equal(out[0], k) and torch.equal(out[1], v)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        hb.hpc_kv_write(k, v, slots, kc, vc)
        hb.hpc_kv_read(kc, vc, table, st, out[0], out[1])
    k.mul_(2), v.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], k) and torch.equal(out[1], v)
    for bad in (lambda: hb.hpc_kv_write(k.float(), v, slots, kc, vc), lambda: hb.hpc_kv_write(k, v[:3], slots, kc, vc),
                lambda: hb.hpc_kv_write(k, v, slots[:4], kc, vc), lambda: hb.hpc_kv_write(k, v, slots.long(), kc, vc),
                lambda: hb.hpc_kv_write(k.transpose(0, 1), v, slots, kc, vc), lambda: hb.hpc_kv_write(k, v, slots.cpu(), kc, vc),
                lambda: hb.hpc_kv_read(kc, vc, table, st, out[0][:, :4], out[1]), lambda: hb.hpc_kv_read(kc, vc, table, st[:1], *out),
                lambda: hb.hpc_kv_read(kc, vc, table[0], st, *out), lambda: hb.hpc_kv_read(kc, vc.half(), table, st, *out)):
        with pytest.raises(hb.HpcError):
            bad()
