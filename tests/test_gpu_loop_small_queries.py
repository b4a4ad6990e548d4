"""Query rows far from one in size over an e4m3 cache, whose queries are split into e4m3 numbers at a power of two:
rows down to bfloat16's smallest numbers and up to its largest, and infinite ones."""
import math

import pytest
import torch

import _gpu
import _loop
import _tiles
from load_balanced_paged_02_gb300 import binding as hb
from load_balanced_paged_02_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


def cache(lens, hkv, seed, size):
    """An e4m3 cache whose keys are about `size`, scales powers of two times as large as _tiles makes them."""
    c = _tiles.make_cache([lens], hkv, "e4m3", seed)
    c["k_scale"] *= size
    c["k"][0] = [k * size for k in c["k"][0]]
    return c


def weights(c, q, starts, lens, lse=None):
    """The call's weights, their definition and the bound on each one's error. A row's codes are multiples of 2^-9 of its
    power of two, which is 2^-126 at least: for rows under 2^-117 a product's error is up to 2^-136 |k| beside the
    bound's own terms."""
    lse = _loop.row_lse(q, starts, c["k"][0], lens) if lse is None else lse
    old = torch.rand((len(lens), c["k_cache"].shape[2], c["tables"][0].shape[1] * 64), device="cuda")
    w = old.clone()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    hb.hpc_attn_weights(q, c["k_cache"], c["tables"][0], _tiles.i32(lens), lse, w, q_starts=_tiles.i32(starts), k_scale=c["k_scale"],
                        error_word=word)
    assert int(word.item()) == 0
    want, bound = _loop.attn_weights(q, starts, lse, c["k"][0], lens, old, fp8=True)
    for b, total in enumerate(lens):
        off = 2.0 ** -136 * c["k"][0][b].abs().sum(-1).max().item() / math.sqrt(128)
        bound[b, :, :total] += 2 * off * want[b, :, :total]
    return w, want, bound


@pytest.mark.parametrize("new", [[1, 3], [8, 40]])
@pytest.mark.parametrize("size, key", [(1e-35, 1.0), (1e-36, 1.0), (1e-37, 1.0), (1e-38, 1.0), (1e-38, 2.0 ** 100),
                                       (2.0 ** -132, 1.0)])
def test_weights_of_small_rows(size, key, new):
    lens = [200, 321]
    c = cache(lens, 2, 5, key)
    starts = _tiles.starts(new)
    q = _tiles.make_q((starts[-1], 16, 128), 6, scale=size)
    q[:, 1, 3:] = 0.0                       # zeros beside small numbers
    q[0, 4] = 0.0
    q[-1, 5] = _tiles.make_q((128,), 7)     # and a row of ordinary size
    if key > 1.0:
        q[-1, 5] *= 1.0 / key
    w, want, bound = weights(c, q, starts, lens)
    assert torch.isfinite(w).all()
    assert ((w.double() - want).abs() <= bound)[bound > 0].all()


@pytest.mark.parametrize("new", [[1, 3], [8, 40]])
@pytest.mark.parametrize("size, key", [(1e-36, 2.0 ** 120), (1e-30, 2.0 ** 100), (1e-37, 2.0 ** 122), (1e-34, 2.0 ** 112)])
def test_weights_of_small_rows_and_large_keys(size, key, new):
    """Scores of about one from numbers at the ends of float32's range, and a token of small keys among the large ones."""
    lens = [200, 321]
    c = cache(lens, 2, 5, key)
    page, slot = int(c["tables"][0][1, 1]), 9
    c["k_scale"][page, :, slot] = 2.0 ** -70
    c["k"][0][1][64 + slot] = c["k_cache"][page, slot].float().double() * 2.0 ** -70
    starts = _tiles.starts(new)
    q = _tiles.make_q((starts[-1], 16, 128), 6, scale=size)
    q[:, 1, 3:] = 0.0
    w, want, bound = weights(c, q, starts, lens)
    assert torch.isfinite(w).all()
    assert ((w.double() - want).abs() <= bound)[bound > 0].all()


def test_scales_behind_the_length():
    """Large scales in unused slots change no bit."""
    lens, starts = [200, 321], [0, 2, 12]
    c = cache(lens, 1, 31, 2.0 ** -80)
    q = (_tiles.make_q((12, 8, 128), 32).float() * 2.0 ** 80).to(torch.bfloat16)
    w0, want, bound = weights(c, q, starts, lens)
    assert ((w0.double() - want).abs() <= bound)[bound > 0].all()
    lse = _loop.row_lse(q, starts, c["k"][0], lens)
    out = []
    for value in (1.0, 2.0 ** 120):
        ks = c["k_scale"].clone()
        for b, n in enumerate(lens):
            ks[int(c["tables"][0][b, n // 64]), :, n % 64:] = value
        w = torch.zeros_like(w0)
        hb.hpc_attn_weights(q, c["k_cache"], c["tables"][0], _tiles.i32(lens), lse, w, q_starts=_tiles.i32(starts), k_scale=ks)
        out.append(w)
    assert torch.equal(out[0], out[1])


def test_a_small_row_without_a_weight():
    """Log-sum-exps of -inf: no weight, whatever the row's size."""
    lens, starts = [200], [0, 2]
    c = cache(lens, 1, 8, 1.0)
    q = _tiles.make_q((2, 8, 128), 9, scale=1e-37)
    q[:, :, ::2] = 0.0
    w, want, bound = weights(c, q, starts, lens, lse=torch.full((2, 8), -math.inf, device="cuda"))
    assert torch.equal(w[0, 0, 198:200], torch.zeros(2, device="cuda"))
    assert ((w.double() - want).abs() <= bound)[bound > 0].all()


def large(shape, seed):
    """bfloat16 numbers up to the largest."""
    q = _tiles.make_q(shape, seed).float().clamp(-4, 4) * 8e37
    q[..., 0] = 3.38e38
    q[..., 1] = -3.1e38
    return q.to(torch.bfloat16)


def tiny_codes(shape, seed):
    """e4m3 codes of about one, for scales of 2^-126."""
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.float8_e4m3fn).to("cuda")


def test_weights_of_large_rows():
    """The largest finite numbers against keys of 2^-126: ordinary scores."""
    lens, starts = [200, 321], [0, 2, 12]
    c = cache(lens, 1, 12, 1.0)
    c["k_cache"].copy_(tiny_codes(c["k_cache"].shape, 11))
    c["k_scale"].fill_(2.0 ** -126)
    c["k"][0] = [(c["k_cache"][c["tables"][0][b, :-(-n // 64)].long()].float().double() * 2.0 ** -126).view(-1, 1, 128)[:n]
                 for b, n in enumerate(lens)]
    w, want, bound = weights(c, large((12, 8, 128), 13), starts, lens)
    assert torch.isfinite(w).all()
    assert ((w.double() - want).abs() <= bound)[bound > 0].all()


def test_weights_of_infinite_rows():
    """A row of one infinity and zeros: exp of plus or minus infinity, by the key's sign, NaN where that is 0, beside the other
    heads' seven rows of zeros."""
    lens, starts = [200], [0, 1]
    c = cache(lens, 1, 14, 1.0)
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    q[0, 2, 17] = math.inf
    old = torch.zeros((1, 1, 256), device="cuda")
    hb.hpc_attn_weights(q, c["k_cache"], c["tables"][0], _tiles.i32(lens), torch.zeros((1, 8), device="cuda"), old, q_starts=_tiles.i32(starts),
                        k_scale=c["k_scale"])
    key = c["k"][0][0][:, 0, 17]
    got = old[0, 0, :200]
    assert torch.isinf(got[key > 0]).all() and torch.equal(got[key < 0], torch.full_like(got[key < 0], 7.0))
    assert torch.isnan(got[key == 0]).all()


@pytest.mark.parametrize("engine", [hb.ENGINE_MMA_SYNC, hb.ENGINE_TCGEN05], ids=["mma_sync", "tcgen05"])
@pytest.mark.parametrize("q_len", [2, 8])
@pytest.mark.parametrize("size", [1e-35, 1e-36, 1e-38, 2.0 ** -132])
def test_decode_of_small_rows(size, q_len, engine):
    """The multi-token decode over an e4m3 cache: all tokens alike."""
    case = wl.make_case(wl.Workload("t", 3, 8, 1, "fp8", 21, lens=[130, 700, 5], q_len=q_len), device="cuda:0")
    case["q"].copy_((case["q"].float() * size).to(torch.bfloat16))
    case["q"][:, :, 3, 5:] = 0.0
    _gpu.check_full(case, _gpu.run(case, num_ctas=7, min_chunks=1, engine=engine))


def test_decode_of_large_rows():
    case = wl.make_case(wl.Workload("t", 3, 8, 1, "fp8", 22, lens=[130, 700, 5], q_len=3), device="cuda:0")
    case["q"].copy_(large(case["q"].shape, 23))
    case["k_cache"].copy_(tiny_codes(case["k_cache"].shape, 24))
    case["k_scale"].fill_(2.0 ** -126)
    _gpu.check_full(case, _gpu.run(case, num_ctas=7, min_chunks=1, engine=hb.ENGINE_TCGEN05))


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_rows_that_are_not_finite_stay_alone(value):
    """One head's row with an infinity or NaN: its weights' KV head and its own output are not numbers, all else has the
    bits that it has beside an ordinary row."""
    lens, starts = [200, 321], [0, 2, 12]
    c = cache(lens, 2, 41, 1.0)
    q = _tiles.make_q((12, 16, 128), 42)
    lse = _loop.row_lse(q, starts, c["k"][0], lens)
    bad = q.clone()
    bad[5, 3, 17] = value
    out = []
    for x in (q, bad):
        w = torch.zeros((2, 2, c["tables"][0].shape[1] * 64), device="cuda")
        hb.hpc_attn_weights(x, c["k_cache"], c["tables"][0], _tiles.i32(lens), lse, w, q_starts=_tiles.i32(starts), k_scale=c["k_scale"])
        out.append(w)
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1, 1], out[1][1, 1])
    assert torch.equal(out[0][1, 0, 315:], out[1][1, 0, 315:])                 # tokens that row 5 does not see
    seen = out[1][1, 0, :315]
    assert (torch.isinf(seen) | torch.isnan(seen) | (seen < out[0][1, 0, :315])).all()   # exp(-inf): less by the row's part

    case = wl.make_case(wl.Workload("t", 3, 8, 1, "fp8", 25, lens=[130, 700, 5], q_len=3), device="cuda:0")
    clean = _gpu.run(case, num_ctas=7, min_chunks=1, engine=hb.ENGINE_TCGEN05)
    case["q"][1, 1, 2, 9] = value
    dirty = _gpu.run(case, num_ctas=7, min_chunks=1, engine=hb.ENGINE_TCGEN05)
    same = torch.ones(clean["out"].shape[:-1], dtype=torch.bool, device="cuda")
    same[1, 1, 2] = False
    assert torch.equal(clean["out"][same], dirty["out"][same]) and torch.equal(clean["lse"][same], dirty["lse"][same])
    assert not torch.equal(clean["out"][1, 1, 2], dirty["out"][1, 1, 2])
