"""hpc_verify_drafts against its definition in 64 bits: whole numbers, which have to be equal."""
import pytest
import torch

import _loop
import _tiles
from load_balanced_paged_02_gb300 import binding as hb

pytestmark = pytest.mark.gpu


def make(B, n, V, kind, seed, given=True, sharp=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    logits = sharp * torch.randn((B, n + 1, V), generator=gen, device="cuda")
    target = torch.softmax(logits, -1).to(kind)
    draft = torch.softmax(logits[:, :n] + 0.5 * torch.randn((B, n, V), generator=gen, device="cuda"), -1).to(kind)
    drafted = torch.zeros((B, n), dtype=torch.int32, device="cuda")
    for i in range(n):
        drafted[:, i] = torch.multinomial(draft[:, i].float(), 1, generator=gen).squeeze(1).to(torch.int32)
    accept = torch.rand((B, n), generator=gen, device="cuda")
    sample = torch.rand((B,), generator=gen, device="cuda")
    return target, draft if given else None, drafted, accept, sample


def check(target, draft, drafted, accept, sample, counts=None, word=0):
    B, n = drafted.shape
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    tok = torch.full((B, n + 1), 77, dtype=torch.int32, device="cuda")
    lens = torch.arange(B, dtype=torch.int32, device="cuda") * 3
    kept = lens.clone()
    hb.hpc_verify_drafts(target, drafted, accept, sample, draft_probs=draft, draft_counts=None if counts is None else _tiles.i32(counts),
                         num_accepted=acc, tokens=tok, seq_lens=kept, kept_lens=kept, error_word=err)
    wa, wt = _loop.verify(target, draft, drafted, accept, sample, counts)
    assert torch.equal(acc.cpu(), wa)
    assert torch.equal(tok.cpu(), wt)
    assert torch.equal(kept, (lens - (n - acc)).clamp(min=0))
    assert int(err.item()) == word
    return wa


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("B, n, V", [
    (1, 3, 32000), (1, 0, 131072), (5, 1, 1), (7, 2, 2), (64, 5, 1000), (40, 31, 257), (3, 7, 100003), (33, 4, 4097), (200, 2, 5000),
    (2, 5, 50001), (80, 3, 33000),
])
def test_against_definition(B, n, V, given, kind):
    check(*make(B, n, V, kind, B * 31 + V, given))


def test_counts():
    t = make(9, 4, 3000, torch.float32, 5)
    check(*t, counts=[0, 1, 2, 3, 4, -3, 9, 0, 4])
    t = make(9, 4, 3000, torch.float32, 6, given=False)
    check(*t, counts=[0, 1, 2, 3, 4, -3, 9, 0, 4])


def test_all_and_none_accepted():
    target, draft, drafted, accept, sample = make(20, 6, 4000, torch.float32, 8)
    assert (check(target, draft, drafted, torch.zeros_like(accept), sample) >= 6).all()
    # drafts that the target gives nothing
    target = target.clone()
    for i in range(6):
        target[torch.arange(20), i, drafted[:, i].long()] = 0.0
    assert (check(target, draft, drafted, accept, sample) == 0).all()


def test_random_numbers_at_the_ends():
    target, draft, drafted, accept, sample = make(30, 2, 5000, torch.float32, 9)
    for u in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0 ** -149):
        check(target, draft, drafted, accept, torch.full_like(sample, u))
        check(target, draft, drafted, torch.full_like(accept, u), sample)


def test_one_candidate_and_gaps():
    """One-hot rows, rows whose weight lies at the ends, and long runs of zeros between."""
    B, V = 24, 40000
    target = torch.zeros((B, 2, V), device="cuda")
    at = torch.randint(0, V, (B, 2, 3), generator=torch.Generator().manual_seed(4)).cuda()
    target.scatter_(2, at, 0.25)
    target[:, :, 0] += 2.0 ** -30
    target[:, :, V - 1] += 2.0 ** -30
    target[0] = 0.0
    target[0, :, 17] = 1.0
    drafted = at[:, 0, :1].to(torch.int32).contiguous()
    gen = torch.Generator(device="cuda").manual_seed(6)
    for k in range(6):
        accept = torch.rand((B, 1), generator=gen, device="cuda")
        sample = torch.rand((B,), generator=gen, device="cuda") if k < 4 else torch.full((B,), float(k == 5), device="cuda")
        check(target, None, drafted, accept, sample)
        check(target, target[:, :1].contiguous(), drafted, accept, sample)


def test_nothing_left():
    """Draft and target alike where a draft is refused; rows of zeros; values that are not probabilities."""
    target, draft, drafted, accept, sample = make(12, 2, 3000, torch.float32, 11)
    draft = target[:, :2].clone()
    draft[torch.arange(12), 0, drafted[:, 0].long()] *= 4.0     # refused at most random numbers, and nothing is above q
    check(target, draft, drafted, torch.full_like(accept, 0.9), sample)
    zero = torch.zeros_like(target)
    check(zero, draft, drafted, accept, sample)
    wild = target.clone()
    wild[:, :, 5] = float("nan")
    wild[:, :, 6] = float("inf")
    wild[:, :, 7] = -float("inf")
    wild[:, :, 8] = -1.0
    d2 = draft.clone()
    d2[:, :, 9] = float("nan")
    d2[:, :, 10] = float("inf")
    check(wild, d2, drafted, accept, sample)
    check(wild, None, drafted, accept, sample)


def test_bad_tokens():
    target, draft, drafted, accept, sample = make(6, 3, 900, torch.float32, 12)
    drafted[1, 0], drafted[2, 1], drafted[3, 2] = -1, 900, 2147483647
    check(target, draft, drafted, torch.zeros_like(accept), sample, word=64)
    check(target, None, drafted, torch.zeros_like(accept), sample, word=64)


def test_sums_beyond_32_bits():
    """Running sums that float32 cannot hold apart: many small entries beside large ones, borders between neighbours."""
    B, V = 16, 131072
    gen = torch.Generator(device="cuda").manual_seed(13)
    target = torch.rand((B, 1, V), generator=gen, device="cuda") * 2.0 ** -20
    target[:, 0, 1000] = 1.0
    target[:, 0, 90000] = 0.5
    drafted = torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    accept = torch.zeros((B, 0), device="cuda")
    for k in range(4):
        check(target, None, drafted, accept, torch.rand((B,), generator=gen, device="cuda"))
    # at a border itself: the token behind it
    p = torch.full((1, 1, 1 << 16), 2.0 ** -16, device="cuda")
    for k in (0, 1, 255, 4096, 65535):
        acc, tok = hb.hpc_verify_drafts(p, drafted[:1], accept[:1], torch.full((1,), k * 2.0 ** -16, device="cuda"))
        assert int(tok[0, 0]) == k and int(acc[0]) == 0


def test_padded_rows_streams_and_graphs():
    target, draft, drafted, accept, sample = make(5, 3, 1001, torch.float32, 14)
    wide = torch.full((5, 4, 1100), 9.0, device="cuda")
    wide[:, :, :1001] = target
    wide_d = torch.full((5, 3, 1007), 9.0, device="cuda")
    wide_d[:, :, :1001] = draft
    check(wide[:, :, :1001], wide_d[:, :, :1001], drafted, accept, sample)
    wa, wt = _loop.verify(target, draft, drafted, accept, sample)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    acc, tok = hb.hpc_verify_drafts(target, drafted, accept, sample, draft_probs=draft, stream=s)
    s.synchronize()
    assert torch.equal(acc.cpu(), wa) and torch.equal(tok.cpu(), wt)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hb.hpc_verify_drafts(target, drafted, accept, sample, draft_probs=draft, num_accepted=acc, tokens=tok)
    t2 = make(5, 3, 1001, torch.float32, 15)
    for x, y in zip((target, draft, drafted, accept, sample), t2):
        x.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    wa, wt = _loop.verify(*t2)
    assert torch.equal(acc.cpu(), wa) and torch.equal(tok.cpu(), wt)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B, V, pad", [(1, 600000, 0), (2, 700001, 0), (300, 150000, 0), (3, 500000, 3), (260, 140001, 5)])
def test_parts_longer_than_a_piece(B, V, pad, kind):
    """A warp's part of the vocabulary in several pieces: dense rows, weight in few places, and rows that are zero but for
    a stretch; rows that begin off 16 bytes."""
    gen = torch.Generator(device="cuda").manual_seed(V + pad)
    target = torch.zeros((B, 2, V + pad), device="cuda", dtype=kind)[:, :, :V]
    draft = torch.zeros((B, 1, V + 2 * pad), device="cuda", dtype=kind)[:, :, :V]
    drafted = torch.randint(0, V, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
    accept = torch.rand((B, 1), generator=gen, device="cuda")
    for step in range(3):
        for x in (target, draft):
            if step == 0:
                x.copy_(torch.rand(x.shape, generator=gen, device="cuda") / V)
            elif step == 1:
                x.zero_()
                x.scatter_(2, torch.randint(0, V, (*x.shape[:2], 40), generator=gen, device="cuda"), 0.025)
            else:
                x.zero_()
                x[:, :, V // 3:V // 3 + 5000] = torch.rand((*x.shape[:2], 5000), generator=gen, device="cuda").to(kind)
        for u in (None, 0.0, 1.0 - 2.0 ** -24, 1.0):
            sample = torch.rand(B, generator=gen, device="cuda") if u is None else torch.full((B,), u, device="cuda")
            check(target, draft, drafted, accept, sample)
            check(target, None, drafted, accept, sample)


def test_rows_beyond_32_bits():
    """Probabilities whose last rows begin beyond 2^31 elements."""
    B, n, V = 3, 2, 3001
    target, draft, drafted, accept, sample = make(B, n, V, torch.bfloat16, 23)
    wide = 300_000_000
    t = torch.empty((B, n + 1, wide), dtype=torch.bfloat16, device="cuda")[:, :, :V]
    d = torch.empty((B, n, wide + 8), dtype=torch.bfloat16, device="cuda")[:, :, :V]
    t.copy_(target)
    d.copy_(draft)
    for u in (0.0, 0.5, 1.0):
        check(t, d, drafted, torch.full_like(accept, u), sample)
