"""hpc_verify_drafts where entries are no probabilities: the one rule that the sum of a row, the search in it and the
acceptance of drafts follow."""
import numpy as np
import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def definition(target, draft, drafted, accept, sample):
    """In 64 bits. A q whose sign is set counts as 0. A p that is accepted or drawn from, and a difference p - q that is drawn
    from, counts as 0 unless it is above 0 and below 2^64; comparisons with NaN refuse."""
    p, q = target.double().cpu().numpy(), draft.double().cpu().numpy()
    q = np.where(np.signbit(q), 0.0, q)
    d, u, us = drafted.cpu().numpy(), accept.double().cpu().numpy(), sample.double().cpu().numpy()

    def clean(x):
        return np.where((x > 0) & (x < 2.0 ** 64), x, 0.0)

    accepted, tokens = [], []
    with np.errstate(invalid="ignore"):
        for b in range(d.shape[0]):
            r = 0
            while r < d.shape[1] and u[b, r] * q[b, r, d[b, r]] < clean(p[b, r, d[b, r]]):
                r += 1
            rest = clean(p[b, r] - q[b, r]) if r < d.shape[1] else clean(p[b, r])
            if rest.sum() == 0:
                rest = clean(p[b, r])
            sums = np.cumsum(rest)
            if sums[-1] == 0:
                token = -1
            else:
                over = np.nonzero((sums > us[b] * sums[-1]) & (rest > 0))[0]
                token = int(over[0]) if len(over) else int(np.nonzero(rest > 0)[0][-1])
            accepted.append(r)
            tokens.append(d[b, :r].tolist() + [token] + [-1] * (d.shape[1] - r))
    return accepted, tokens


def check(target, draft, drafted, accept, sample):
    acc, tok = hb.hpc_verify_drafts(target, drafted, accept, sample, draft_probs=draft)
    wa, wt = definition(target, draft, drafted, accept, sample)
    assert acc.tolist() == wa
    assert tok.tolist() == wt


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("V", [257, 5003, 100003, 131072])
@pytest.mark.parametrize("share", [0.0, 0.02, 1.0])
def test_negative_entries(V, pad, share, kind):
    """Draft entries below 0 in some places or all (with share 0: one of them), target entries below 0 and NaN among those
    too, rows on 16 bytes and off them."""
    B = 24
    gen = torch.Generator(device="cuda").manual_seed(V + pad)
    target = torch.zeros((B, 3, V + pad), dtype=kind, device="cuda")[:, :, :V]
    draft = torch.zeros((B, 2, V + pad), dtype=kind, device="cuda")[:, :, :V]
    target.copy_(torch.rand(target.shape, generator=gen, device="cuda") / V)
    draft.copy_(torch.rand(draft.shape, generator=gen, device="cuda") / V)
    drafted = torch.randint(0, V, (B, 2), generator=gen, device="cuda", dtype=torch.int32)
    accept = torch.rand((B, 2), generator=gen, device="cuda")
    sample = torch.rand(B, generator=gen, device="cuda")
    check(target, draft, drafted, accept, sample)
    if share:
        draft[torch.rand(draft.shape, generator=gen, device="cuda") < share] *= -3.0
    else:
        draft[:, :, V // 2] = -0.25
    check(target, draft, drafted, accept, sample)
    target[torch.rand(target.shape, generator=gen, device="cuda") < 0.3] *= -1.0   # both below 0 where q is
    check(target, draft, drafted, accept, sample)
    target[:, :, 7] = NAN
    draft[:, :, 7] = -0.5
    target[:, :, 9], draft[:, :, 9] = -1.0, -INF
    target[:, :, 11], draft[:, :, 11] = 0.125, -INF
    target[:, :, 13], draft[:, :, 13] = 0.25, NAN
    target[:, :, 15], draft[:, :, 15] = 0.25, INF
    target[:, :, 17], draft[:, :, 17] = INF, -1.0
    target[:, :, 19], draft[:, :, 19] = 0.25, -0.0
    for u in (None, 0.0, 1.0 - 2.0 ** -24, 1.0):
        check(target, draft, drafted, accept, sample if u is None else torch.full_like(sample, u))


def test_acceptance():
    """(p, q) of the drafted token, and whether it is accepted, for random numbers from 0 on."""
    pairs = [(0.0, -1.0, False), (-0.5, -2.0, False), (-1.0, -0.5, False), (0.25, -1.0, True), (0.25, -INF, True), (INF, 0.25, False),
             (2.0 ** 64, 0.25, False), (2.0 ** 63, 0.25, True), (INF, INF, False), (0.25, INF, False), (0.25, NAN, False), (NAN, 0.25, False),
             (NAN, -1.0, False), (0.25, -0.0, True), (0.25, 0.0, True), (0.0, 0.0, False)]
    B, V = len(pairs), 40
    target = torch.full((B, 2, V), 1 / 64, device="cuda")
    draft = torch.full((B, 1, V), 1 / 128, device="cuda")
    for b, (p, q, _) in enumerate(pairs):
        target[b, 0, 5], draft[b, 0, 5] = p, q
    drafted = torch.full((B, 1), 5, dtype=torch.int32, device="cuda")
    sample = torch.full((B,), 0.5, device="cuda")
    for u in (0.0, 2.0 ** -30, 0.5, 1.0 - 2.0 ** -24):
        accept = torch.full((B, 1), u, device="cuda")
        acc, _ = hb.hpc_verify_drafts(target, drafted, accept, sample, draft_probs=draft)
        assert [bool(x) for x in acc.tolist()] == [ok for _, _, ok in pairs]
        check(target, draft, drafted, accept, sample)


@pytest.mark.parametrize("kind, bits", [(torch.float32, torch.int32), (torch.bfloat16, torch.int16)])
def test_signs_of_nan(kind, bits):
    """A NaN whose sign is set, as some processors make them, counts as 0 like every q whose sign is set; another leaves
    nothing. 40000 entries: several warps' parts."""
    B, V = 6, 40000
    gen = torch.Generator(device="cuda").manual_seed(3)
    target = (torch.rand((B, 2, V), generator=gen, device="cuda") / V).to(kind)
    draft = (torch.rand((B, 1, V), generator=gen, device="cuda") / V).to(kind)
    plus, minus = (0x7fc00000, 0xffc00000 - (1 << 32)) if kind == torch.float32 else (0x7fc0, 0xffc0 - (1 << 16))
    draft.view(bits)[:, :, 100:300] = minus
    draft.view(bits)[:, :, 300:500] = plus
    target[:, :, 100:500] = 0.25
    drafted = torch.tensor([[100], [200], [300], [400], [100], [39999]], dtype=torch.int32, device="cuda")
    for u in (0.0, 0.25, 0.75):
        check(target, draft, drafted, torch.full((B, 1), u, device="cuda"), torch.rand(B, generator=gen, device="cuda"))


def test_random_numbers_that_are_none():
    """A sample_rand of NaN gives the last entry above 0, one below 0 the first; an accept_rand of NaN refuses."""
    B, V = 3, 50000
    target = torch.zeros((B, 2, V), device="cuda")
    target[:, :, 7000:9000] = 2.0 ** -12
    draft = torch.full((B, 1, V), 2.0 ** -16, device="cuda")
    drafted = torch.full((B, 1), 8000, dtype=torch.int32, device="cuda")
    sample = torch.tensor([NAN, -1.0, 2.0], device="cuda")
    for accept, r in ((0.0, 1), (NAN, 0)):
        acc, tok = hb.hpc_verify_drafts(target, drafted, torch.full((B, 1), accept, device="cuda"), sample, draft_probs=draft)
        assert acc.tolist() == [r] * B
        assert [row[r] for row in tok.tolist()] == [8999, 7000, 8999]
