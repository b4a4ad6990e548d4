"""One request's tokens in the place of its drafts."""
import pytest
import torch

import _loop
from load_balanced_paged_02_gb300 import binding as hb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [300, 4097, 131072])
@pytest.mark.parametrize("given", [True, False])
def test_one_request(V, given):
    n = 7
    gen = torch.Generator(device="cuda").manual_seed(V)
    target = torch.softmax(torch.randn((1, n + 1, V), generator=gen, device="cuda"), -1)
    draft = torch.softmax(torch.randn((1, n, V), generator=gen, device="cuda"), -1) if given else None
    for k in range(20):
        buf = torch.randint(0, V, (1, n + 1), generator=gen, device="cuda", dtype=torch.int32)
        drafted = buf[:, :n].clone()
        accept = torch.rand((1, n), generator=gen, device="cuda") * (0.1 if given else 0.5 / V)
        sample = torch.rand(1, generator=gen, device="cuda")
        wa, wt = _loop.verify(target, draft, drafted, accept, sample)
        acc, tok = hb.hpc_verify_drafts(target, buf[:, :n], accept, sample, draft_probs=draft, tokens=buf)
        assert tok is buf and torch.equal(acc.cpu(), wa) and torch.equal(buf.cpu(), wt)
