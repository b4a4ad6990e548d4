"""The lengths that hpc_verify_drafts gives back, at the ends of int32."""
import pytest
import torch

from load_balanced_paged_02_gb300 import binding as hb

pytestmark = pytest.mark.gpu


def test_lengths_at_the_lower_end():
    """Lengths of int32's least numbers, that the refused tokens would take below it: 0, as all that fall below 0."""
    B, n, V = 4, 3, 100
    lens = torch.tensor([-2147483648, -2147483647, 2, 2147483647], dtype=torch.int32, device="cuda")
    target = torch.full((B, n + 1, V), 0.01, device="cuda")
    drafted = torch.full((B, n), 100, dtype=torch.int32, device="cuda")     # all refused
    kept = torch.full((B,), 7, dtype=torch.int32, device="cuda")
    acc, _ = hb.hpc_verify_drafts(target, drafted, torch.zeros((B, n), device="cuda"), torch.zeros(B, device="cuda"), seq_lens=lens,
                                  kept_lens=kept)
    assert acc.tolist() == [0] * B and kept.tolist() == [0, 0, 0, 2147483644]
