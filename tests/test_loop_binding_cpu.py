"""Refusals of the calls between two attention steps in the Python binding, by shapes and types alone (CPU tensors,
which the calls refuse too, but later: each test looks for the earlier message)."""
import pytest
import torch

from load_balanced_paged_02_gb300 import _build
from load_balanced_paged_02_gb300 import binding as hb


@pytest.fixture(scope="module", autouse=True)
def L():
    _build.build()
    return hb.lib()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f32(*shape):
    return torch.zeros(shape)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def refused(call, match):
    with pytest.raises(hb.HpcError, match=match):
        call()


def test_attn_weights():
    def call(q=None, k=None, table=None, lens=None, lse=None, w=None, **kw):
        q = bf16(2, 8, 128) if q is None else q
        return hb.hpc_attn_weights(q, bf16(4, 64, 1, 128) if k is None else k, i32(2, 3) if table is None else table,
                                   i32(2) if lens is None else lens, f32(*q.shape[:-1]) if lse is None else lse,
                                   f32(2, 1, 192) if w is None else w, **kw)
    refused(call, "CUDA device")
    refused(lambda: call(k=bf16(4, 64, 1, 64)), "heads, 128")
    refused(lambda: call(q=f32(2, 8, 128)), "bfloat16")
    refused(lambda: call(q=bf16(3, 8, 128)), "differ in requests")
    refused(lambda: call(q=bf16(2, 2, 8, 128), q_starts=i32(3)), "dimensions")
    refused(lambda: call(q_starts=i32(2)), "3 values")
    refused(lambda: call(table=i32(3, 3)), "2 rows")
    refused(lambda: call(lens=f32(2)), "int32")
    refused(lambda: call(lse=f32(2, 7)), "shape")
    refused(lambda: call(w=f32(2, 2, 192)), "batch, KV heads, tokens")
    refused(lambda: call(w=f32(2, 1, 192).half()), "float32")
    refused(lambda: call(w=f32(2, 1, 400)[:, :, :192]), "contiguous")
    refused(lambda: call(counts=i32(3)), "2 values")
    refused(lambda: call(num_pages=5), "4")
    refused(lambda: call(k=torch.zeros((4, 64, 1, 128), dtype=torch.uint8)), "scales")
    refused(lambda: call(k=torch.zeros((4, 64, 1, 128), dtype=torch.uint8), k_scale=f32(4, 64, 1)), "shape")
    refused(lambda: call(error_word=f32(1)), "error_word")


def test_kv_select():
    def call(w=None, lens=None, budget=8, **kw):
        return hb.hpc_kv_select(f32(2, 1, 100) if w is None else w, i32(2) if lens is None else lens, budget, **kw)
    refused(call, "CUDA device")
    refused(lambda: call(w=f32(3, 1, 100)), "batch")
    refused(lambda: call(w=f32(2, 100)), "batch")
    refused(lambda: call(lens=i32(2).long()), "int32")
    refused(lambda: call(budget=0), "budget")
    refused(lambda: call(keep=i32(2, 1, 9)), "shape")
    refused(lambda: call(keep_lens=i32(3)), "2 values")


def test_kv_compact():
    cache = bf16(4, 64, 1, 128)

    def call(k=cache, v=cache, table=None, keep=None, kl=None, new=None, **kw):
        return hb.hpc_kv_compact(k, v, i32(2, 3) if table is None else table, i32(2, 1, 70) if keep is None else keep,
                                 i32(2) if kl is None else kl, i32(2, 2) if new is None else new, **kw)
    refused(call, "CUDA device")
    refused(lambda: call(v=bf16(4, 64, 2, 128)), "one type")
    refused(lambda: call(keep=i32(2, 2, 70)), "batch, 1, tokens")
    refused(lambda: call(kl=i32(3)), "2 values")
    refused(lambda: call(table=i32(3, 3)), "2 rows")
    refused(lambda: call(new=i32(1, 2)), "2 rows")
    refused(lambda: call(weights=f32(2, 1, 192)), "together")
    refused(lambda: call(weights=f32(2, 1, 192), weights_out=f32(2, 2, 70)), "batch")


def test_verify_drafts():
    def call(p=None, d=None, u=None, us=None, **kw):
        return hb.hpc_verify_drafts(f32(2, 4, 50) if p is None else p, i32(2, 3) if d is None else d, f32(2, 3) if u is None else u,
                                    f32(2) if us is None else us, **kw)
    refused(call, "CUDA device")
    refused(lambda: call(p=f32(2, 4, 50).half()), "dtype")
    refused(lambda: call(p=f32(2, 3, 50)), "shape")
    refused(lambda: call(p=f32(2, 4, 0)), "vocabulary")
    refused(lambda: call(p=f32(2, 4, 100)[:, :, ::2]), "contiguous")
    refused(lambda: call(p=f32(3, 4, 50)[::2]), "evenly")
    refused(lambda: call(draft_probs=f32(2, 4, 50)), "shape")
    refused(lambda: call(draft_probs=bf16(2, 3, 50)), "float32")
    refused(lambda: call(u=f32(2, 4)), "shape")
    refused(lambda: call(us=f32(3)), "shape")
    refused(lambda: call(d=i32(2, 3).long()), "int32")
    refused(lambda: call(draft_counts=i32(3)), "2 values")
    refused(lambda: call(tokens=i32(2, 3)), "shape")
    refused(lambda: call(kept_lens=i32(2)), "seq_lens")


def test_numbers_are_not_cut_to_32_bits():
    def weights(window):
        return hb.hpc_attn_weights(bf16(2, 8, 128), bf16(4, 64, 1, 128), i32(2, 3), i32(2), f32(2, 8), f32(2, 1, 192), window=window)

    def select(budget=8, **kw):
        return hb.hpc_kv_select(f32(2, 1, 100), i32(2), budget, **kw)
    for x in ((1 << 32) + 5, 1 << 31, -1):
        refused(lambda: weights(x), "window")
        refused(lambda: select(num_first=x), "num_first")
        refused(lambda: select(num_recent=x), "num_recent")
    refused(lambda: select(budget=(1 << 32) + 5), "budget")


def test_the_package_names_them():
    import load_balanced_paged_02_gb300 as pkg
    for name in ("hpc_attn_weights", "hpc_kv_select", "hpc_kv_compact", "hpc_verify_drafts"):
        assert getattr(pkg, name) is getattr(hb, name)
