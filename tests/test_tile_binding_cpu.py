"""Refusals of the prompt, shared-prefix and cache calls in the Python binding, by shapes alone (CPU tensors, which
the calls refuse too, but later: each test looks for the earlier message)."""
import pytest
import torch

from load_balanced_paged_02_gb300 import _build
from load_balanced_paged_02_gb300 import binding as hb


@pytest.fixture(scope="module", autouse=True)
def L():
    _build.build()
    return hb.lib()


def cache(dim=128, pages=4, heads=1):
    return torch.zeros((pages, 64, heads, dim), dtype=torch.bfloat16)


def i32(*values):
    return torch.tensor(values, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def prefill(q=None, k=None, v=None, **kw):
    return hb.prefill(bf16(9, 8, 128) if q is None else q, cache() if k is None else k, cache() if v is None else v,
                      i32(0).view(1, 1), i32(0, 9), i32(9), num_ctas=4, **kw)


def shared(q=None, k=None, v=None, batch=2, **kw):
    return hb.decode_shared_prefix(bf16(batch, 8, 128) if q is None else q, cache() if k is None else k,
                                   cache() if v is None else v, torch.zeros((batch, 1), dtype=torch.int32),
                                   torch.zeros(batch, dtype=torch.int32), i32(0).view(1, 1), i32(9), i32(0, batch), num_ctas=4,
                                   prefix_num_ctas=4, **kw)


@pytest.mark.parametrize("dim", [64, 96, 256])
def test_caches_of_another_head_dimension(dim):
    """The kernels read rows of 128 elements whatever the cache's last dimension is."""
    k = cache(dim)
    calls = [lambda: prefill(k=k, v=k), lambda: shared(k=k, v=k),
             lambda: hb.hpc_kv_write(bf16(3, 1, 128), bf16(3, 1, 128), i32(0, 1, 2), k, k),
             lambda: hb.hpc_kv_read(k, k, i32(0).view(1, 1), i32(0, 3), bf16(3, 1, 128), bf16(3, 1, 128))]
    for call in calls:
        with pytest.raises(hb.HpcError, match="heads, 128"):
            call()


def test_queries_and_outputs_of_other_dimensions():
    """[64, 128] would pass for 64 requests of 64 heads, and be read far past its end."""
    flat = bf16(64, 128)
    plan = type("Plan", (), {"buf": i32(0), "struct": hb.TilePlanStruct(0, 0, 1, 64, 8, 4, 1, 32, 1, 1)})()
    for call in (lambda: shared(q=flat, k=cache(heads=8), v=cache(heads=8), batch=64),
                 lambda: shared(q=bf16(1, 2, 1, 8, 128)),
                 lambda: prefill(q=flat), lambda: prefill(q=bf16(9, 1, 8, 128)),
                 lambda: hb.hpc_prefix_attn(flat, cache(heads=8), cache(heads=8), i32(0).view(1, 1), plan, None, None),
                 lambda: hb.hpc_prefill_attn(flat, cache(), cache(), i32(0).view(1, 1), plan, None, None, flat),
                 lambda: hb.hpc_prefix_combine(plan, None, None, None, None, None, flat),
                 lambda: hb.hpc_prefill_combine(plan, None, None, flat)):
        with pytest.raises(hb.HpcError, match="dimensions"):
            call()


def test_workspaces_with_gaps():
    """A workspace's bytes are counted from its first one on: a repeated or strided view does not have them."""
    need = hb.prefill_workspace_bytes(1, 4)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(need), torch.zeros(2 * need, dtype=torch.uint8)[::2]):
        for call in (prefill, shared):
            with pytest.raises(hb.HpcError, match="workspace"):
                call(workspace=ws)


def test_the_package_shows_the_binding_as_it_is(monkeypatch):
    """A binding function replaced later is the one that the package gives."""
    import load_balanced_paged_02_gb300 as pkg
    assert pkg.prefill is hb.prefill and pkg.hpc_kv_read is hb.hpc_kv_read
    monkeypatch.setattr(hb, "prefill", lambda: "other")
    assert pkg.prefill() == "other"
    monkeypatch.undo()
    assert pkg.prefill is hb.prefill
    with pytest.raises(AttributeError):
        pkg.no_such_name
    # and a name set on the package itself is the package's, until it is taken away
    monkeypatch.setattr(pkg, "prefill", len)
    assert pkg.prefill is len and hb.prefill is not len
    monkeypatch.delattr(pkg, "prefill")
    assert pkg.prefill is hb.prefill


@pytest.mark.parametrize("shape,dtype", [((4096,), torch.uint8), ((2, 2048), torch.uint8), ((1023,), torch.int32), ((4099,), torch.uint8)])
def test_maps_within_workspaces_of_any_shape(shape, dtype):
    ws = torch.zeros(shape, dtype=dtype)
    flat = ws.view(-1).view(torch.uint8)
    flat[256:256 + 80] = torch.arange(80, dtype=torch.uint8)
    flat[:64] = 7
    plan = hb._WorkspacePlan(hb.PlanStruct(ws.data_ptr() + 256, 80, 2, 1, 4, 2, 0, 10), ws)
    assert torch.equal(plan.buf, torch.arange(80, dtype=torch.uint8).view(torch.int32)) and plan.split_capacity == 2 + 4 - 1
    tiles = hb.TilePlan.of_workspace(hb.TilePlanStruct(ws.data_ptr(), 64, 1, 1, 1, 1, 0, 32, 1, 1), ws)
    assert tiles.words().tolist() == [0x07070707] * 16
