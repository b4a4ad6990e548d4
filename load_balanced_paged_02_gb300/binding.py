"""Thin ctypes binding of libhpcdecode (include/hpc_decode.h).

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of the library. Torch tensors supply device pointers and the current
CUDA stream; nothing here computes attention, and every call raises HpcError
when the library is missing or returns a non-OK status.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from . import _build

KV_BF16 = 0
KV_FP8_E4M3 = 1
ENGINE_AUTO, ENGINE_MMA_SYNC, ENGINE_TCGEN05 = 0, 1, 2
ATTN_EARLY_KV = 1  # flags of hpc_decode_attn_ex
ATTN_TEST_WAIT_EXPIRY = 2
HEAD_DIM = 128
PAGE = 64
GROUP = 8
TILE_CTA, TILE_PAIR = 32, 64  # query tokens of a tile: one CTA's, or a pair's

_STATUS = {0: "HPC_OK", 1: "HPC_ERR_INVALID_ARG", 2: "HPC_ERR_UNSUPPORTED",
           3: "HPC_ERR_WORKSPACE_TOO_SMALL", 4: "HPC_ERR_CUDA", 5: "HPC_ERR_DEVICE_CHECK"}

# Every function include/hpc_decode.h declares: name -> (restype, argtypes).
_i = ctypes.c_int
_sz = ctypes.c_size_t
_vp = ctypes.c_void_p


class HpcError(RuntimeError):
    def __init__(self, where, status=None, detail=""):
        self.status = status
        name = _STATUS.get(status, str(status)) if status is not None else ""
        super().__init__(f"{where}: {name} {detail}".strip())


class PlanStruct(ctypes.Structure):
    _fields_ = [("buf", _vp), ("bytes", _sz), ("batch", _i), ("num_kv_heads", _i),
                ("num_ctas", _i), ("min_chunks", _i), ("mode", _i), ("max_tasks", _i)]


class TilePlanStruct(ctypes.Structure):
    _fields_ = [("buf", _vp), ("bytes", _sz), ("num_seqs", _i), ("num_tokens", _i), ("num_kv_heads", _i),
                ("num_workers", _i), ("mode", _i), ("tile_tokens", _i), ("q_len", _i), ("table_stride", _i)]


_P = ctypes.POINTER(PlanStruct)
_TP = ctypes.POINTER(TilePlanStruct)
_ll = ctypes.c_longlong
SIGNATURES = {
    "hpc_decode_plan_bytes": (_sz, [_i, _i, _i]),
    "hpc_decode_split_capacity": (_sz, [_i, _i, _i]),
    "hpc_decode_default_num_ctas": (_i, [_i]),
    "hpc_decode_suggest_num_ctas": (_i, [_vp, _i, _i, _i, _i, _i]),
    "hpc_decode_attn_multi_auto_engine": (_i, [_i, _i]),
    "hpc_decode_plan": (_i, [_vp, _i, _i, _i, _i, _P, _vp]),
    "hpc_decode_plan_static": (_i, [_vp, _i, _i, _i, _P, _vp]),
    "hpc_decode_attn": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _i, _i, _i, _i, _i, _P,
                             _vp, _vp, _vp]),
    "hpc_decode_attn_q8": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _i, _i, _i, _P,
                                _vp, _vp, _vp]),
    "hpc_decode_attn_multi": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _i, _i, _i, _i, _i,
                                   _P, _vp, _vp, _vp]),
    "hpc_decode_attn_multi_engine": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _i, _i, _i, _i,
                                          _i, _P, _vp, _vp, _i, _vp]),
    "hpc_decode_attn_ex": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _i, _i, _i, _i, _i,
                                _P, _vp, _vp, _i, _i, _vp]),
    "hpc_decode_combine": (_i, [_P, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "hpc_decode_combine_multi": (_i, [_P, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "hpc_rope_norm": (_i, [_vp, _vp, _vp, _i, _vp, _vp, ctypes.c_float, _vp, _i, _i, _i, _i, _i, _vp, _vp,
                           _vp, _vp, _vp, _vp, _i, _i, _vp, _vp]),
    "hpc_decode_step_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "hpc_decode_step_host": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                  _i, _i, _vp, _sz, _vp, _vp, _vp]),
    "hpc_decode_step_graph_create": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                                          _i, _vp, _sz, _vp, _vp, ctypes.POINTER(_vp)]),
    "hpc_decode_step_graph_launch": (_i, [_vp, _vp]),
    "hpc_decode_step_graph_destroy": (_i, [_vp]),
    "hpc_decode_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _i, _i, _i, _i, _i, _i,
                                _i, _vp, _vp, _vp]),
    "hpc_decode_read_error": (_i, [_P, ctypes.POINTER(_i)]),
    "hpc_status_string": (ctypes.c_char_p, [_i]),
    "hpc_tile_plan_bytes": (_sz, [_i, _i]),
    "hpc_tile_default_num_ctas": (_i, []),
    "hpc_prefill_split_rows": (_sz, [_i]),
    "hpc_prefix_split_rows": (_sz, [_i, _i, _i, _i, _i]),
    "hpc_prefill_plan": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _i, _TP, _vp]),
    "hpc_prefill_attn": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _i, _i, _i, _i, _TP, _vp, _vp, _vp, _vp,
                              _vp]),
    "hpc_prefill_combine": (_i, [_TP, _vp, _vp, _vp, _vp, _i, _i, _i, _vp]),
    "hpc_prefix_plan": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _TP, _vp]),
    "hpc_prefix_attn": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _i, _i, _i, _i, _TP, _vp, _vp, _vp]),
    "hpc_prefix_combine": (_i, [_TP, _vp, _vp, _P, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "hpc_prefill_workspace_bytes": (_sz, [_i, _i]),
    "hpc_prefill": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _sz,
                         _TP, _vp, _vp, _vp]),
    "hpc_decode_shared_prefix_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "hpc_decode_shared_prefix": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i,
                                      _i, _i, _i, _i, _i, _i, _i, _vp, _sz, _TP, _P, _vp, _vp, _vp]),
    "hpc_tile_read_error": (_i, [_TP, ctypes.POINTER(_i)]),
    "hpc_kv_write": (_i, [_vp, _vp, _ll, _ll, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _i, _vp, _vp]),
    "hpc_kv_read": (_i, [_vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp]),
}

_lock = threading.Lock()
_LIB = None


def build(force: bool = False) -> str:
    """Compile libhpcdecode.so for sm_103a in-tree (nvcc)."""
    return _build.build(force=force)


def lib():
    """The loaded library; raises HpcError if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    with _lock:
        if _LIB is None:
            if not os.path.exists(_build.LIB_PATH):
                raise HpcError("libhpcdecode.so", detail="is not built; call "
                               "load_balanced_paged_02_gb300.build() (needs nvcc)")
            L = ctypes.CDLL(_build.LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _LIB = L
        return _LIB


def _check(name, rc):
    if rc != 0:
        msg = lib().hpc_status_string(rc).decode()
        raise HpcError(name, rc, f"({msg})")


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda_i32(t, what):
    if not (t.is_cuda and t.dtype == torch.int32 and t.is_contiguous()):
        raise HpcError(what, detail="must be a contiguous int32 CUDA tensor")
    return t


def kv_dtype_of(cache: torch.Tensor) -> int:
    if cache.dtype == torch.bfloat16:
        return KV_BF16
    if cache.dtype in (torch.float8_e4m3fn, torch.uint8):
        return KV_FP8_E4M3
    raise HpcError("k_cache", detail=f"unsupported dtype {cache.dtype}")


def sm_count(device=None) -> int:
    return torch.cuda.get_device_properties(device or torch.cuda.current_device()).multi_processor_count


def auto_engine(kv_dtype: int, q_len: int) -> int:
    """ENGINE_MMA_SYNC or ENGINE_TCGEN05: the kernel ENGINE_AUTO runs."""
    e = lib().hpc_decode_attn_multi_auto_engine(kv_dtype, q_len)
    if e == 0:
        raise HpcError("hpc_decode_attn_multi_auto_engine", detail=f"kv_dtype {kv_dtype}, q_len {q_len}")
    return e


def default_num_ctas(kv_dtype: int = KV_BF16) -> int:
    n = lib().hpc_decode_default_num_ctas(kv_dtype)
    if n <= 0:
        raise HpcError("hpc_decode_default_num_ctas", detail="device query failed")
    return n


def suggest_num_ctas(seq_lens, num_kv_heads: int, kv_dtype: int = KV_BF16, min_chunks_per_cta: int = 2,
                     q_len: int = 1) -> int:
    """hpc_decode_suggest_num_ctas on host lengths (a CPU int32 tensor or array)."""
    import numpy as np
    sl = np.ascontiguousarray(seq_lens.cpu().numpy() if isinstance(seq_lens, torch.Tensor) else seq_lens,
                              dtype=np.int32)
    n = lib().hpc_decode_suggest_num_ctas(ctypes.c_void_p(sl.ctypes.data), int(sl.shape[0]), num_kv_heads,
                                          min_chunks_per_cta, kv_dtype, q_len)
    if n <= 0:
        raise HpcError("hpc_decode_suggest_num_ctas", detail="bad arguments or device query failed")
    return n


class Plan:
    """A task map in caller-owned device memory (``buf``) plus its host header."""

    def __init__(self, batch: int, num_kv_heads: int, num_ctas: int, device):
        nbytes = lib().hpc_decode_plan_bytes(batch, num_kv_heads, num_ctas)
        if nbytes == 0:
            raise HpcError("hpc_decode_plan_bytes", detail="sizes outside the supported limits")
        self.buf = torch.empty(nbytes // 4, dtype=torch.int32, device=device)
        self.struct = PlanStruct(self.buf.data_ptr(), nbytes, 0, 0, 0, 0, 0, 0)
        self.capacity_ctas = num_ctas
        self.split_capacity = int(lib().hpc_decode_split_capacity(batch, num_kv_heads, num_ctas))

    @property
    def num_ctas(self):
        return self.struct.num_ctas

    @property
    def mode(self):
        return self.struct.mode

    def ref(self):
        return ctypes.byref(self.struct)


def hpc_decode_plan(seq_lens: torch.Tensor, num_kv_heads: int, num_ctas: int | None = None,
                    min_chunks_per_cta: int = 2, plan: Plan | None = None, stream=None) -> Plan:
    """Load-balanced task map from device-side lengths (one launch, no host sync)."""
    _cuda_i32(seq_lens, "seq_lens")
    B = seq_lens.numel()
    if num_ctas is None:
        num_ctas = default_num_ctas(KV_BF16)
    if plan is None:
        plan = Plan(B, num_kv_heads, num_ctas, seq_lens.device)
    rc = lib().hpc_decode_plan(_ptr(seq_lens), B, num_kv_heads, num_ctas, min_chunks_per_cta,
                               plan.ref(), _stream(stream))
    _check("hpc_decode_plan", rc)
    plan.split_capacity = int(lib().hpc_decode_split_capacity(B, num_kv_heads, num_ctas))
    return plan


def hpc_decode_plan_static(seq_lens: torch.Tensor, num_kv_heads: int, num_splits: int = 16,
                           plan: Plan | None = None, stream=None) -> Plan:
    """Static split-KV task map with a fixed split count (the comparison schedule)."""
    _cuda_i32(seq_lens, "seq_lens")
    B = seq_lens.numel()
    C = num_kv_heads * B * num_splits
    if plan is None:
        plan = Plan(B, num_kv_heads, C, seq_lens.device)
    rc = lib().hpc_decode_plan_static(_ptr(seq_lens), B, num_kv_heads, num_splits, plan.ref(),
                                      _stream(stream))
    _check("hpc_decode_plan_static", rc)
    plan.split_capacity = int(lib().hpc_decode_split_capacity(B, num_kv_heads, C))
    return plan


def split_buffers(plan: Plan, device=None, q_len: int = 1):
    """Allocate split_o [capacity, 8, 128] and split_lse [capacity, 8] (float32);
    with q_len > 1, [capacity, q_len, 8, 128] and [capacity, q_len, 8]."""
    device = device or plan.buf.device
    cap = plan.split_capacity
    rows = (cap, GROUP) if q_len == 1 else (cap, q_len, GROUP)
    return (torch.empty(rows + (HEAD_DIM,), dtype=torch.float32, device=device),
            torch.empty(rows, dtype=torch.float32, device=device))


def hpc_decode_attn(q, k_cache, v_cache, page_table, seq_lens, plan: Plan, split_o, split_lse,
                    k_scale=None, v_scale=None, num_pages: int | None = None, stream=None,
                    q_scale=None, engine: int | None = None, early_kv: bool = False):
    """Persistent attention over the task map; writes split_o / split_lse.
    A float8_e4m3fn q with its q_scale [B, Hq] goes to hpc_decode_attn_q8; a
    bf16 q of shape [B, q_len, Hq, 128] (several new tokens per request, causal)
    goes to hpc_decode_attn_multi. A given ``engine`` (ENGINE_AUTO, ENGINE_MMA_SYNC
    or ENGINE_TCGEN05) goes to hpc_decode_attn_multi_engine for a bf16 q of any
    q_len (hpc_decode_attn_ex for an e4m3 q). ``early_kv`` goes
    to hpc_decode_attn_ex with HPC_ATTN_EARLY_KV: the kernel gathers the KV of
    chunks without a new token before it waits for the previous kernel (the
    caller's contract is in the header)."""
    kvd = kv_dtype_of(k_cache)
    q_len = q.shape[1] if q.dim() == 4 else 1
    B, Hq, D = q.shape[0], q.shape[-2], q.shape[-1]
    Hkv = k_cache.shape[2]
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (split_o, "split_o"),
                 (split_lse, "split_lse")):
        if not (t.is_cuda and t.is_contiguous()):
            raise HpcError(n, detail="must be a contiguous CUDA tensor")
    _cuda_i32(page_table, "page_table")
    _cuda_i32(seq_lens, "seq_lens")
    need = plan.split_capacity * q_len * GROUP
    if split_o.numel() < need * HEAD_DIM or split_lse.numel() < need:
        raise HpcError("split buffers", detail=f"need {plan.split_capacity} x {q_len} x 8 rows")
    npages = int(num_pages if num_pages is not None else k_cache.shape[0])
    q8 = q.dtype in (torch.float8_e4m3fn, torch.uint8)
    if q8 and q_scale is None:
        raise HpcError("hpc_decode_attn_q8", detail="an e4m3 q needs q_scale")
    if early_kv or (q8 and engine is not None):
        rc = lib().hpc_decode_attn_ex(
            _ptr(q), _ptr(q_scale), q_len, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), kvd,
            npages, _ptr(page_table), int(page_table.shape[1]), _ptr(seq_lens), B, Hq, Hkv, D,
            int(k_cache.shape[1]), plan.ref(), _ptr(split_o), _ptr(split_lse),
            ENGINE_AUTO if engine is None else int(engine), ATTN_EARLY_KV if early_kv else 0, _stream(stream))
        _check("hpc_decode_attn_ex", rc)
        return
    if q8:
        rc = lib().hpc_decode_attn_q8(
            _ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), npages,
            _ptr(page_table), int(page_table.shape[1]), _ptr(seq_lens), B, Hq, Hkv, D,
            int(k_cache.shape[1]), plan.ref(), _ptr(split_o), _ptr(split_lse), _stream(stream))
        _check("hpc_decode_attn_q8", rc)
        return
    if engine is not None:  # also for one new token ([B, Hq, 128] is [B, 1, Hq, 128])
        rc = lib().hpc_decode_attn_multi_engine(
            _ptr(q), q_len, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), kvd, npages,
            _ptr(page_table), int(page_table.shape[1]), _ptr(seq_lens), B, Hq, Hkv, D, int(k_cache.shape[1]),
            plan.ref(), _ptr(split_o), _ptr(split_lse), int(engine), _stream(stream))
        _check("hpc_decode_attn_multi_engine", rc)
        return
    if q.dim() == 4:
        rc = lib().hpc_decode_attn_multi(
            _ptr(q), q_len, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), kvd, npages,
            _ptr(page_table), int(page_table.shape[1]), _ptr(seq_lens), B, Hq, Hkv, D, int(k_cache.shape[1]),
            plan.ref(), _ptr(split_o), _ptr(split_lse), _stream(stream))
        _check("hpc_decode_attn_multi", rc)
        return
    rc = lib().hpc_decode_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), kvd, npages, _ptr(page_table),
        int(page_table.shape[1]), _ptr(seq_lens), B, Hq, Hkv, D, int(k_cache.shape[1]), plan.ref(),
        _ptr(split_o), _ptr(split_lse), _stream(stream))
    _check("hpc_decode_attn", rc)


def hpc_decode_combine(plan: Plan, split_o, split_lse, out, out_lse=None, num_kv_heads=None,
                       stream=None):
    """LSE-weighted merge of the partials into out (bf16) and out_lse (float32).
    A 4-D out [B, q_len, Hq, 128] merges the partials of hpc_decode_attn_multi."""
    B, Hq, D = out.shape[0], out.shape[-2], out.shape[-1]
    Hkv = num_kv_heads if num_kv_heads is not None else Hq // GROUP
    if out.dim() == 4:
        rc = lib().hpc_decode_combine_multi(plan.ref(), int(out.shape[1]), _ptr(split_o), _ptr(split_lse),
                                            _ptr(out), _ptr(out_lse), B, Hq, Hkv, D, _stream(stream))
        _check("hpc_decode_combine_multi", rc)
        return
    rc = lib().hpc_decode_combine(plan.ref(), _ptr(split_o), _ptr(split_lse), _ptr(out),
                                  _ptr(out_lse), B, Hq, Hkv, D, _stream(stream))
    _check("hpc_decode_combine", rc)


def decode(q, k_cache, v_cache, page_table, seq_lens, k_scale=None, v_scale=None,
           num_ctas: int | None = None, min_chunks_per_cta: int = 2, static_splits: int | None = None,
           stream=None, q_scale=None):
    """plan -> attn -> combine with freshly allocated buffers. Returns (out, lse, plan)."""
    Hkv = k_cache.shape[2]
    if static_splits:
        plan = hpc_decode_plan_static(seq_lens, Hkv, static_splits, stream=stream)
    else:
        if num_ctas is None:
            num_ctas = default_num_ctas(kv_dtype_of(k_cache))
        plan = hpc_decode_plan(seq_lens, Hkv, num_ctas, min_chunks_per_cta, stream=stream)
    so, sl = split_buffers(plan, q_len=q.shape[1] if q.dim() == 4 else 1)
    hpc_decode_attn(q, k_cache, v_cache, page_table, seq_lens, plan, so, sl, k_scale, v_scale,
                    stream=stream, q_scale=q_scale)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    hpc_decode_combine(plan, so, sl, out, lse, Hkv, stream=stream)
    return out, lse, plan


def hpc_decode_read_error(plan: Plan) -> int:
    """Synchronise and read the task map's device error word (HPC_DEVERR_* bits)."""
    w = ctypes.c_int(0)
    rc = lib().hpc_decode_read_error(plan.ref(), ctypes.byref(w))
    if rc not in (0, 5):
        _check("hpc_decode_read_error", rc)
    return int(w.value)


def step_workspace_bytes(batch, num_q_heads, num_kv_heads, page_table_stride, num_ctas) -> int:
    return int(lib().hpc_decode_step_workspace_bytes(batch, num_q_heads, num_kv_heads,
                                                      page_table_stride, num_ctas))


def hpc_decode_step_host(h_q, h_seq_lens, h_page_table, k_cache, v_cache, workspace, h_out,
                         h_out_lse=None, k_scale=None, v_scale=None, num_ctas=None,
                         min_chunks_per_cta: int = 2, num_pages=None, stream=None):
    """One step from host tensors (pinned CPU): H2D copies, plan, attn, combine, D2H.
    Asynchronous on ``stream``; synchronise before reading h_out."""
    B, Hq, D = h_q.shape
    Hkv = k_cache.shape[2]
    if num_ctas is None:
        num_ctas = default_num_ctas(kv_dtype_of(k_cache))
    rc = lib().hpc_decode_step_host(
        _ptr(h_q), _ptr(h_seq_lens), _ptr(h_page_table), int(h_page_table.shape[1]),
        _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), kv_dtype_of(k_cache),
        int(num_pages if num_pages is not None else k_cache.shape[0]), B, Hq, Hkv, D,
        int(k_cache.shape[1]), num_ctas, min_chunks_per_cta, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(h_out), _ptr(h_out_lse), _stream(stream))
    _check("hpc_decode_step_host", rc)


class StepGraph:
    """hpc_decode_step_host captured once as a CUDA graph (hpc_decode_step_graph_*).
    The tensors given here are fixed: refill the pinned host inputs in place,
    call launch(), synchronise the stream, then read h_out / h_out_lse."""

    def __init__(self, h_q, h_seq_lens, h_page_table, k_cache, v_cache, workspace, h_out, h_out_lse=None,
                 k_scale=None, v_scale=None, num_ctas=None, min_chunks_per_cta: int = 2, num_pages=None):
        B, Hq, D = h_q.shape
        Hkv = k_cache.shape[2]
        if num_ctas is None:
            num_ctas = default_num_ctas(kv_dtype_of(k_cache))
        # keep every tensor the graph points into alive as long as the graph
        self._keep = (h_q, h_seq_lens, h_page_table, k_cache, v_cache, workspace, h_out, h_out_lse, k_scale,
                      v_scale)
        handle = _vp()
        rc = lib().hpc_decode_step_graph_create(
            _ptr(h_q), _ptr(h_seq_lens), _ptr(h_page_table), int(h_page_table.shape[1]),
            _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), kv_dtype_of(k_cache),
            int(num_pages if num_pages is not None else k_cache.shape[0]), B, Hq, Hkv, D,
            int(k_cache.shape[1]), num_ctas, min_chunks_per_cta, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(h_out), _ptr(h_out_lse), ctypes.byref(handle))
        _check("hpc_decode_step_graph_create", rc)
        self._handle = handle

    def launch(self, stream=None):
        if not self._handle:
            raise HpcError("hpc_decode_step_graph_launch", detail="the graph was closed")
        _check("hpc_decode_step_graph_launch", lib().hpc_decode_step_graph_launch(self._handle, _stream(stream)))

    def close(self):
        if self._handle:
            rc = lib().hpc_decode_step_graph_destroy(self._handle)
            self._handle = _vp()
            _check("hpc_decode_step_graph_destroy", rc)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def hpc_rope_norm(qkv, positions, cos_sin, q_weight, k_weight, slot_mapping, q_out, k_cache, v_cache,
                  q_scale=None, k_scale=None, v_scale=None, eps: float = 1e-6, num_kv_heads=None,
                  num_pages=None, error_word=None, stream=None):
    """Fused prologue: QK-norm + rotary embedding on Q and K, K/V into the cache
    slots, Q to q_out (bf16, or e4m3 codes with q_scale [T, Hq])."""
    T, H3, D = qkv.shape
    Hkv = num_kv_heads if num_kv_heads is not None else k_cache.shape[2]
    Hq = H3 - 2 * Hkv
    rc = lib().hpc_rope_norm(
        _ptr(qkv), _ptr(positions), _ptr(cos_sin), int(cos_sin.shape[0]), _ptr(q_weight), _ptr(k_weight),
        float(eps), _ptr(slot_mapping), T, Hq, Hkv, D, int(k_cache.shape[1]), _ptr(q_out), _ptr(q_scale),
        _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), kv_dtype_of(k_cache),
        int(num_pages if num_pages is not None else k_cache.shape[0]), _ptr(error_word), _stream(stream))
    _check("hpc_rope_norm", rc)


# ---------------------------------------------------------------- prompts, shared prefixes, cache write / read
#
# A decode step's calls take microseconds on the device, so these bindings keep
# their own cost down: integers for pointers, one pass of checks, and the
# one-call forms with a workspace.

def _addr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, device_index):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device_index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _on_device(what, *tensors):
    """The device index that all tensors (None passed over) share, which must be the current one."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise HpcError(what, detail=f"tensors on {tensors[0].device} and {t.device}")
    if index < 0:
        raise HpcError(what, detail="tensors must be on a CUDA device")
    current = torch._C._cuda_getDevice()
    if index != current:
        raise HpcError(what, detail=f"tensors on cuda:{index}, but the current device is cuda:{current}")
    return index


def _i32(what, t, numel=None):
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise HpcError(what, detail="must be a contiguous int32 tensor")
    if numel is not None and t.numel() != numel:
        raise HpcError(what, detail=f"must hold {numel} values")


def _table(what, t, rows):
    _i32(what, t)
    if t.dim() != 2 or t.shape[0] != rows:
        raise HpcError(what, detail=f"must have {rows} rows")


def _tensor(what, t, shape, dtype):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise HpcError(what, detail=f"must be a contiguous {dtype} tensor of shape {tuple(shape)}")


def _query(what, q, new_tokens=False):
    """A packed query [tokens, heads, 128], or with new_tokens one of a decode step: [B, heads, 128] or
    [B, q_len, heads, 128]."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise HpcError(what, detail="q must be a contiguous bfloat16 tensor")
    if not (q.dim() == 3 or new_tokens and q.dim() == 4):
        raise HpcError(what, detail="q must have 3 or 4 dimensions" if new_tokens else "q must have 3 dimensions")


def _workspace(what, t):
    if t is not None and not t.is_contiguous():
        raise HpcError(what, detail="workspace must be a contiguous tensor")


def _caches(what, k_cache, v_cache, k_scale, v_scale, num_pages):
    """Checks of a paged cache; returns its hpc_kv_dtype, pages in use, page size and KV heads."""
    kvd = kv_dtype_of(k_cache)
    shape = k_cache.shape
    if len(shape) != 4 or shape[3] != HEAD_DIM or v_cache.shape != shape or v_cache.dtype != k_cache.dtype:
        raise HpcError(what, detail="k_cache and v_cache must be [pages, 64, heads, 128] of one type")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise HpcError(what, detail="k_cache and v_cache must be contiguous")
    pages, page, heads, _ = shape
    if kvd == KV_FP8_E4M3:
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is None:
                raise HpcError(n, detail="an e4m3 cache needs scales")
            _tensor(n, t, (pages, heads, page), torch.float32)
    if num_pages is not None:
        if num_pages > pages:
            raise HpcError("num_pages", detail=f"{num_pages}, but the cache has {pages}")
        pages = num_pages
    return kvd, pages, page, heads


class TilePlan:
    """A tile map in device memory (``buf``, int32) plus its host header."""

    def __init__(self, num_seqs: int, num_ctas: int, device):
        nbytes = lib().hpc_tile_plan_bytes(num_seqs, num_ctas)
        if nbytes == 0:
            raise HpcError("hpc_tile_plan_bytes", detail="sizes outside the supported limits")
        self.buf = torch.empty(nbytes // 4, dtype=torch.int32, device=device)
        self.struct = TilePlanStruct(self.buf.data_ptr(), nbytes, 0, 0, 0, 0, 0, 0, 0, 0)

    @classmethod
    def of_workspace(cls, struct, workspace):
        """The map that a one-call form left at the start of its workspace."""
        plan = cls.__new__(cls)
        plan.buf = workspace
        plan.struct = struct
        return plan

    @property
    def num_ctas(self):
        """CTAs of the attention call."""
        return self.struct.num_workers * (self.struct.tile_tokens // TILE_CTA)

    @property
    def tile_tokens(self):
        return self.struct.tile_tokens

    def words(self):
        """The map as an int32 tensor."""
        return self.buf.view(-1).view(torch.uint8)[:self.struct.bytes].view(torch.int32)

    def ref(self):
        return ctypes.byref(self.struct)


_CTAS = {}  # what each device answered


def tile_num_ctas() -> int:
    """hpc_tile_default_num_ctas: one CTA per SM of the current device."""
    key = ("tile", torch.cuda.current_device())
    if key not in _CTAS:
        n = lib().hpc_tile_default_num_ctas()
        if n <= 0:
            raise HpcError("hpc_tile_default_num_ctas", detail="device query failed")
        _CTAS[key] = n
    return _CTAS[key]


def _decode_num_ctas(kvd):
    key = (kvd, torch.cuda.current_device())
    if key not in _CTAS:
        _CTAS[key] = default_num_ctas(kvd)
    return _CTAS[key]


_HERE = contextlib.nullcontext()


def _on(stream):
    """Allocations for work on ``stream`` belong to it."""
    if stream is None:
        return _HERE
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


def _split_rows(rows, device):
    return (torch.empty((rows, HEAD_DIM), dtype=torch.float32, device=device),
            torch.empty(rows, dtype=torch.float32, device=device))


def _check_splits(what, rows, split_o, split_lse):
    for t, n in ((split_o, rows * HEAD_DIM), (split_lse, rows)):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() < n:
            raise HpcError(what, detail=f"split buffers need {rows} rows of contiguous float32")


def hpc_prefill_plan(q_starts, seq_lens, num_tokens: int, num_kv_heads: int, page_table_stride: int,
                     num_ctas: int | None = None, min_blocks_per_cta: int = 1, tile_tokens: int = 0,
                     plan: TilePlan | None = None, stream=None) -> TilePlan:
    """Tile map of packed prompts from device-side starts and lengths (one launch, no host sync)."""
    _i32("seq_lens", seq_lens)
    B = seq_lens.numel()
    _i32("q_starts", q_starts, B + 1)
    dev = _on_device("hpc_prefill_plan", seq_lens, q_starts, None if plan is None else plan.buf)
    num_ctas = tile_num_ctas() if num_ctas is None else num_ctas
    if plan is None:
        with _on(stream):
            plan = TilePlan(B, num_ctas, seq_lens.device)
    rc = lib().hpc_prefill_plan(q_starts.data_ptr(), seq_lens.data_ptr(), B, num_tokens, num_kv_heads, page_table_stride,
                                num_ctas, min_blocks_per_cta, tile_tokens, plan.ref(), _raw_stream(stream, dev))
    _check("hpc_prefill_plan", rc)
    return plan


def prefill_split_buffers(plan: TilePlan):
    """split_o and split_lse of hpc_prefill_attn for this map."""
    return _split_rows(int(lib().hpc_prefill_split_rows(plan.num_ctas)), plan.buf.device)


def hpc_prefill_attn(q, k_cache, v_cache, page_table, plan: TilePlan, split_o, split_lse, out, out_lse=None, k_scale=None,
                     v_scale=None, num_pages: int | None = None, stream=None):
    """Causal attention of packed prompts over the paged cache; whole tiles go to
    out [T, Hq, 128] (and out_lse [T, Hq]), pieces of cut ones to the split buffers."""
    what = "hpc_prefill_attn"
    kvd, pages, page, Hkv = _caches(what, k_cache, v_cache, k_scale, v_scale, num_pages)
    _query(what, q)
    T, Hq, D = q.shape
    _table("page_table", page_table, plan.struct.num_seqs)
    dev = _on_device(what, q, k_cache, v_cache, k_scale, v_scale, page_table, split_o, split_lse, out, out_lse,
                     plan.buf)
    if T != plan.struct.num_tokens:
        raise HpcError(what, detail=f"q has {T} tokens, the plan {plan.struct.num_tokens}")
    _tensor("out", out, (T, Hq, D), torch.bfloat16)
    if out_lse is not None:
        _tensor("out_lse", out_lse, (T, Hq), torch.float32)
    _check_splits(what, int(lib().hpc_prefill_split_rows(plan.num_ctas)), split_o, split_lse)
    rc = lib().hpc_prefill_attn(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale), kvd, pages,
        page_table.data_ptr(), page_table.shape[1], Hq, Hkv, D, page, plan.ref(), split_o.data_ptr(), split_lse.data_ptr(),
        out.data_ptr(), _addr(out_lse), _raw_stream(stream, dev))
    _check(what, rc)


def hpc_prefill_combine(plan: TilePlan, split_o, split_lse, out, out_lse=None, stream=None):
    """Merges the pieces of cut tiles into out and out_lse."""
    what = "hpc_prefill_combine"
    if out.dim() != 3:
        raise HpcError(what, detail="out must have 3 dimensions")
    T, Hq, D = out.shape
    dev = _on_device(what, out, split_o, split_lse, out_lse, plan.buf)
    _tensor("out", out, (plan.struct.num_tokens, Hq, D), torch.bfloat16)
    if out_lse is not None:
        _tensor("out_lse", out_lse, (T, Hq), torch.float32)
    _check_splits(what, int(lib().hpc_prefill_split_rows(plan.num_ctas)), split_o, split_lse)
    rc = lib().hpc_prefill_combine(plan.ref(), split_o.data_ptr(), split_lse.data_ptr(), out.data_ptr(), _addr(out_lse), Hq,
                                   plan.struct.num_kv_heads, D, _raw_stream(stream, dev))
    _check(what, rc)


def prefill(q, k_cache, v_cache, page_table, q_starts, seq_lens, k_scale=None, v_scale=None, num_ctas: int | None = None,
            min_blocks_per_cta: int = 1, tile_tokens: int = 0, num_pages: int | None = None, out=None, out_lse=None,
            workspace=None, stream=None):
    """Causal attention of packed prompts, q bf16 [T, Hq, 128], over the paged cache: plan,
    attention and combine in one call (hpc_prefill). Buffers that are not given are allocated
    here; a given ``workspace`` is a uint8 tensor of prefill_workspace_bytes. Returns (out,
    lse, plan)."""
    what = "hpc_prefill"
    kvd, pages, page, Hkv = _caches(what, k_cache, v_cache, k_scale, v_scale, num_pages)
    _query(what, q)
    T, Hq, D = q.shape
    _i32("seq_lens", seq_lens)
    B = seq_lens.numel()
    _i32("q_starts", q_starts, B + 1)
    _table("page_table", page_table, B)
    _workspace(what, workspace)
    dev = _on_device(what, q, k_cache, v_cache, k_scale, v_scale, page_table, q_starts, seq_lens, out, out_lse, workspace)
    num_ctas = tile_num_ctas() if num_ctas is None else num_ctas
    L = lib()
    if out is not None:
        _tensor("out", out, q.shape, torch.bfloat16)
    if out_lse is not None:
        _tensor("out_lse", out_lse, (T, Hq), torch.float32)
    if workspace is None or out is None or out_lse is None:
        with _on(stream):
            if workspace is None:
                workspace = torch.empty(L.hpc_prefill_workspace_bytes(B, num_ctas), dtype=torch.uint8, device=q.device)
            if out is None:
                out = torch.empty_like(q)
            if out_lse is None:
                out_lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    plan = TilePlan.of_workspace(TilePlanStruct(), workspace)
    rc = L.hpc_prefill(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale), kvd, pages,
        page_table.data_ptr(), page_table.shape[1], q_starts.data_ptr(), seq_lens.data_ptr(), B, T, Hq, Hkv, D, page,
        num_ctas, min_blocks_per_cta, tile_tokens, workspace.data_ptr(), workspace.nbytes, plan.ref(), out.data_ptr(),
        out_lse.data_ptr(), _raw_stream(stream, dev))
    _check(what, rc)
    return out, out_lse, plan


def prefill_workspace_bytes(batch: int, num_ctas: int | None = None) -> int:
    """Bytes of the workspace that prefill takes for this many sequences."""
    return int(lib().hpc_prefill_workspace_bytes(batch, tile_num_ctas() if num_ctas is None else num_ctas))


def hpc_prefix_plan(group_starts, prefix_lens, batch: int, num_kv_heads: int, prefix_table_stride: int, q_len: int = 1,
                    num_ctas: int | None = None, min_blocks_per_cta: int = 1, tile_tokens: int = 0,
                    plan: TilePlan | None = None, stream=None) -> TilePlan:
    """Tile map of the prefixes that groups of a decode batch share."""
    _i32("prefix_lens", prefix_lens)
    G = prefix_lens.numel()
    _i32("group_starts", group_starts, G + 1)
    dev = _on_device("hpc_prefix_plan", prefix_lens, group_starts, None if plan is None else plan.buf)
    num_ctas = tile_num_ctas() if num_ctas is None else num_ctas
    if plan is None:
        with _on(stream):
            plan = TilePlan(G, num_ctas, prefix_lens.device)
    rc = lib().hpc_prefix_plan(group_starts.data_ptr(), prefix_lens.data_ptr(), G, batch, q_len, num_kv_heads,
                               prefix_table_stride, num_ctas, min_blocks_per_cta, tile_tokens, plan.ref(),
                               _raw_stream(stream, dev))
    _check("hpc_prefix_plan", rc)
    return plan


def _prefix_rows(plan: TilePlan):
    p = plan.struct
    return int(lib().hpc_prefix_split_rows(p.num_seqs, p.num_tokens // p.q_len, p.q_len, p.num_kv_heads, plan.num_ctas))


def prefix_split_buffers(plan: TilePlan):
    """split_o and split_lse of hpc_prefix_attn for this map."""
    return _split_rows(_prefix_rows(plan), plan.buf.device)


def hpc_prefix_attn(q, k_cache, v_cache, prefix_table, plan: TilePlan, split_o, split_lse, k_scale=None, v_scale=None,
                    num_pages: int | None = None, stream=None):
    """Attention of every query row of a decode batch (q bf16 [B, Hq, 128] or
    [B, q_len, Hq, 128]) over its group's prefix; partial rows for hpc_prefix_combine."""
    what = "hpc_prefix_attn"
    kvd, pages, page, Hkv = _caches(what, k_cache, v_cache, k_scale, v_scale, num_pages)
    _query(what, q, new_tokens=True)
    Hq, D = q.shape[-2:]
    _table("prefix_table", prefix_table, plan.struct.num_seqs)
    dev = _on_device(what, q, k_cache, v_cache, k_scale, v_scale, prefix_table, split_o, split_lse, plan.buf)
    if q.numel() != plan.struct.num_tokens * Hq * D or (q.shape[1] if q.dim() == 4 else 1) != plan.struct.q_len:
        raise HpcError(what, detail="q and the plan differ in requests or new tokens")
    _check_splits(what, _prefix_rows(plan), split_o, split_lse)
    rc = lib().hpc_prefix_attn(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale), kvd, pages,
        prefix_table.data_ptr(), prefix_table.shape[1], Hq, Hkv, D, page, plan.ref(), split_o.data_ptr(),
        split_lse.data_ptr(), _raw_stream(stream, dev))
    _check(what, rc)


def hpc_prefix_combine(prefix_plan: TilePlan, prefix_o, prefix_lse, plan: Plan, split_o, split_lse, out, out_lse=None,
                       stream=None):
    """Merges the prefix pieces and the splits of the requests' own tokens into out
    ([B, Hq, 128] or [B, q_len, Hq, 128] bf16) and out_lse."""
    what = "hpc_prefix_combine"
    if out.dim() not in (3, 4):
        raise HpcError(what, detail="out must have 3 or 4 dimensions")
    B, Hq, D = out.shape[0], out.shape[-2], out.shape[-1]
    q_len = out.shape[1] if out.dim() == 4 else 1
    dev = _on_device(what, out, prefix_o, prefix_lse, split_o, split_lse, out_lse, prefix_plan.buf, plan.buf)
    _tensor("out", out, out.shape, torch.bfloat16)
    if out_lse is not None:
        _tensor("out_lse", out_lse, out.shape[:-1], torch.float32)
    _check_splits(what, _prefix_rows(prefix_plan), prefix_o, prefix_lse)
    _check_splits(what, plan.split_capacity * q_len * GROUP, split_o, split_lse)
    rc = lib().hpc_prefix_combine(prefix_plan.ref(), prefix_o.data_ptr(), prefix_lse.data_ptr(), plan.ref(),
                                  split_o.data_ptr(), split_lse.data_ptr(), out.data_ptr(), _addr(out_lse), B, q_len, Hq,
                                  Hq // GROUP, D, _raw_stream(stream, dev))
    _check(what, rc)


class _WorkspacePlan(Plan):
    """The task map that decode_shared_prefix left in its workspace, for the decode calls that take one."""

    def __init__(self, struct, workspace):
        self.struct = struct
        self.workspace = workspace

    @property
    def buf(self):
        at = self.struct.buf - self.workspace.data_ptr()
        return self.workspace.view(-1).view(torch.uint8)[at:at + self.struct.bytes].view(torch.int32)

    @property
    def split_capacity(self):
        p = self.struct
        return int(lib().hpc_decode_split_capacity(p.batch, p.num_kv_heads, p.num_ctas))

    @property
    def capacity_ctas(self):
        return self.struct.num_ctas


def decode_shared_prefix(q, k_cache, v_cache, page_table, seq_lens, prefix_table, prefix_lens, group_starts, k_scale=None,
                         v_scale=None, num_ctas: int | None = None, min_chunks_per_cta: int = 2,
                         prefix_num_ctas: int | None = None, min_blocks_per_cta: int = 1, tile_tokens: int = 0,
                         num_pages: int | None = None, workspace=None, stream=None, out=None, out_lse=None):
    """One decode step of a batch whose groups share prefixes: requests
    [group_starts[g], group_starts[g + 1]) see the prefix_lens[g] tokens that
    prefix_table[g] names, then their own seq_lens[b] tokens (page_table). Each
    prefix is computed once for its group. q bf16 [B, Hq, 128] or [B, q_len, Hq, 128]. Buffers
    that are not given are allocated here; a given ``workspace`` is a uint8 tensor of
    decode_shared_prefix_workspace_bytes. Returns (out, lse, prefix_plan, plan)."""
    what = "hpc_decode_shared_prefix"
    kvd, pages, page, Hkv = _caches(what, k_cache, v_cache, k_scale, v_scale, num_pages)
    _query(what, q, new_tokens=True)
    B, Hq, D = q.shape[0], q.shape[-2], q.shape[-1]
    q_len = q.shape[1] if q.dim() == 4 else 1
    _i32("seq_lens", seq_lens, B)
    _table("page_table", page_table, B)
    _i32("prefix_lens", prefix_lens)
    G = prefix_lens.numel()
    _i32("group_starts", group_starts, G + 1)
    _table("prefix_table", prefix_table, G)
    _workspace(what, workspace)
    if out is not None:
        _tensor("out", out, q.shape, torch.bfloat16)
    if out_lse is not None:
        _tensor("out_lse", out_lse, q.shape[:-1], torch.float32)
    dev = _on_device(what, q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, prefix_table, prefix_lens,
                     group_starts, workspace, out, out_lse)
    num_ctas = _decode_num_ctas(kvd) if num_ctas is None else num_ctas
    prefix_num_ctas = tile_num_ctas() if prefix_num_ctas is None else prefix_num_ctas
    L = lib()
    if workspace is None or out is None or out_lse is None:
        with _on(stream):
            if workspace is None:
                need = L.hpc_decode_shared_prefix_workspace_bytes(G, B, q_len, Hkv, prefix_num_ctas, num_ctas)
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            if out is None:
                out = torch.empty_like(q)
            if out_lse is None:
                out_lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    pplan, plan = TilePlan.of_workspace(TilePlanStruct(), workspace), _WorkspacePlan(PlanStruct(), workspace)
    rc = L.hpc_decode_shared_prefix(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale), kvd, pages,
        page_table.data_ptr(), page_table.shape[1], seq_lens.data_ptr(), prefix_table.data_ptr(), prefix_table.shape[1],
        prefix_lens.data_ptr(), group_starts.data_ptr(), G, B, q_len, Hq, Hkv, D, page, num_ctas, min_chunks_per_cta,
        prefix_num_ctas, min_blocks_per_cta, tile_tokens, workspace.data_ptr(), workspace.nbytes, pplan.ref(), plan.ref(),
        out.data_ptr(), out_lse.data_ptr(), _raw_stream(stream, dev))
    _check(what, rc)
    return out, out_lse, pplan, plan


def decode_shared_prefix_workspace_bytes(num_groups: int, batch: int, num_kv_heads: int, q_len: int = 1,
                                         kv_dtype: int = KV_BF16, prefix_num_ctas: int | None = None,
                                         num_ctas: int | None = None) -> int:
    """Bytes of the workspace that decode_shared_prefix takes."""
    return int(lib().hpc_decode_shared_prefix_workspace_bytes(
        num_groups, batch, q_len, num_kv_heads, tile_num_ctas() if prefix_num_ctas is None else prefix_num_ctas,
        _decode_num_ctas(kv_dtype) if num_ctas is None else num_ctas))


def hpc_tile_read_error(plan: TilePlan) -> int:
    """Synchronise and read the tile map's device error word (HPC_DEVERR_* bits)."""
    w = ctypes.c_int(0)
    rc = lib().hpc_tile_read_error(plan.ref(), ctypes.byref(w))
    if rc not in (0, 5):
        _check("hpc_tile_read_error", rc)
    return int(w.value)


def hpc_kv_write(k, v, slot_mapping, k_cache, v_cache, k_scale=None, v_scale=None, num_pages: int | None = None,
                 error_word=None, stream=None):
    """K and V (bf16 [T, Hkv, 128]; any token stride, such as slices of a fused
    projection's output) into the cache slots, bf16 or quantised to e4m3."""
    what = "hpc_kv_write"
    kvd, pages, page, Hkv = _caches(what, k_cache, v_cache, k_scale, v_scale, num_pages)
    shape = k.shape
    if len(shape) != 3 or v.shape != shape or shape[1] != Hkv or shape[2] != HEAD_DIM:
        raise HpcError(what, detail=f"k and v must be [tokens, {Hkv}, {HEAD_DIM}]")
    T = shape[0]
    _i32("slot_mapping", slot_mapping, T)
    dev = _on_device(what, k_cache, v_cache, k_scale, v_scale, k, v, slot_mapping, error_word)
    strides = []
    for t, n in ((k, "k"), (v, "v")):
        st = t.stride()
        if t.dtype != torch.bfloat16 or (T > 0 and (st[2] != 1 or (Hkv > 1 and st[1] != HEAD_DIM))):
            raise HpcError(n, detail="must be bfloat16 with each token's heads contiguous")
        strides.append(st[0] if T > 1 else Hkv * HEAD_DIM)
    if error_word is not None:
        _i32("error_word", error_word)
    rc = lib().hpc_kv_write(k.data_ptr(), v.data_ptr(), strides[0], strides[1], slot_mapping.data_ptr(), T, Hkv, HEAD_DIM,
                            page, k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale), kvd, pages,
                            _addr(error_word), _raw_stream(stream, dev))
    _check(what, rc)


def hpc_kv_read(k_cache, v_cache, page_table, out_starts, k_out, v_out, k_scale=None, v_scale=None, first=None,
                num_pages: int | None = None, error_word=None, stream=None):
    """Tokens first[b], first[b] + 1, ... of each request into rows
    [out_starts[b], out_starts[b + 1]) of k_out and v_out (bf16 [rows, Hkv, 128])."""
    what = "hpc_kv_read"
    kvd, pages, page, Hkv = _caches(what, k_cache, v_cache, k_scale, v_scale, num_pages)
    _i32("page_table", page_table)
    if page_table.dim() != 2:
        raise HpcError("page_table", detail="must be [batch, pages]")
    B, width = page_table.shape
    _i32("out_starts", out_starts, B + 1)
    if first is not None:
        _i32("first", first, B)
    rows = k_out.shape[0]
    _tensor("k_out", k_out, (rows, Hkv, HEAD_DIM), torch.bfloat16)
    _tensor("v_out", v_out, (rows, Hkv, HEAD_DIM), torch.bfloat16)
    if error_word is not None:
        _i32("error_word", error_word)
    dev = _on_device(what, k_cache, v_cache, k_scale, v_scale, page_table, out_starts, first, k_out, v_out, error_word)
    rc = lib().hpc_kv_read(k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale), kvd, pages,
                           page_table.data_ptr(), width, _addr(first), out_starts.data_ptr(), B, rows, Hkv, HEAD_DIM, page,
                           k_out.data_ptr(), v_out.data_ptr(), _addr(error_word), _raw_stream(stream, dev))
    _check(what, rc)
