"""Load-balanced paged GQA decode attention for GB300 (sm_103a).

The compute path is the C-ABI library ``libhpcdecode.so`` (CUDA kernels in
``csrc/``); :mod:`.binding` marshals torch tensors into its calls. Nothing in
this package computes attention on the CPU: if the library is missing the
calls raise.

The binding is imported on first attribute access, so that
:mod:`.workloads` (the seeded input generator) can be used on its own.
"""
import importlib

_BINDING_NAMES = {
    "KV_BF16", "KV_FP8_E4M3", "HpcError", "Plan", "build", "default_num_ctas",
    "hpc_decode_attn", "hpc_decode_combine", "hpc_decode_plan", "hpc_decode_plan_static",
    "hpc_decode_read_error", "hpc_decode_step_host", "lib", "split_buffers", "decode",
    "sm_count", "hpc_rope_norm", "TilePlan", "hpc_prefill_plan", "hpc_prefill_attn", "hpc_prefill_combine",
    "prefill_split_buffers", "prefill", "hpc_prefix_plan", "hpc_prefix_attn", "hpc_prefix_combine",
    "prefix_split_buffers", "decode_shared_prefix", "hpc_tile_read_error", "tile_num_ctas", "hpc_kv_write",
    "hpc_kv_read", "prefill_workspace_bytes", "decode_shared_prefix_workspace_bytes",
}


_module = None  # the binding, once imported (looking it up costs 1 us, and some calls' kernels take two)


def __getattr__(name):
    global _module
    if name in _BINDING_NAMES:
        if _module is None:
            _module = importlib.import_module(".binding", __name__)
        return getattr(_module, name)
    raise AttributeError(name)
