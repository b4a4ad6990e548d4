"""Load-balanced paged GQA decode attention for GB300 (sm_103a).

The compute path is the C-ABI library ``libhpcdecode.so`` (CUDA kernels in
``csrc/``); :mod:`.binding` marshals torch tensors into its calls. Nothing in
this package computes attention on the CPU: if the library is missing the
calls raise.

The binding is imported on first attribute access, so that
:mod:`.workloads` (the seeded input generator) can be used on its own.
"""
import importlib
import sys
import types

_BINDING_NAMES = {
    "KV_BF16", "KV_FP8_E4M3", "HpcError", "Plan", "build", "default_num_ctas",
    "hpc_decode_attn", "hpc_decode_combine", "hpc_decode_plan", "hpc_decode_plan_static",
    "hpc_decode_read_error", "hpc_decode_step_host", "lib", "split_buffers", "decode",
    "sm_count", "hpc_rope_norm", "TilePlan", "hpc_prefill_plan", "hpc_prefill_attn", "hpc_prefill_combine",
    "prefill_split_buffers", "prefill", "hpc_prefix_plan", "hpc_prefix_attn", "hpc_prefix_combine",
    "prefix_split_buffers", "decode_shared_prefix", "hpc_tile_read_error", "tile_num_ctas", "hpc_kv_write",
    "hpc_kv_read", "prefill_workspace_bytes", "decode_shared_prefix_workspace_bytes",
}


class _Package(types.ModuleType):
    """This package: an attribute of the binding is looked up there at each access. (Descriptors of the
    module's class: a module's __getattr__ costs a microsecond, and some calls' kernels take two.)"""


class _BindingName:
    def __init__(self, name):
        self.name = name

    def __get__(self, package, cls):
        module = _BindingName.module
        if module is None:
            module = _BindingName.module = importlib.import_module(".binding", __name__)
        return getattr(module, self.name)

    module = None


for _name in _BINDING_NAMES:
    setattr(_Package, _name, _BindingName(_name))
del _name
sys.modules[__name__].__class__ = _Package
