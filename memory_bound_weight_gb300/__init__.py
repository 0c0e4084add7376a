"""GB300 (sm_103a) weight-streaming GEMV library: y = W.x and Y = X.W^T with
BF16, INT4 group-64, AWQ-style INT4 group-128 and symmetric per-channel INT8
weights; products of any number of rows in 8-bit floating point with a scale
for each block of 128; and, around these products in a decode step, a 4-bit
paged key/value cache with its attention, also behind a prefix that requests
share, and the log probabilities of tokens.

The compute path is libmbw.so (C ABI in include/mbw.h); this package is its
binding. Submodules ``inputs`` and ``workloads`` (synthetic data and byte
accounting) import without loading the CUDA library.
"""
_EXPORTS = frozenset((
    "gemv_bf16", "gemv_int4_g64", "gemv_int4_awq_g128", "gemm_skinny_bf16", "gemv_int8_pc", "quantize_int8_pc",
    "gemv_fused", "gemv_fused_awq_g128", "MbwFusion", "FUSE_NORM", "FUSE_GLU", "FUSE_RESIDUAL", "repack_int4", "REPACKED",
    "dequant_int4_g64", "dequant_int4_awq_g128", "autotune", "plan_describe", "plan_candidates", "plan_select", "plan_index", "workspace_bytes",
    "launch_count", "check_device_error", "selftest_wait_expiry", "inject_launch_failures", "output_fp32", "MbwError",
    "OP_GEMV_BF16", "OP_GEMV_INT4_G64", "OP_GEMV_INT4_AWQ_G128", "OP_GEMM_SKINNY_BF16",
    "OP_GEMV_INT8_PC",
    "Kv4Cache", "kv4_page_bytes", "kv4_append", "kv4_gather", "kv4_attention", "kv4_attention_workspace",
    "token_logprobs", "token_logprobs_workspace", "TokenLogprobs",
    "quantize_fp8_g128", "quantize_fp8_b128", "dequant_fp8_g128", "dequant_fp8_b128", "gemm_fp8_b128",
    "kv4_attention_shared", "kv4_attention_shared_workspace",
))


_PLAN_FILES = ("save_plans", "load_plans")


def __getattr__(name):
    if name in _EXPORTS:
        from . import _binding

        value = globals()[name] = getattr(_binding, name)  # found here from now on; the binding keeps it its own (_Module)
        return value
    if name == "rope_table":
        from .rope import rope_table

        return rope_table
    if name in _PLAN_FILES:
        from . import plans

        return getattr(plans, name)
    raise AttributeError(name)
