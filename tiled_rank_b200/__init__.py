"""TileQ fused MoE-layer forward for NVIDIA B200 (sm_100a).

The computation lives in libtileq.so (C ABI, include/tileq.h); this package is
its thin ctypes binding plus a helper that keeps a layer's device tensors.
"""
from ._lib import (  # noqa: F401
    TILEQ_LINEAR, TILEQ_SWIGLU, TILEQ_ROUTE_FULL_SOFTMAX, TILEQ_ROUTE_TOPK_SOFTMAX, TileQError,
    TILEQ_ERR_TIMEOUT, TILEQ_ERR_RANGE,
    status_string, tileq_device_status,
    tileq_moe_forward, tileq_moe_forward_unfused, tileq_pack, tileq_pack_per_expert,
    tileq_packed_per_expert_size, tileq_packed_size, tileq_route, tileq_route_static,
    tileq_selftest_bounded_wait,
    tileq_workspace_size, tileq_set_stage_events, tileq_launch_count,
    tileq_wbig, tileq_sketch_workspace_size, tileq_sketch_lowrank,
    tileq_place_in, tileq_place_out, place_in, tileq_place_workspace_size, tileq_place_experts,
    TILEQ_DT_BF16, TILEQ_DT_F16, TILEQ_DT_F32, TILEQ_DT_E4M3, tileq_grouped,
    tileq_grouped_gemm, tileq_grouped_gemm_dx, tileq_grouped_gemm_dw, tileq_fp8_rows,
    tileq_fp8_quantize, tileq_fp8_quantize_weights, tileq_fp8_gemm,
)
from .layer import DeviceLayer  # noqa: F401

# the products with the experts' uncompressed weights work on torch tensors: torch is imported with their first use
_EXPERTS = ("expert_status", "fp8_gemm", "fp8_quantize", "fp8_quantize_weights", "grouped_gemm",
            "grouped_gemm_dw", "grouped_gemm_dx")


def __getattr__(name):
    if name in _EXPERTS:
        from . import experts
        globals().update({n: getattr(experts, n) for n in _EXPERTS})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted([*globals(), *_EXPERTS])
