"""GB300 (sm_103a) fused "reduce R partials -> add residual -> RMSNorm ->
optional FP8 / NVFP4 quantise" epilogue and sharded MiniMax QK-RMSNorm, with
the NVFP4 and expert-routing operators that take up its outputs and the
attention over a 4-bit cache.

The computation runs in ``libts_fused_norm.so`` (hand-written CUDA, C ABI in
include/ts_fused_norm.h, include/ts_nvfp4_moe.h and include/ts_attention.h); this package is its thin
Python binding plus the seeded synthetic workloads (``workloads``).  The library is loaded lazily, on
the first call.
"""
from ._attention import (KVCache, ts_kv_cache, ts_kv_cache_read, ts_nvfp4_attention, ts_qk_norm_rope,  # noqa: F401
                         ts_qk_norm_rope_grad)
from ._binding import (EXPORTS, TS_FLAG_PDL, AGPattern, Pattern, RSPattern, SFLayout, TsError,  # noqa: F401
                       TsOuts, library, new_outputs, rs_token_split, sf_shape, sf_swizzled_shape,
                       ts_allgather_fused_norm, ts_fused_reduce_norm, ts_qk_norm_sharded,
                       ts_reducescatter_fused_norm, ts_rms_norm_sharded, ts_status_string)
from ._nvfp4_moe import (MoERows, ts_moe_combine, ts_moe_combine_grad, ts_moe_dispatch, ts_moe_rows,  # noqa: F401
                         ts_moe_sort, ts_nvfp4_dequantize, ts_nvfp4_gemm, ts_nvfp4_grouped_gemm, ts_nvfp4_quantize,
                         ts_stalled_waits)
