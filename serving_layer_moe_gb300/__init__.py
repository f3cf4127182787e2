"""GB300-native expert-slot cache for MoE layers (FreeToken's decode hot path).

The work runs in libmoecache.so (hand-written CUDA for sm_103a, C ABI in
include/moe_cache.h and include/moe_operators.h); this package is its thin
Python binding.
"""
from .binding import (DTYPES, SYMBOLS, MoECache, MoEError, bench_bw, load_library)  # noqa: F401
from .operators import (OPERATOR_SYMBOLS, ExpertGroups, FP4Rows, check_operators, combine, dequantize_fp4,  # noqa: F401
                        fp4_scale, group_pairs, grouped_matmul, grouped_matmul_fp4, quantize_fp4, route)

__all__ = ["MoECache", "MoEError", "bench_bw", "load_library", "DTYPES", "SYMBOLS",
           "OPERATOR_SYMBOLS", "ExpertGroups", "FP4Rows", "check_operators", "combine", "dequantize_fp4", "fp4_scale",
           "group_pairs", "grouped_matmul", "grouped_matmul_fp4", "quantize_fp4", "route"]
