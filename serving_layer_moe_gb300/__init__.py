"""GB300-native expert-slot cache for MoE layers (FreeToken's decode hot path).

The work runs in libmoecache.so (hand-written CUDA for sm_103a, C ABI in
include/moe_cache.h and include/moe_operators.h); this package is its thin
Python binding.  The cache needs no torch until it is given torch tensors; the
operators are torch's, and come with the first use of one of their names.
"""
import importlib as _importlib
import importlib.util as _util

from .binding import (DTYPES, SYMBOLS, MoECache, MoEError, bench_bw, load_library)  # noqa: F401

_OPERATORS = ("OPERATOR_SYMBOLS", "ExpertGroups", "FP4Rows", "check_operators", "combine", "dequantize_fp4", "fp4_scale",
              "group_pairs", "grouped_matmul", "grouped_matmul_fp4", "quantize_fp4", "route")

__all__ = ["MoECache", "MoEError", "bench_bw", "load_library", "DTYPES", "SYMBOLS"]
if _util.find_spec("torch") is not None:
    __all__ += _OPERATORS


def __getattr__(name):
    if name != "operators" and name not in _OPERATORS:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    operators = _importlib.import_module(".operators", __name__)
    globals().update({n: getattr(operators, n) for n in _OPERATORS})
    return globals()[name]


def __dir__():
    return sorted({*globals(), *_OPERATORS, "operators"})
