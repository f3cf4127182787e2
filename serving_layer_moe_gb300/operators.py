"""The operators around a cache of experts, on torch tensors (libmoecache.so, include/moe_operators.h).

    ids, w, groups = route(logits, top_k, groups=True)     # router, pairs in expert order
    xq = quantize_fp4(x, "nvfp4", g=gx, groups=groups)     # rows gathered by expert, 4-bit
    h = grouped_matmul_fp4(xq, gate_up, groups, act="swiglu", quantize=True, g_out=gh)
    y = grouped_matmul_fp4(h, down, groups)
    out = combine(y, groups, w)

Argument checks, output tensors and pointers only: the work is in the library's kernels, there is no
fallback.  Everything is enqueued on `stream` (torch's current stream if None); outputs are allocated for
that stream.  As with torch's own calls, a stream that is not the inputs' own has to be ordered behind what makes
them (Stream.wait_stream), and they have to stay until it is done (Tensor.record_stream).  Wrong arguments raise
ValueError before anything is enqueued.

One decoded token runs all five calls in the time of a few launches, so the ordinary call goes straight to
csrc/operators_host.cpp, which checks, allocates and launches.  What that leaves alone (it returns None) is
looked at here: a wrong argument raises, another device or stream is made current and the call made again.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import DTYPES, _check, load_library

OPERATOR_SYMBOLS = ("moe_grouped_tiles", "moe_group_workspace", "moe_route", "moe_group_pairs", "moe_fp4_scale",
                    "moe_quantize_fp4", "moe_dequantize_fp4", "moe_grouped_matmul_workspace", "moe_grouped_matmul",
                    "moe_grouped_matmul_fp4",
                    "moe_combine", "moe_operators_check", "moe_quantize_fp8", "moe_quantize_fp8_weights", "moe_dequantize_fp8",
                    "moe_grouped_matmul_fp8", "moe_combine_norm")

SCORING = {"softmax": 0, "sigmoid": 1}
ACTS = {None: 0, "none": 0, "swiglu": 1}
FP4_BLOCK = {"nvfp4": 16, "mxfp4": 32}
_FLOATS = {torch.float32: DTYPES["f32"], torch.bfloat16: DTYPES["bf16"]}
_MOST_PAIRS, _MOST_MATRICES, _MOST_ROWS, _MOST_K = 0x70000000, 65535, 0x7FFFFFFF, 1 << 24       # the library's limits
_F32, _BF16, _I32, _U8, _F8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8, torch.float8_e4m3fn
_MOST_WIDTH = 32768        # of a row of combine_norm

_lib = None
_host_module = None


def _host():
    """The C++ side of the binding (_operators.so)."""
    global _host_module
    if _host_module is None:
        _operators()
        try:
            import importlib
            host = importlib.import_module("._operators", __package__)
        except ImportError as e:
            raise RuntimeError(f"_operators.so is not built ({e}); build it with serving_layer_moe_gb300.build.build()") from e
        host.init(_check)
        _host_module = host
    return _host_module


def _operators():
    """The library with the operators' signatures declared."""
    global _lib
    if _lib is None:
        lib = load_library()
        P, I32, I64, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        sig = {
            "moe_grouped_tiles": [I64, I32],
            "moe_group_workspace": [I32, I32, I32],
            "moe_route": [I32, I32, I32, I32, P, I32, P, I32, I32, I32, F32, P, P, P, P, P, P, P, I64, P],
            "moe_group_pairs": [I32, I32, I32, P, P, P, P, P, P, I64, P],
            "moe_fp4_scale": [I32, I64, I32, P, P, P],
            "moe_quantize_fp4": [I32, I32, I32, I32, P, I32, P, I32, I32, I32, P, P, P, P, P, P],
            "moe_dequantize_fp4": [I32, I32, I32, I32, P, P, P, I32, I32, P, P, I32, P, P],
            "moe_grouped_matmul_workspace": [I32, I32, I32, I32],
            "moe_grouped_matmul": [I32, I32, I32, I32, P, I32, P, P, I32, P, P, P, I32, I32, P, P, I64, P],
            "moe_grouped_matmul_fp4": [I32, I32, I32, I32, I32, P, P, P, P, P, P, I32, P, P, I32, I32, P, P, P, P, P],
            "moe_combine": [I32, I32, I32, I32, P, P, P, I32, P, P],
            "moe_operators_check": [P],
            "moe_quantize_fp8": [I32, I32, I32, P, I32, P, P, P, P],
            "moe_quantize_fp8_weights": [I32, I32, I32, I32, P, P, P, P],
            "moe_dequantize_fp8": [I32, I32, I32, I32, P, P, I32, P, P],
            "moe_grouped_matmul_fp8": [I32, I32, I32, I32, P, P, P, P, P, I32, I32, P, P, P, P],
            "moe_combine_norm": [I32, I32, I32, I32, P, P, P, P, I32, P, I32, P, F32, I32, P, I32, P, F32, P, I32, P, P],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int64 if name == "moe_grouped_tiles" or name.endswith("_workspace") else ctypes.c_int
        _lib = lib
    return _lib


class _On:
    """A stream other than torch's current one, or another device: both current inside the block."""

    def __init__(self, index, stream):
        self.ctx = []
        if index != torch.cuda.current_device():
            self.ctx.append(torch.cuda.device(index))
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=index)
            self.ctx.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.ctx:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.ctx):
            c.__exit__(*exc)
        return False


def _stream(index):
    return torch.cuda.current_stream(index).cuda_stream


def _again(call, index, stream):
    """Make a call that was left alone again, on its own device and stream, now that its arguments are right."""
    if stream is None and index == torch.cuda.current_device():
        raise ValueError("the call was not made: tensors that its arguments hold were resized, moved or replaced since")
    with _On(index, stream):
        return call()


def _bad(t, name, dtypes, dim, index=None):
    """Raise what is wrong with an argument that should be a contiguous CUDA tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.dim() != dim or not t.is_contiguous():
        got = f"{t.dtype} {tuple(t.shape)}{'' if t.is_contiguous() else ' (not contiguous)'}" if isinstance(t, torch.Tensor) else type(t)
        raise ValueError(f"{name} must be a contiguous {dim}-dimensional tensor of {' or '.join(map(str, dtypes))}, got {got}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device, is on {t.device}")
    raise ValueError(f"{name} is on {t.device}, the other arguments on cuda:{index}")


def _shaped(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, is {tuple(t.shape)}")


def _floats(t, name, dim, index=None):
    """dtype code of a contiguous fp32 or bf16 CUDA tensor of `dim` dimensions (of device `index`)."""
    if not (isinstance(t, torch.Tensor) and t.dtype in _FLOATS and t.dim() == dim and t.is_contiguous() and t.is_cuda
            and (index is None or t.get_device() == index)):
        _bad(t, name, tuple(_FLOATS), dim, index)
    return _FLOATS[t.dtype]


def _typed(t, name, dtype, dim, index=None):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == dim and t.is_contiguous() and t.is_cuda
            and (index is None or t.get_device() == index)):
        _bad(t, name, (dtype,), dim, index)
    return t


def _matrices(G, N, K, multiple):
    """Sizes of a stack of matrices."""
    if K == 0 or K % multiple or K > _MOST_K:
        raise ValueError(f"K must be a multiple of {multiple}, {_MOST_K} at most, is {K}")
    if G > _MOST_MATRICES or N > _MOST_ROWS:
        raise ValueError(f"at most {_MOST_MATRICES} matrices of {_MOST_ROWS} rows are taken, got {G} of {N}")


def _scale(g, name, most, index):
    """An fp32 matrix scale of 1 or `most` values (None: no scale)."""
    if g is not None:
        _typed(g, name, _F32, 1, index)
        if g.numel() != 1 and g.numel() != most:
            raise ValueError(f"{name} must hold {'1' if most == 1 else f'1 or {most}'} values, holds {g.numel()}")


class ExpertGroups:
    """The (token, expert) pairs of a call in expert order: offsets and tiles [E + 1], order [T * k] and
    place [T, k], all int32 (include/moe_operators.h, "Expert order").  Types and sizes are checked here; the tensors
    cannot be exchanged after.  What they hold is not: other than a grouping it gives wrong results, inside the arrays."""

    __slots__ = ("_c", "_views")

    def __init__(self, offsets, tiles, order, place):
        self._c = _host().groups_of(offsets, tiles, order, place)
        if self._c is None:
            _typed(offsets, "offsets", _I32, 1)
            i = offsets.get_device()
            _typed(tiles, "tiles", _I32, 1, i)
            _typed(order, "order", _I32, 1, i)
            _typed(place, "place", _I32, 2, i)
            if tiles.numel() != offsets.numel() or not 2 <= offsets.numel() <= 4097:
                raise ValueError(f"offsets and tiles must hold E + 1 values each (1 <= E <= 4096), hold {offsets.numel()} and {tiles.numel()}")
            raise ValueError(f"order and place must hold the same number of pairs, {_MOST_PAIRS} at most, hold {order.numel()} and {place.numel()}")
        self._views = self._c[5:]

    @classmethod
    def _of(cls, c):
        """Of the host module's tuple, with all four in one buffer."""
        self = cls.__new__(cls)
        self._c, self._views = c, None
        return self

    def _view(self, i):
        if self._views is None:
            self._views = _host().views(self._c)
        return self._views[i]

    _index = property(lambda self: self._c[0])
    E = property(lambda self: self._c[1])
    P = property(lambda self: self._c[2])
    T = property(lambda self: self._c[3])
    k = property(lambda self: self._c[4])
    offsets = property(lambda self: self._view(0))
    tiles = property(lambda self: self._view(1))
    order = property(lambda self: self._view(2))
    place = property(lambda self: self._view(3))


def _described(groups):
    """What the host module takes for groups: their tuple, None, or False for anything else (which it leaves alone)."""
    return None if groups is None else groups._c if isinstance(groups, ExpertGroups) else False


def _groups_on(groups, index):
    if not isinstance(groups, ExpertGroups):
        raise ValueError(f"groups must be ExpertGroups, is {type(groups)}")
    if groups._index != index:
        raise ValueError(f"groups are on cuda:{groups._index}, the other arguments on cuda:{index}")
    return groups


class FP4Rows:
    """4-bit matrices: codes uint8 [..., K/2] and scale tiles uint8 [row tiles, block groups, 512]
    (include/moe_operators.h, "4-bit matrices"), wdtype "nvfp4" or "mxfp4", g the fp32 matrix scales (1 or one
    per matrix; None = 1).  groups: of rows in expert order; None for a stack of matrices [G, N, K] or one [N, K].
    Types and sizes are checked here; the tensors cannot be exchanged after."""

    __slots__ = ("_wdtype", "_groups", "_c")

    def __init__(self, codes, scales, wdtype, g=None, groups=None):
        if wdtype not in FP4_BLOCK:
            raise ValueError(f"wdtype must be 'nvfp4' or 'mxfp4', is {wdtype!r}")
        self._c = _host().rows_of(codes, scales, DTYPES[wdtype], g, _described(groups))
        if self._c is None:
            self._refuse(codes, scales, wdtype, g, groups)
        self._wdtype, self._groups = wdtype, groups

    @staticmethod
    def _refuse(codes, scales, wdtype, g, groups):
        dim = 2 if groups is not None or not isinstance(codes, torch.Tensor) or codes.dim() != 3 else 3
        _typed(codes, "codes", _U8, dim)
        i = codes.get_device()
        _typed(scales, "scales", _U8, 3, i)
        K = 2 * codes.shape[-1]
        _matrices(*((1, *codes.shape) if dim == 2 else codes.shape)[:2], K, 32)
        if groups is not None:
            _groups_on(groups, i)
            if codes.shape[0] != groups.P:
                raise ValueError(f"codes hold {codes.shape[0]} rows, groups {groups.P} pairs")
            G, n = 1, (groups.P + 127 * min(groups.P, groups.E)) // 128
        else:
            G, N = (1, codes.shape[0]) if dim == 2 else codes.shape[:2]
            n = G * -(-N // 128)
        want = (n, -(-K // (4 * FP4_BLOCK[wdtype])), 512)
        if tuple(scales.shape) != want:
            raise ValueError(f"scales must be {want}, is {tuple(scales.shape)}")
        _scale(g, "g", G, i)
        raise ValueError("codes and scales must be 16-byte aligned")

    @classmethod
    def _of(cls, wdtype, groups, c):
        """Of the host module's tuple."""
        self = cls.__new__(cls)
        self._wdtype, self._groups, self._c = wdtype, groups, c
        return self

    _index = property(lambda self: self._c[0])
    codes = property(lambda self: self._c[5])
    scales = property(lambda self: self._c[6])
    wdtype = property(lambda self: self._wdtype)
    g = property(lambda self: self._c[7])
    groups = property(lambda self: self._groups)
    K = property(lambda self: self._c[3])
    shape = property(lambda self: (*self.codes.shape[:-1], self._c[3]))


def _pairs(T, k):
    if T * k > _MOST_PAIRS:
        raise ValueError(f"{T} tokens of {k} experts are more than {_MOST_PAIRS} pairs")


def route(logits, top_k, *, scoring="softmax", bias=None, n_group=1, topk_group=1, renormalize=True, scale=1.0,
          groups=False, stream=None):
    """Experts and gates of each token: (topk_ids int32 [T, k], topk_w fp32 [T, k]), or with groups=True also the
    ExpertGroups of the picked pairs.  logits [T, E] fp32 or bf16; scoring "softmax" (by logit) or "sigmoid"
    (with an optional selection bias [E] and topk_group of n_group expert groups): moe_route.  ids and
    gates share an allocation, with the groups too up to 256 pairs."""
    if stream is None:
        r = (_host_module or _host()).route(logits, top_k, SCORING.get(scoring, -1), bias, n_group, topk_group, renormalize, scale, groups)
        if r is not None:
            return (r[0], r[1], ExpertGroups._of(r[2])) if groups else r[:2]
    _floats(logits, "logits", 2)
    E, k, index = logits.shape[1], int(top_k), logits.get_device()
    if scoring not in SCORING:
        raise ValueError(f"scoring must be 'softmax' or 'sigmoid', is {scoring!r}")
    if not 1 <= k <= E <= 4096:
        raise ValueError(f"1 <= top_k <= E <= 4096 is needed, got top_k {k}, E {E}")
    if scoring == "softmax" and (bias is not None or n_group != 1):
        raise ValueError("softmax scoring takes no bias and no expert groups")
    if bias is not None:
        _typed(bias, "bias", _F32, 1, index)
        if bias.numel() != E:
            raise ValueError(f"bias must hold E = {E} values, holds {bias.numel()}")
    if not (1 <= n_group <= 32 and E % n_group == 0 and 1 <= topk_group <= n_group and topk_group * (E // n_group) >= k):
        raise ValueError(f"n_group (1 to 32) must divide E and topk_group groups must hold top_k experts, got n_group {n_group}, "
                         f"topk_group {topk_group}, E {E}, top_k {k}")
    _pairs(logits.shape[0], k)
    return _again(lambda: route(logits, k, scoring=scoring, bias=bias, n_group=n_group, topk_group=topk_group, renormalize=renormalize,
                                scale=scale, groups=groups), index, stream)


def group_pairs(topk_ids, n_experts, *, stream=None):
    """ExpertGroups of topk_ids int32 [T, k]; pairs whose id is outside [0, n_experts) are dropped (place -1)."""
    _typed(topk_ids, "topk_ids", _I32, 2)
    T, k = topk_ids.shape
    E, index = int(n_experts), topk_ids.get_device()
    if not (1 <= E <= 4096 and k >= 1):
        raise ValueError(f"1 <= n_experts <= 4096 and k >= 1 are needed, got {E} and {k}")
    _pairs(T, k)
    if stream is not None or index != torch.cuda.current_device():
        return _again(lambda: group_pairs(topk_ids, E), index, stream)
    ops = _operators()
    ws, P = ops.moe_group_workspace(T, k, E), T * k
    buffer = torch.empty(2 * (E + 1 + P), dtype=_I32, device=topk_ids.device)
    scratch = torch.empty(ws // 4, dtype=_I32, device=topk_ids.device) if ws else None
    off = buffer.data_ptr()
    til = off + 4 * (E + 1)
    order = til + 4 * (E + 1)
    place = order + 4 * P
    _check(ops.moe_group_pairs(T, E, k, topk_ids.data_ptr(), off, til, order, place, scratch.data_ptr() if ws else None, ws,
                                _stream(index)))
    return ExpertGroups._of((index, E, P, T, k, buffer, 0, None, None))


def fp4_scale(x, *, stream=None):
    """NVFP4 matrix scales: max |x| times 1 / (6 * 448), of x [N, K] or of each matrix of x [G, N, K]; fp32 [1] or [G]."""
    dim = 3 if isinstance(x, torch.Tensor) and x.dim() == 3 else 2
    dt = _floats(x, "x", dim)
    index, n = x.get_device(), x.numel()
    if n == 0:
        raise ValueError(f"x is empty: {tuple(x.shape)}")
    if dim == 3 and x.shape[0] > _MOST_ROWS:
        raise ValueError(f"at most {_MOST_ROWS} matrices are taken, got {x.shape[0]}")
    if stream is not None or index != torch.cuda.current_device():
        return _again(lambda: fp4_scale(x), index, stream)
    G = x.shape[0] if dim == 3 else 1
    g = torch.empty(G, dtype=_F32, device=x.device)
    _check(_operators().moe_fp4_scale(G, n // G, dt, x.data_ptr(), g.data_ptr(), _stream(index)))
    return g


def quantize_fp4(x, wdtype, *, g=None, groups=None, stream=None):
    """x in 4 bits (moe_quantize_fp4).  Without groups: x [N, K] or a stack [G, N, K], g fp32 [1] or [G].  With
    groups: x [T, K], and the result holds row order[i] // k of x at grouped row i.  K a multiple of 32; g only
    for "nvfp4" (None = 1)."""
    if wdtype not in FP4_BLOCK:
        raise ValueError(f"wdtype must be 'nvfp4' or 'mxfp4', is {wdtype!r}")
    if stream is None:
        r = (_host_module or _host()).quantize(x, DTYPES[wdtype], g, _described(groups))
        if r is not None:
            return FP4Rows._of(wdtype, groups, r)
    dim = 2 if groups is not None or not isinstance(x, torch.Tensor) or x.dim() != 3 else 3
    _floats(x, "x", dim)
    index, K = x.get_device(), x.shape[-1]
    _matrices(*((1, *x.shape) if dim == 2 else x.shape)[:2], K, 32)
    if x.data_ptr() % 16:
        raise ValueError("x must be 16-byte aligned")
    if g is not None and wdtype != "nvfp4":
        raise ValueError("only nvfp4 takes a matrix scale g")
    if groups is not None:
        _groups_on(groups, index)
        if groups.T != x.shape[0]:
            raise ValueError(f"x has {x.shape[0]} rows, groups hold {groups.T} tokens")
    _scale(g, "g", x.shape[0] if dim == 3 else 1, index)
    return _again(lambda: quantize_fp4(x, wdtype, g=g, groups=groups), index, stream)


def _rows(q, name):
    if not isinstance(q, FP4Rows):
        raise ValueError(f"{name} must be FP4Rows, is {type(q)}")
    return q


def dequantize_fp4(q, *, out_dtype=torch.bfloat16, stream=None):
    """The values that q stands for, in q.shape; rows that no pair fills are zero (moe_dequantize_fp4)."""
    _rows(q, "q")
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    if stream is None:
        out = _host().dequantize(q._c, None if q.groups is None else q.groups._c, q.codes.dim() == 3, _FLOATS[out_dtype])
        if out is not None:
            return out
    return _again(lambda: dequantize_fp4(q, out_dtype=out_dtype), q._index, stream)


def _columns(groups, E, N, act, out_dtype):
    if groups.E != E:
        raise ValueError(f"w holds {E} experts, groups {groups.E}")
    if act not in ACTS:
        raise ValueError(f"act must be 'none' or 'swiglu', is {act!r}")
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    if ACTS[act] and N % 32:
        raise ValueError(f"swiglu needs w rows a multiple of 32, got {N}")
    return N // 2 if ACTS[act] else N


def grouped_matmul(x, w, groups, *, act="none", gather=False, out_dtype=torch.bfloat16, stream=None):
    """Row i of expert e: x[i] @ w[e].T, w [E, N, K] bf16, x bf16 [P, K] in expert order, or with gather=True
    [T, K] and grouped row i reads x[order[i] // k].  act="swiglu": w holds gate rows, then up rows, and the
    result has N/2 columns.  K a multiple of 8 (moe_grouped_matmul).  Rows that no pair fills are undefined.

    out_dtype: bf16 results are half the bytes on their way to combine.  fp32 ones save a rounding of each expert's
    row and are summed more exactly: a 4-bit layer on normal weights is then 0.0017 from 64 bits instead of 0.0024.
    One token takes the same time, 8192 tokens (NVFP4, K 2048, I 768) 441 us instead of 333."""
    if stream is None and isinstance(groups, ExpertGroups) and act in ACTS and out_dtype in _FLOATS:
        out = (_host_module or _host()).matmul(x, w, groups._c, ACTS[act], gather, _FLOATS[out_dtype])
        if out is not None:
            return out
    _typed(w, "w", _BF16, 3)
    index = w.get_device()
    _typed(x, "x", _BF16, 2, index)
    _groups_on(groups, index)
    E, N, K = w.shape
    _columns(groups, E, N, act, out_dtype)
    if N == 0:
        raise ValueError(f"w must be [E, N, K], is {tuple(w.shape)}")
    _matrices(E, N, K, 8)
    rows = groups.T if gather else groups.P
    if tuple(x.shape) != (rows, K):
        raise ValueError(f"x must be {(rows, K)}, is {tuple(x.shape)}")
    if (x.data_ptr() | w.data_ptr()) % 16:
        raise ValueError("x and w must be 16-byte aligned")
    return _again(lambda: grouped_matmul(x, w, groups, act=act, gather=gather, out_dtype=out_dtype), index, stream)


def grouped_matmul_fp4(x, w, groups, *, act="none", quantize=False, g_out=None, out_dtype=torch.bfloat16, stream=None):
    """grouped_matmul of 4-bit rows x (FP4Rows laid out by these groups) and 4-bit weights w (FP4Rows [E, N, K]) of one
    format.  quantize=True (act="swiglu" only): the result as FP4Rows of that format with the matrix scale g_out
    [1] (None = 1; "nvfp4" only), rounded from the fp32 values (moe_grouped_matmul_fp4).  out_dtype: as there."""
    _rows(x, "x")
    _rows(w, "w")
    if stream is None and x.groups is not None and isinstance(groups, ExpertGroups) and act in ACTS and out_dtype in _FLOATS and \
            w.codes.dim() == 3 and w.groups is None and (quantize or g_out is None):
        out = (_host_module or _host()).matmul_fp4(x._c, w._c, x.groups._c, groups._c, ACTS[act], g_out if quantize else False, _FLOATS[out_dtype])
        if out is not None:
            return FP4Rows._of(x.wdtype, groups, out) if quantize else out
    index = w._index
    _groups_on(groups, index)
    if w.codes.dim() != 3 or w.groups is not None:
        raise ValueError(f"w must be [E, N, K], is {w.shape}")
    E, N, K = w.shape
    cols = _columns(groups, E, N, act, out_dtype)
    if x.groups is None or x._index != index or x.groups.E != E or N == 0:
        raise ValueError("x must hold rows in the order of w's experts, on the same device")
    if x.wdtype != w.wdtype:
        raise ValueError(f"x is {x.wdtype}, w is {w.wdtype}")
    if x.shape != (groups.P, K):
        raise ValueError(f"x must be {(groups.P, K)}, is {x.shape}")
    if x.groups.offsets.data_ptr() != groups.offsets.data_ptr() or x.groups.tiles.data_ptr() != groups.tiles.data_ptr():
        raise ValueError("x is laid out by other groups than the call's")
    if quantize and not (ACTS[act] and cols % 32 == 0):
        raise ValueError("quantize needs act='swiglu' and w rows a multiple of 64")
    if g_out is not None and not (quantize and x.wdtype == "nvfp4"):
        raise ValueError("g_out goes with quantize=True and nvfp4")
    _scale(g_out, "g_out", 1, index)
    return _again(lambda: grouped_matmul_fp4(x, w, groups, act=act, quantize=quantize, g_out=g_out, out_dtype=out_dtype), index, stream)


def combine(y, groups, topk_w, *, out_dtype=torch.float32, stream=None):
    """out[t] = sum_j topk_w[t, j] * y[place[t, j]], y [P, N] bf16 or fp32 in expert order; pairs dropped from the
    groups contribute nothing (moe_combine)."""
    if stream is None and isinstance(groups, ExpertGroups) and out_dtype in _FLOATS:
        out = (_host_module or _host()).combine(y, groups._c, topk_w, _FLOATS[out_dtype])
        if out is not None:
            return out
    _floats(y, "y", 2)
    index = y.get_device()
    _groups_on(groups, index)
    _typed(topk_w, "topk_w", _F32, 2, index)
    if tuple(topk_w.shape) != (groups.T, groups.k):
        raise ValueError(f"topk_w must be {(groups.T, groups.k)}, is {tuple(topk_w.shape)}")
    if y.shape[0] != groups.P or y.shape[1] == 0:
        raise ValueError(f"y must be [{groups.P}, N], is {tuple(y.shape)}")
    if y.shape[1] % 8 == 0 and y.data_ptr() % 16:
        raise ValueError("y must be 16-byte aligned where its rows are multiples of 16 bytes")
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    return _again(lambda: combine(y, groups, topk_w, out_dtype=out_dtype), index, stream)


class _Blocks8:
    """8-bit codes and the scales of their blocks, of one device.  The tensors cannot be exchanged after."""

    __slots__ = ("_codes", "_scales")
    _rows = False

    def __init__(self, codes, scales):
        if not (_host_module or _host()).blocks8(codes, scales, self._rows):
            self._check(codes, scales)
        self._codes, self._scales = codes, scales

    @classmethod
    def _of(cls, codes, scales):
        """Of the host module's tensors."""
        self = cls.__new__(cls)
        self._codes, self._scales = codes, scales
        return self

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    shape = property(lambda self: tuple(self._codes.shape))
    K = property(lambda self: self._codes.shape[-1])
    _index = property(lambda self: self._codes.get_device())


def _aligned(**tensors):
    for name, t in tensors.items():
        if t.data_ptr() % 16:
            raise ValueError(f"{name} must be 16-byte aligned")


class FP8Rows(_Blocks8):
    """8-bit rows: codes float8_e4m3fn [R, K] and fp32 scales [ceil(K / 128), R], one for 128 elements of a row
    (include/moe_operators.h, "8-bit blocks").  Rows in expert order are rows like others."""

    __slots__ = ()
    _rows = True

    @staticmethod
    def _check(codes, scales):
        _typed(codes, "codes", _F8, 2)
        _typed(scales, "scales", _F32, 2, codes.get_device())
        R, K = codes.shape
        _matrices(1, R, K, 16)
        _shaped(scales, "scales", (-(-K // 128), R))
        _aligned(codes=codes)


class FP8Weights(_Blocks8):
    """8-bit weights: codes float8_e4m3fn [N, K] and fp32 scales [ceil(N / 128), ceil(K / 128)], one for 128 x 128 elements, or
    a stack of G of both (include/moe_operators.h, "8-bit blocks")."""

    __slots__ = ()

    @staticmethod
    def _check(codes, scales):
        dim = 3 if isinstance(codes, torch.Tensor) and codes.dim() == 3 else 2
        _typed(codes, "codes", _F8, dim)
        _typed(scales, "scales", _F32, dim, codes.get_device())
        G, N, K = codes.shape if dim == 3 else (1, *codes.shape)
        _matrices(G, N, K, 16)
        _shaped(scales, "scales", (*codes.shape[:-2], -(-N // 128), -(-K // 128)))
        _aligned(codes=codes)


def _blocks8(q, name, kind):
    if not isinstance(q, kind):
        raise ValueError(f"{name} must be {kind.__name__ if isinstance(kind, type) else 'FP8Rows or FP8Weights'}, is {type(q)}")
    kind = type(q)
    kind._check(q._codes, q._scales)      # they may have been resized since
    return q


def quantize_fp8(x, *, groups=None, stream=None):
    """Rows x [T, K] fp32 or bf16 as FP8Rows, K a multiple of 16 (moe_quantize_fp8).  With groups the result holds row
    order[i] // k of x at grouped row i; rows that no pair fills are undefined."""
    if stream is None:
        r = (_host_module or _host()).quantize8(x, _described(groups))
        if r is not None:
            return FP8Rows._of(*r)
    _floats(x, "x", 2)
    index = x.get_device()
    T, K = x.shape
    _matrices(1, T, K, 16)
    _aligned(x=x)
    if groups is not None:
        _groups_on(groups, index)
        if groups.T != T:
            raise ValueError(f"x has {T} rows, groups hold {groups.T} tokens")
        if groups.k < 1:
            raise ValueError("groups hold no experts a token")
    else:
        _pairs(T, 1)
    return _again(lambda: quantize_fp8(x, groups=groups), index, stream)


def quantize_fp8_weights(w, *, stream=None):
    """Weights w [N, K] or [G, N, K], fp32 or bf16, as FP8Weights, K a multiple of 16 (moe_quantize_fp8_weights)."""
    if stream is None:
        r = (_host_module or _host()).quantize_weights8(w)
        if r is not None:
            return FP8Weights._of(*r)
    dim = 3 if isinstance(w, torch.Tensor) and w.dim() == 3 else 2
    _floats(w, "w", dim)
    index = w.get_device()
    G, N, K = w.shape if dim == 3 else (1, *w.shape)
    _matrices(G, N, K, 16)
    if -(-N // 128) * -(-K // 128) > _MOST_ROWS:
        raise ValueError(f"a matrix may have {_MOST_ROWS} blocks at most, got {N} x {K} elements")
    _aligned(w=w)
    return _again(lambda: quantize_fp8_weights(w), index, stream)


def dequantize_fp8(q, *, out_dtype=torch.bfloat16, stream=None):
    """The values that q (FP8Rows or FP8Weights) stands for, in q.shape (moe_dequantize_fp8)."""
    if stream is None and isinstance(q, _Blocks8) and out_dtype in _FLOATS:
        out = (_host_module or _host()).dequantize8(q._codes, q._scales, q._rows, _FLOATS[out_dtype])
        if out is not None:
            return out
    _blocks8(q, "q", (FP8Rows, FP8Weights))
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    return _again(lambda: dequantize_fp8(q, out_dtype=out_dtype), q._index, stream)


def _product8(x, w, groups, act, quantize, out_dtype, stream):
    if stream is None and isinstance(x, FP8Rows) and isinstance(w, FP8Weights) and act in ACTS and out_dtype in _FLOATS:
        r = (_host_module or _host()).matmul8(x._codes, x._scales, w._codes, w._scales, _described(groups), ACTS[act], quantize, _FLOATS[out_dtype])
        if r is not None:
            return FP8Rows._of(*r) if isinstance(r, tuple) else r
    _blocks8(x, "x", FP8Rows)
    _blocks8(w, "w", FP8Weights)
    index = w._index
    want = 2 if groups is None else 3
    if len(w.shape) != want:
        raise ValueError(f"w must be {'[N, K]' if groups is None else '[E, N, K]'}, is {w.shape}")
    E, N, K = (1, *w.shape) if groups is None else w.shape
    P = x.shape[0]
    if groups is not None:
        _groups_on(groups, index)
        if groups.E != E:
            raise ValueError(f"w holds {E} experts, groups {groups.E}")
        if not 1 <= E <= 4096:
            raise ValueError(f"1 <= E <= 4096 is needed, got {E}")
        P = groups.P
    if x._index != index:
        raise ValueError(f"x is on cuda:{x._index}, w on cuda:{index}")
    if x.shape != (P, K):
        raise ValueError(f"x must be {(P, K)}, is {x.shape}")
    if N == 0:
        raise ValueError(f"w must have rows, is {w.shape}")
    _pairs(P, 1)
    if act not in ACTS:
        raise ValueError(f"act must be 'none' or 'swiglu', is {act!r}")
    if ACTS[act] and N % 128:
        raise ValueError(f"swiglu needs w rows a multiple of 128, got {N}")
    if quantize and not ACTS[act]:
        raise ValueError("quantize needs act='swiglu'")
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    return _again(lambda: _product8(x, w, groups, act, quantize, out_dtype, None), index, stream)


def matmul_fp8(x, w, *, act="none", quantize=False, out_dtype=torch.bfloat16, stream=None):
    """x @ w.T of FP8Rows x [R, K] and FP8Weights w [N, K], in out_dtype (moe_grouped_matmul_fp8 of one matrix).
    act="swiglu": w holds gate rows, then up rows (N a multiple of 128), and the result has N/2 columns; quantize=True: that
    result as FP8Rows, rounded from the fp32 values.

    out_dtype: bf16 results are half the bytes on their way to combine_norm, and each is off by up to half a bf16 step.  The sum of
    eight experts' rows (K 768, N 2048) is 0.0017 from 64 bits with bf16 rows and 9e-8 with fp32 ones; 8192 tokens' product takes
    136 us and 173."""
    return _product8(x, w, None, act, quantize, out_dtype, stream)


def grouped_matmul_fp8(x, w, groups, *, act="none", quantize=False, out_dtype=torch.bfloat16, stream=None):
    """matmul_fp8 for rows in expert order: row i of expert e is x[i] @ w[e].T, w FP8Weights [E, N, K] (moe_grouped_matmul_fp8).
    Rows that no pair fills are undefined.  out_dtype: as there."""
    if not isinstance(groups, ExpertGroups):
        raise ValueError(f"groups must be ExpertGroups, is {type(groups)}")
    return _product8(x, w, groups, act, quantize, out_dtype, stream)


def _block_end(y, groups, topk_w, residual, shared, post, gate, scale, pre, eps, out_dtype, stream):
    """The calls that the host module has left alone."""
    _floats(residual, "residual", 2)
    index = residual.get_device()
    T, N = residual.shape
    if not 1 <= N <= _MOST_WIDTH:
        raise ValueError(f"rows of 1 to {_MOST_WIDTH} elements are taken, got {N}")
    if y is not None:
        _floats(y, "y", 2, index)
        if groups is not None:
            _groups_on(groups, index)
            _typed(topk_w, "topk_w", _F32, 2, index)
            _shaped(topk_w, "topk_w", (groups.T, groups.k))
            if groups.T != T:
                raise ValueError(f"residual has {T} rows, groups hold {groups.T} tokens")
            if groups.k < 1:
                raise ValueError("groups hold no experts a token")
        _shaped(y, "y", (T if groups is None else groups.P, N))
        _pairs(T, 1 if groups is None else groups.k)
    else:
        _pairs(T, 1)
    if shared is not None:
        _typed(shared, "shared", y.dtype, 2, index)
        _shaped(shared, "shared", (T, N))
    for name, t in (("post", post), ("pre", pre)):
        if t is not None:
            _floats(t, name, 1, index)
            _shaped(t, name, (N,))
    if gate is not None:
        _typed(gate, "gate", _F32, 2 if isinstance(gate, torch.Tensor) and gate.dim() == 2 else 1, index)
        _shaped(gate, "gate", (T, 1) if gate.dim() == 2 else (N,))
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    if not 1.1754944e-38 <= eps <= 3e38:
        raise ValueError(f"eps must be a positive normal number, is {eps}")
    if not abs(scale) <= 3.4e38:
        raise ValueError(f"residual_scale must be finite, is {scale}")
    if N % 8 == 0:
        for name, t in (("y", y), ("residual", residual), ("shared", shared), ("post", post), ("pre", pre), ("gate", gate)):
            if t is not None and (name != "gate" or t.dim() == 1) and t.data_ptr() % 16:
                raise ValueError(f"{name} must be 16-byte aligned where rows are a multiple of 8 elements")
    call = _host().block_end
    r = _again(lambda: call(y, _described(groups), topk_w, residual, shared, post, gate, scale, pre, eps, _FLOATS[out_dtype]), index, stream)
    if r is None:
        raise ValueError("the call was not made: tensors that its groups hold were resized, moved or replaced since")
    return r


def combine_norm(y, groups, topk_w, residual, *, shared=None, post=None, gate=None, residual_scale=1.0, pre=None, eps=1e-6,
                 out_dtype=torch.bfloat16, stream=None):
    """The end of a block of experts: c = combine(y, groups, topk_w) + shared, its RMS norm with weights post, times gate;
    h = residual_scale * residual + c, in residual's type; with the next block's norm weights pre also z = its RMS norm,
    in out_dtype: (h, z), else h (moe_combine_norm).  y [P, N], shared [T, N] in y's type, residual [T, N], fp32 or bf16;
    post and pre [N], fp32 or bf16; gate fp32, [N] for a value a channel or [T, 1] for one a token."""
    if not isinstance(groups, ExpertGroups):
        raise ValueError(f"groups must be ExpertGroups, is {type(groups)}")
    if y is None:
        raise ValueError("y must be a tensor, is None")
    if stream is None and out_dtype in _FLOATS:
        r = (_host_module or _host()).block_end(y, groups._c, topk_w, residual, shared, post, gate, residual_scale, pre, eps, _FLOATS[out_dtype])
        if r is not None:
            return r
    return _block_end(y, groups, topk_w, residual, shared, post, gate, residual_scale, pre, eps, out_dtype, stream)


def residual_norm(y, residual, *, post=None, gate=None, residual_scale=1.0, pre=None, eps=1e-6, out_dtype=torch.bfloat16, stream=None):
    """combine_norm for a block that is no mixture: y [T, N] holds a row for each token."""
    if y is None:
        raise ValueError("y must be a tensor, is None")
    if stream is None and out_dtype in _FLOATS:
        r = (_host_module or _host()).block_end(y, None, None, residual, None, post, gate, residual_scale, pre, eps, _FLOATS[out_dtype])
        if r is not None:
            return r
    return _block_end(y, None, None, residual, None, post, gate, residual_scale, pre, eps, out_dtype, stream)


def rms_norm(x, weight, *, eps=1e-6, out_dtype=torch.bfloat16, stream=None):
    """x / sqrt(mean(x^2) + eps) * weight of the rows of x [T, N], in out_dtype: the norm before the first block (moe_combine_norm)."""
    if weight is None:
        raise ValueError("weight must be a tensor, is None")
    if stream is None and out_dtype in _FLOATS:
        r = (_host_module or _host()).block_end(None, None, None, x, None, None, None, 1.0, weight, eps, _FLOATS[out_dtype])
        if r is not None:
            return r
    return _block_end(None, None, None, x, None, None, None, 1.0, weight, eps, out_dtype, stream)


def check_operators(stream=None):
    """Synchronise the stream; MoEError if a bounded wait inside an operator kernel ran out since the last check."""
    if stream is None:
        stream = torch.cuda.current_stream()
    _check(_operators().moe_operators_check(getattr(stream, "cuda_stream", stream)))
