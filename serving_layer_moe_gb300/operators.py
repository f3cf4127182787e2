"""The operators around a cache of experts, on torch tensors (libmoecache.so, include/moe_operators.h).

    ids, w, groups = route(logits, top_k, groups=True)     # router, pairs in expert order
    xq = quantize_fp4(x, "nvfp4", g=gx, groups=groups)     # rows gathered by expert, 4-bit
    h = grouped_matmul_fp4(xq, gate_up, groups, act="swiglu", quantize=True, g_out=gh)
    y = grouped_matmul_fp4(h, down, groups)
    out = combine(y, groups, w)

Argument checks, output tensors and pointers only: the work is in the library's kernels, there is no
fallback.  Everything is enqueued on `stream` (torch's current stream if None); outputs are allocated for
that stream.  Wrong arguments raise ValueError before anything is enqueued.

One decoded token runs all five calls in the time of a few launches, so the calls are kept short: a whole
argument is checked in one expression, and only a failed one is looked at again for its message.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import DTYPES, _check, load_library

OPERATOR_SYMBOLS = ("moe_grouped_tiles", "moe_group_workspace", "moe_route", "moe_group_pairs", "moe_fp4_scale",
                    "moe_quantize_fp4", "moe_dequantize_fp4", "moe_grouped_matmul_workspace", "moe_grouped_matmul",
                    "moe_grouped_matmul_fp4",
                    "moe_combine", "moe_operators_check")

SCORING = {"softmax": 0, "sigmoid": 1}
ACTS = {None: 0, "none": 0, "swiglu": 1}
FP4_BLOCK = {"nvfp4": 16, "mxfp4": 32}
_FLOATS = {torch.float32: DTYPES["f32"], torch.bfloat16: DTYPES["bf16"]}
_F32, _BF16, _I32, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8

_lib = None


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
            "moe_grouped_matmul": [I32, I32, I32, I32, P, I32, P, I32, P, P, P, I32, I32, P, P, I64, P],
            "moe_grouped_matmul_fp4": [I32, I32, I32, I32, I32, P, P, P, P, P, P, I32, P, P, I32, I32, P, P, P, P, P],
            "moe_combine": [I32, I32, I32, I32, P, P, P, I32, P, P],
            "moe_operators_check": [P],
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


def _elsewhere(index, stream):
    """Whether a call for tensors of device `index` has to make another stream or device current first."""
    return stream is not None or index != torch.cuda.current_device()


def _stream(index):
    return torch.cuda.current_stream(index).cuda_stream


try:    # the same without building Stream objects, where this torch has it
    _stream = torch._C._cuda_getCurrentRawStream
except AttributeError:
    pass


def _bad(t, name, dtypes, dim, index=None):
    """Raise what is wrong with an argument that should be a contiguous CUDA tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.dim() != dim or not t.is_contiguous():
        got = f"{t.dtype} {tuple(t.shape)}{'' if t.is_contiguous() else ' (not contiguous)'}" if isinstance(t, torch.Tensor) else type(t)
        raise ValueError(f"{name} must be a contiguous {dim}-dimensional tensor of {' or '.join(map(str, dtypes))}, got {got}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device, is on {t.device}")
    raise ValueError(f"{name} is on {t.device}, the other arguments on cuda:{index}")


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


def _scale_ptr(g, name, most, index):
    """Pointer and count of an fp32 matrix scale of 1 or `most` values (None: no scale)."""
    if g is None:
        return None, 0
    _typed(g, name, _F32, 1, index)
    n = g.numel()
    if not (n == 1 or n == most):
        raise ValueError(f"{name} must hold {'1' if most == 1 else f'1 or {most}'} values, holds {n}")
    return g.data_ptr(), n


class ExpertGroups:
    """The (token, expert) pairs of a call in expert order: offsets and tiles [E + 1], order [T * k] and
    place [T, k], all int32 (include/moe_operators.h, "Expert order").  Checked here, once, and not changed after."""

    __slots__ = ("E", "P", "T", "k", "_index", "_ptrs", "_all", "_views")

    def __init__(self, offsets, tiles, order, place):
        _typed(offsets, "offsets", _I32, 1)
        i = offsets.get_device()
        _typed(tiles, "tiles", _I32, 1, i)
        _typed(order, "order", _I32, 1, i)
        _typed(place, "place", _I32, 2, i)
        self.E, self.P, self._index = offsets.numel() - 1, order.numel(), i
        self.T, self.k = place.shape
        if not (1 <= self.E <= 4096 and tiles.numel() == self.E + 1):
            raise ValueError(f"offsets and tiles must hold E + 1 values each (1 <= E <= 4096), hold {offsets.numel()} and {tiles.numel()}")
        if self.T * self.k != self.P:
            raise ValueError(f"order holds {self.P} pairs, place {self.T * self.k}")
        self._ptrs = (offsets.data_ptr(), tiles.data_ptr(), order.data_ptr(), place.data_ptr())
        self._views = [offsets, tiles, order, place]
        self._all = None

    @classmethod
    def _empty(cls, T, k, E, like):
        """Room for the grouping of T tokens, on the device of `like`, and the call's arguments for it."""
        self = cls.__new__(cls)
        P = T * k
        self.E, self.P, self.T, self.k, self._index = E, P, T, k, like.get_device()
        ws = _operators().moe_group_workspace(T, k, E)
        n = 2 * (E + 1) + 2 * P
        self._all = torch.empty(n + ws // 4, dtype=_I32, device=like.device)     # the workspace last
        p = self._all.data_ptr()
        self._ptrs = (p, p + 4 * (E + 1), p + 8 * (E + 1), p + 8 * (E + 1) + 4 * P)
        self._views = None
        return self, (*self._ptrs, p + 4 * n if ws else None, ws)

    def _view(self, i):
        if self._views is None:
            e = self.E + 1
            v = list(self._all[:2 * (e + self.P)].split((e, e, self.P, self.P)))
            v[3] = v[3].view(self.T, self.k)
            self._views = v
        return self._views[i]

    offsets = property(lambda self: self._view(0))
    tiles = property(lambda self: self._view(1))
    order = property(lambda self: self._view(2))
    place = property(lambda self: self._view(3))


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
    Checked here, once, and not changed after."""

    __slots__ = ("codes", "scales", "wdtype", "g", "groups", "shape", "K", "_stack", "_index", "_ptrs")

    def __init__(self, codes, scales, wdtype, g=None, groups=None):
        if wdtype not in FP4_BLOCK:
            raise ValueError(f"wdtype must be 'nvfp4' or 'mxfp4', is {wdtype!r}")
        dim = 2 if groups is not None or not isinstance(codes, torch.Tensor) or codes.dim() != 3 else 3
        _typed(codes, "codes", _U8, dim)
        i = codes.get_device()
        _typed(scales, "scales", _U8, 3, i)
        K = 2 * codes.shape[-1]
        if not (K > 0 and K % 32 == 0):
            raise ValueError(f"K must be a multiple of 32, is {K}")
        if groups is not None:
            _groups_on(groups, i)
            if codes.shape[0] != groups.P:
                raise ValueError(f"codes hold {codes.shape[0]} rows, groups {groups.P} pairs")
            n = _grouped_tiles(groups.P, groups.E)
            self._stack = (1, groups.P)
        else:
            self._stack = (1, codes.shape[0]) if dim == 2 else (codes.shape[0], codes.shape[1])
            n = self._stack[0] * -(-self._stack[1] // 128)
        want = (n, _block_groups(wdtype, K), 512)
        if tuple(scales.shape) != want:
            raise ValueError(f"scales must be {want}, is {tuple(scales.shape)}")
        cp, sp = codes.data_ptr(), scales.data_ptr()
        if (cp | sp) % 16:
            raise ValueError("codes and scales must be 16-byte aligned")
        gp, gn = _scale_ptr(g, "g", self._stack[0], i)
        self.codes, self.scales, self.wdtype, self.g, self.groups = codes, scales, wdtype, g, groups
        self.K, self._index, self._ptrs = K, i, (cp, sp, gp, gn)
        self.shape = (*codes.shape[:-1], K)

    @classmethod
    def _empty(cls, shape, wdtype, g, gp, groups, stack, like):
        """Room for rows of `shape`, on the device of `like`; gp: pointer and count of g."""
        self = cls.__new__(cls)
        K = shape[-1]
        n = _grouped_tiles(groups.P, groups.E) if groups is not None else stack[0] * -(-stack[1] // 128)
        self.codes = torch.empty((*shape[:-1], K // 2), dtype=_U8, device=like.device)
        self.scales = torch.empty((n, _block_groups(wdtype, K), 512), dtype=_U8, device=like.device)
        self.wdtype, self.g, self.groups, self.shape, self.K, self._stack = wdtype, g, groups, shape, K, stack
        self._index = like.get_device()
        self._ptrs = (self.codes.data_ptr(), self.scales.data_ptr(), *gp)
        return self


def _block_groups(wdtype, K):
    return -(-K // (4 * FP4_BLOCK[wdtype]))


def _grouped_tiles(P, E):
    return (P + 127 * min(P, E)) // 128


def route(logits, top_k, *, scoring="softmax", bias=None, n_group=1, topk_group=1, renormalize=True, scale=1.0,
          groups=False, stream=None):
    """Experts and gates of each token: (topk_ids int32 [T, k], topk_w fp32 [T, k]), or with groups=True also the
    ExpertGroups of the picked pairs.  logits [T, E] fp32 or bf16; scoring "softmax" (by logit) or "sigmoid"
    (with an optional selection bias [E] and topk_group of n_group expert groups): moe_route."""
    dt = _floats(logits, "logits", 2)
    T, E = logits.shape
    k, index = int(top_k), logits.get_device()
    if scoring not in SCORING:
        raise ValueError(f"scoring must be 'softmax' or 'sigmoid', is {scoring!r}")
    if not 1 <= k <= E <= 4096:
        raise ValueError(f"1 <= top_k <= E <= 4096 is needed, got top_k {k}, E {E}")
    sc = SCORING[scoring]
    if not (sc or (bias is None and n_group == 1)):
        raise ValueError("softmax scoring takes no bias and no expert groups")
    if bias is not None:
        _typed(bias, "bias", _F32, 1, index)
        if bias.numel() != E:
            raise ValueError(f"bias must hold E = {E} values, holds {bias.numel()}")
    if n_group != 1 or topk_group != 1:
        if not (1 <= n_group <= 32 and E % n_group == 0 and 1 <= topk_group <= n_group and topk_group * (E // n_group) >= k):
            raise ValueError(f"n_group (1 to 32) must divide E and topk_group groups must hold top_k experts, got n_group {n_group}, "
                                 f"topk_group {topk_group}, E {E}, top_k {k}")
    if _elsewhere(index, stream):
        with _On(index, stream):
            return route(logits, k, scoring=scoring, bias=bias, n_group=n_group, topk_group=topk_group,
                         renormalize=renormalize, scale=scale, groups=groups)
    ids = torch.empty((T, k), dtype=_I32, device=logits.device)
    w = torch.empty((T, k), dtype=_F32, device=logits.device)
    if groups:
        gr, rest = ExpertGroups._empty(T, k, E, logits)
    else:
        rest = (None, None, None, None, None, 0)
    _check(_operators().moe_route(T, E, k, dt, logits.data_ptr(), sc, None if bias is None else bias.data_ptr(), n_group,
                                  topk_group, 1 if renormalize else 0, scale, ids.data_ptr(), w.data_ptr(), *rest, _stream(index)))
    return (ids, w, gr) if groups else (ids, w)


def group_pairs(topk_ids, n_experts, *, stream=None):
    """ExpertGroups of topk_ids int32 [T, k]; pairs whose id is outside [0, n_experts) are dropped (place -1)."""
    _typed(topk_ids, "topk_ids", _I32, 2)
    T, k = topk_ids.shape
    E, index = int(n_experts), topk_ids.get_device()
    if not (1 <= E <= 4096 and k >= 1):
        raise ValueError(f"1 <= n_experts <= 4096 and k >= 1 are needed, got {E} and {k}")
    if _elsewhere(index, stream):
        with _On(index, stream):
            return group_pairs(topk_ids, E)
    gr, rest = ExpertGroups._empty(T, k, E, topk_ids)
    _check(_operators().moe_group_pairs(T, E, k, topk_ids.data_ptr(), *rest, _stream(index)))
    return gr


def fp4_scale(x, *, stream=None):
    """NVFP4 matrix scales: max |x| / (6 * 448) of x [N, K] or of each matrix of x [G, N, K]; fp32 [1] or [G]."""
    dim = 3 if isinstance(x, torch.Tensor) and x.dim() == 3 else 2
    dt = _floats(x, "x", dim)
    index, n = x.get_device(), x.numel()
    if n == 0:
        raise ValueError(f"x is empty: {tuple(x.shape)}")
    if _elsewhere(index, stream):
        with _On(index, stream):
            return fp4_scale(x)
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
    dim = 2 if groups is not None or not isinstance(x, torch.Tensor) or x.dim() != 3 else 3
    dt = _floats(x, "x", dim)
    index, K, xp = x.get_device(), x.shape[-1], x.data_ptr()
    if not (K > 0 and K % 32 == 0):
        raise ValueError(f"K must be a multiple of 32, is {K}")
    if xp % 16:
        raise ValueError("x must be 16-byte aligned")
    if not (g is None or wdtype == "nvfp4"):
        raise ValueError("only nvfp4 takes a matrix scale g")
    if groups is not None:
        _groups_on(groups, index)
        if groups.T != x.shape[0]:
            raise ValueError(f"x has {x.shape[0]} rows, groups hold {groups.T} tokens")
        stack, shape = (1, groups.P), (groups.P, K)
        off, til, _, place = groups._ptrs
        rest = (groups.E, groups.k, off, til, place)
    else:
        stack = (x.shape[0], x.shape[1]) if dim == 3 else (1, x.shape[0])
        shape, rest = tuple(x.shape), (0, 0, None, None, None)
    gp = _scale_ptr(g, "g", stack[0], index)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return quantize_fp4(x, wdtype, g=g, groups=groups)
    q = FP4Rows._empty(shape, wdtype, g, gp, groups, stack, x)
    _check(_operators().moe_quantize_fp4(*stack, K, dt, xp, DTYPES[wdtype], *gp, *rest, *q._ptrs[:2], _stream(index)))
    return q


def _rows(q, name):
    if not isinstance(q, FP4Rows):
        raise ValueError(f"{name} must be FP4Rows, is {type(q)}")
    return q


def dequantize_fp4(q, *, out_dtype=torch.bfloat16, stream=None):
    """The values that q stands for, in q.shape; rows that no pair fills are zero (moe_dequantize_fp4)."""
    _rows(q, "q")
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    index = q._index
    if _elsewhere(index, stream):
        with _On(index, stream):
            return dequantize_fp4(q, out_dtype=out_dtype)
    rest = (0, None, None) if q.groups is None else (q.groups.E, *q.groups._ptrs[:2])
    out = torch.empty(q.shape, dtype=out_dtype, device=q.codes.device)
    _check(_operators().moe_dequantize_fp4(*q._stack, q.K, DTYPES[q.wdtype], *q._ptrs, *rest, _FLOATS[out_dtype],
                                           out.data_ptr(), _stream(index)))
    return out


def _columns(groups, E, N, act, out_dtype):
    if groups.E != E:
        raise ValueError(f"w holds {E} experts, groups {groups.E}")
    if act not in ACTS:
        raise ValueError(f"act must be 'none' or 'swiglu', is {act!r}")
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    if not ACTS[act]:
        return N
    if N % 32:
        raise ValueError(f"swiglu needs w rows a multiple of 32, got {N}")
    return N // 2


def grouped_matmul(x, w, groups, *, act="none", gather=False, out_dtype=torch.bfloat16, stream=None):
    """Row i of expert e: x[i] @ w[e].T, w [E, N, K] bf16, x bf16 [P, K] in expert order, or with gather=True
    [T, K] and grouped row i reads x[order[i] // k].  act="swiglu": w holds gate rows, then up rows, and the
    result has N/2 columns.  K a multiple of 8 (moe_grouped_matmul).  Rows that no pair fills are undefined."""
    _typed(w, "w", _BF16, 3)
    index = w.get_device()
    _typed(x, "x", _BF16, 2, index)
    _groups_on(groups, index)
    E, N, K = w.shape
    cols = _columns(groups, E, N, act, out_dtype)
    if not (N > 0 and K > 0 and K % 8 == 0):
        raise ValueError(f"w must be [E, N, K] with K a multiple of 8, is {tuple(w.shape)}")
    rows = groups.T if gather else groups.P
    if x.shape[0] != rows or x.shape[1] != K:
        raise ValueError(f"x must be {(rows, K)}, is {tuple(x.shape)}")
    xp, wp = x.data_ptr(), w.data_ptr()
    if (xp | wp) % 16:
        raise ValueError("x and w must be 16-byte aligned")
    if _elsewhere(index, stream):
        with _On(index, stream):
            return grouped_matmul(x, w, groups, act=act, gather=gather, out_dtype=out_dtype)
    off, til, order, _ = groups._ptrs
    out = torch.empty((groups.P, cols), dtype=out_dtype, device=x.device)
    ops, ws, n = _operators(), None, 0
    if gather:
        n = ops.moe_grouped_matmul_workspace(groups.P, E, K, 1)
        if n:
            ws = torch.empty(n, dtype=_U8, device=x.device)
    _check(ops.moe_grouped_matmul(groups.P, E, N, K, xp, rows, order if gather else None, groups.k, wp, off, til, ACTS[act],
                                  _FLOATS[out_dtype], out.data_ptr(), ws.data_ptr() if n else None, n, _stream(index)))
    return out


def grouped_matmul_fp4(x, w, groups, *, act="none", quantize=False, g_out=None, out_dtype=torch.bfloat16, stream=None):
    """grouped_matmul of 4-bit rows x (FP4Rows in expert order) and 4-bit weights w (FP4Rows [E, N, K]) of one
    format.  quantize=True (act="swiglu" only): the result as FP4Rows of that format with the matrix scale g_out
    [1] (None = 1; "nvfp4" only), rounded from the fp32 values (moe_grouped_matmul_fp4)."""
    _rows(x, "x")
    _rows(w, "w")
    index = w._index
    _groups_on(groups, index)
    if not (len(w.shape) == 3 and w.groups is None):
        raise ValueError(f"w must be [E, N, K], is {w.shape}")
    E, N, K = w.shape
    cols = _columns(groups, E, N, act, out_dtype)
    if not (x.groups is not None and x._index == index and x.groups.E == E and N > 0):
        raise ValueError("x must hold rows in the order of w's experts, on the same device")
    if x.wdtype != w.wdtype:
        raise ValueError(f"x is {x.wdtype}, w is {w.wdtype}")
    if not (x.shape == (groups.P, K)):
        raise ValueError(f"x must be {(groups.P, K)}, is {x.shape}")
    if not (not quantize or (ACTS[act] and cols % 32 == 0)):
        raise ValueError("quantize needs act='swiglu' and w rows a multiple of 64")
    if not (g_out is None or (quantize and x.wdtype == "nvfp4")):
        raise ValueError("g_out goes with quantize=True and nvfp4")
    go = _scale_ptr(g_out, "g_out", 1, index)
    if _elsewhere(index, stream):
        with _On(index, stream):
            return grouped_matmul_fp4(x, w, groups, act=act, quantize=quantize, g_out=g_out, out_dtype=out_dtype)
    if quantize:
        out = FP4Rows._empty((groups.P, cols), x.wdtype, g_out, go, groups, (1, groups.P), x.codes)
        dst = (None, out._ptrs[0], out._ptrs[1], go[0])
    else:
        out = torch.empty((groups.P, cols), dtype=out_dtype, device=x.codes.device)
        dst = (out.data_ptr(), None, None, None)
    _check(_operators().moe_grouped_matmul_fp4(groups.P, E, N, K, DTYPES[x.wdtype], *x._ptrs[:3], *w._ptrs, *groups._ptrs[:2],
                                               ACTS[act], _FLOATS[out_dtype], *dst, _stream(index)))
    return out


def combine(y, groups, topk_w, *, out_dtype=torch.float32, stream=None):
    """out[t] = sum_j topk_w[t, j] * y[place[t, j]], y [P, N] bf16 or fp32 in expert order; pairs dropped from the
    groups contribute nothing (moe_combine)."""
    dt = _floats(y, "y", 2)
    index = y.get_device()
    _groups_on(groups, index)
    _typed(topk_w, "topk_w", _F32, 2, index)
    T, k, N = groups.T, groups.k, y.shape[1]
    if topk_w.shape[0] != T or topk_w.shape[1] != k:
        raise ValueError(f"topk_w must be {(T, k)}, is {tuple(topk_w.shape)}")
    if not (y.shape[0] == groups.P and N > 0):
        raise ValueError(f"y must be [{groups.P}, N], is {tuple(y.shape)}")
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    if _elsewhere(index, stream):
        with _On(index, stream):
            return combine(y, groups, topk_w, out_dtype=out_dtype)
    out = torch.empty((T, N), dtype=out_dtype, device=y.device)
    _check(_operators().moe_combine(T, k, N, dt, y.data_ptr(), groups._ptrs[3], topk_w.data_ptr(), _FLOATS[out_dtype],
                                    out.data_ptr(), _stream(index)))
    return out


def check_operators(stream=None):
    """Synchronise the stream; MoEError if a bounded wait inside an operator kernel ran out since the last check."""
    if stream is None:
        stream = torch.cuda.current_stream()
    _check(_operators().moe_operators_check(getattr(stream, "cuda_stream", stream)))
