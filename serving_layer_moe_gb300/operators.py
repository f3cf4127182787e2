"""The operators around a cache of experts, on torch tensors (libmoecache.so, include/moe_operators.h).

    ids, w, groups = route(logits, top_k, groups=True)     # router, pairs in expert order
    xq = quantize_fp4(x, "nvfp4", g=gx, groups=groups)     # rows gathered by expert, 4-bit
    h = grouped_matmul_fp4(xq, gate_up, groups, act="swiglu", quantize=True, g_out=gh)
    y = grouped_matmul_fp4(h, down, groups)
    out = combine(y, groups, w)

Argument checks, output tensors and pointers only: the work is in the library's kernels, there is no
fallback.  Everything is enqueued on `stream` (torch's current stream if None); outputs are allocated for
that stream.  Wrong arguments raise ValueError before anything is enqueued.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import DTYPES, _check, load_library

OPERATOR_SYMBOLS = ("moe_grouped_tiles", "moe_group_workspace", "moe_route", "moe_group_pairs", "moe_fp4_scale",
                    "moe_quantize_fp4", "moe_dequantize_fp4", "moe_grouped_matmul", "moe_grouped_matmul_fp4",
                    "moe_combine", "moe_operators_check")

SCORING = {"softmax": 0, "sigmoid": 1}
ACTS = {None: 0, "none": 0, "swiglu": 1}
FP4_BLOCK = {"nvfp4": 16, "mxfp4": 32}
_FLOATS = {torch.float32: DTYPES["f32"], torch.bfloat16: DTYPES["bf16"]}

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
            "moe_grouped_matmul": [I32, I32, I32, I32, P, I32, P, I32, P, P, P, I32, I32, P, P],
            "moe_grouped_matmul_fp4": [I32, I32, I32, I32, I32, P, P, P, P, P, P, I32, P, P, I32, I32, P, P, P, P, P],
            "moe_combine": [I32, I32, I32, I32, P, P, P, I32, P, P],
            "moe_operators_check": [P],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int64 if name in ("moe_grouped_tiles", "moe_group_workspace") else ctypes.c_int
        _lib = lib
    return _lib


class _On:
    """The device and stream that a call runs on, with both current inside the block."""

    __slots__ = ("handle", "_ctx")

    def __init__(self, device, stream):
        self._ctx = []
        if device.index is not None and device.index != torch.cuda.current_device():
            self._ctx.append(torch.cuda.device(device))
        if stream is None:
            self.handle = None
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)
            self._ctx.append(torch.cuda.stream(stream))
            self.handle = stream.cuda_stream

    def __enter__(self):
        for c in self._ctx:
            c.__enter__()
        if self.handle is None:
            self.handle = torch.cuda.current_stream().cuda_stream
        return self.handle

    def __exit__(self, *exc):
        for c in reversed(self._ctx):
            c.__exit__(*exc)
        return False


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _tensor(t, name, dtypes, dim, device=None):
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.dim() != dim or not t.is_contiguous():
        got = f"{t.dtype} {tuple(t.shape)}{'' if t.is_contiguous() else ' (not contiguous)'}" if isinstance(t, torch.Tensor) else type(t)
        raise ValueError(f"{name} must be a contiguous {dim}-dimensional tensor of {' or '.join(map(str, dtypes))}, got {got}")
    if device is None:
        _need(t.device.type == "cuda", f"{name} must be on a CUDA device, is on {t.device}")
    else:
        _need(t.device == device, f"{name} is on {t.device}, the other arguments on {device}")
    return t


def _scale_arg(g, name, counts, device):
    if g is None:
        return None, 0
    _tensor(g, name, (torch.float32,), 1, device)
    _need(g.numel() in counts, f"{name} must hold {' or '.join(map(str, sorted(set(counts))))} values, holds {g.numel()}")
    return g.data_ptr(), g.numel()


_I32 = (torch.int32,)


class ExpertGroups:
    """The (token, expert) pairs of a call in expert order: offsets and tiles [E + 1], order [T * k] and
    place [T, k], all int32 (include/moe_operators.h, "Expert order")."""

    __slots__ = ("offsets", "tiles", "order", "place")

    def __init__(self, offsets, tiles, order, place):
        self.offsets, self.tiles, self.order, self.place = offsets, tiles, order, place

    @property
    def E(self):
        return self.offsets.numel() - 1

    @property
    def P(self):
        return self.order.numel()

    @property
    def k(self):
        return self.place.shape[1]

    def _checked(self, device=None):
        _tensor(self.offsets, "groups.offsets", _I32, 1, device)
        device = self.offsets.device
        _tensor(self.tiles, "groups.tiles", _I32, 1, device)
        _tensor(self.order, "groups.order", _I32, 1, device)
        _tensor(self.place, "groups.place", _I32, 2, device)
        _need(self.offsets.numel() >= 2 and self.tiles.numel() == self.offsets.numel(),
              f"groups.offsets and groups.tiles must hold E + 1 values each, hold {self.offsets.numel()} and {self.tiles.numel()}")
        _need(self.place.numel() == self.order.numel(),
              f"groups.order holds {self.order.numel()} pairs, groups.place {self.place.numel()}")
        return self


class FP4Rows:
    """4-bit matrices: codes uint8 [..., K/2] and scale tiles uint8 [row tiles, block groups, 512]
    (include/moe_operators.h, "4-bit matrices"), wdtype "nvfp4" or "mxfp4", g the fp32 matrix scales (1 or one
    per matrix; None = 1).  groups: of rows in expert order; None for a stack of matrices [G, N, K] or one [N, K]."""

    __slots__ = ("codes", "scales", "wdtype", "g", "groups")

    def __init__(self, codes, scales, wdtype, g=None, groups=None):
        self.codes, self.scales, self.wdtype, self.g, self.groups = codes, scales, wdtype, g, groups

    @property
    def K(self):
        return 2 * self.codes.shape[-1]

    @property
    def shape(self):
        return (*self.codes.shape[:-1], self.K)

    def _checked(self, name, dims, device=None):
        _need(self.wdtype in FP4_BLOCK, f"{name}.wdtype must be 'nvfp4' or 'mxfp4', is {self.wdtype!r}")
        dim = self.codes.dim() if isinstance(self.codes, torch.Tensor) else dims[0]
        _tensor(self.codes, f"{name}.codes", (torch.uint8,), dim if dim in dims else dims[0], device)
        _tensor(self.scales, f"{name}.scales", (torch.uint8,), 3, self.codes.device)
        _need(self.K > 0 and self.K % 32 == 0, f"{name}: K must be a multiple of 32, is {self.K}")
        if self.groups is not None:
            n = _grouped_tiles(self.codes.shape[0], self.groups.E)
        else:
            G, N = self._stack()
            n = G * -(-N // 128)
        want = (n, _block_groups(self.wdtype, self.K), 512)
        _need(tuple(self.scales.shape) == want, f"{name}.scales must be {want}, is {tuple(self.scales.shape)}")
        _need(self.codes.data_ptr() % 16 == 0 and self.scales.data_ptr() % 16 == 0,
              f"{name}: codes and scales must be 16-byte aligned")
        return self

    def _stack(self):
        return (1, self.codes.shape[0]) if self.codes.dim() == 2 else (self.codes.shape[0], self.codes.shape[1])


def _block_groups(wdtype, K):
    return -(-K // (4 * FP4_BLOCK[wdtype]))


def _grouped_tiles(P, E):
    return (P + 127 * min(P, E)) // 128


def _workspace(T, k, E, device):
    n = int(_operators().moe_group_workspace(T, k, E))
    return torch.empty(n, dtype=torch.uint8, device=device), n


def _empty_groups(T, k, E, device):
    e = E + 1
    ints = torch.empty(2 * e + 2 * T * k, dtype=torch.int32, device=device)
    return ExpertGroups(ints[:e], ints[e:2 * e], ints[2 * e:2 * e + T * k], ints[2 * e + T * k:].view(T, k))


def route(logits, top_k, *, scoring="softmax", bias=None, n_group=1, topk_group=1, renormalize=True, scale=1.0,
          groups=False, stream=None):
    """Experts and gates of each token: (topk_ids int32 [T, k], topk_w fp32 [T, k]), or with groups=True also the
    ExpertGroups of the picked pairs.  logits [T, E] fp32 or bf16; scoring "softmax" (by logit) or "sigmoid"
    (with an optional selection bias [E] and topk_group of n_group expert groups): moe_route."""
    _tensor(logits, "logits", tuple(_FLOATS), 2)
    T, E = logits.shape
    k, dev = int(top_k), logits.device
    _need(scoring in SCORING, f"scoring must be 'softmax' or 'sigmoid', is {scoring!r}")
    _need(1 <= E <= 4096 and 1 <= k <= E, f"1 <= top_k <= E <= 4096 is needed, got top_k {k}, E {E}")
    if scoring == "softmax":
        _need(bias is None and n_group == 1, "softmax scoring takes no bias and no expert groups")
    if bias is not None:
        _tensor(bias, "bias", (torch.float32,), 1, dev)
        _need(bias.numel() == E, f"bias must hold E = {E} values, holds {bias.numel()}")
    _need(1 <= n_group <= 32 and E % n_group == 0 and 1 <= topk_group <= n_group and topk_group * (E // n_group) >= k,
          f"n_group (1 to 32) must divide E and topk_group groups must hold top_k experts, got n_group {n_group}, "
          f"topk_group {topk_group}, E {E}, top_k {k}")
    with _On(dev, stream) as s:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        w = torch.empty((T, k), dtype=torch.float32, device=dev)
        gr, ws, n = None, None, 0
        if groups:
            gr = _empty_groups(T, k, E, dev)
            ws, n = _workspace(T, k, E, dev)
        _check(_operators().moe_route(
            T, E, k, _FLOATS[logits.dtype], logits.data_ptr(), SCORING[scoring],
            None if bias is None else bias.data_ptr(), n_group, topk_group, 1 if renormalize else 0, scale,
            ids.data_ptr(), w.data_ptr(), *((gr.offsets.data_ptr(), gr.tiles.data_ptr(), gr.order.data_ptr(),
                                            gr.place.data_ptr(), ws.data_ptr()) if groups else (None,) * 5), n, s))
    return (ids, w, gr) if groups else (ids, w)


def group_pairs(topk_ids, n_experts, *, stream=None):
    """ExpertGroups of topk_ids int32 [T, k]; pairs whose id is outside [0, n_experts) are dropped (place -1)."""
    _tensor(topk_ids, "topk_ids", _I32, 2)
    T, k = topk_ids.shape
    E, dev = int(n_experts), topk_ids.device
    _need(1 <= E <= 4096 and k >= 1, f"1 <= n_experts <= 4096 and k >= 1 are needed, got {E} and {k}")
    with _On(dev, stream) as s:
        gr = _empty_groups(T, k, E, dev)
        ws, n = _workspace(T, k, E, dev)
        _check(_operators().moe_group_pairs(T, E, k, topk_ids.data_ptr(), gr.offsets.data_ptr(), gr.tiles.data_ptr(),
                                            gr.order.data_ptr(), gr.place.data_ptr(), ws.data_ptr(), n, s))
    return gr


def fp4_scale(x, *, stream=None):
    """NVFP4 matrix scales: max |x| / (6 * 448) of x [N, K] or of each matrix of x [G, N, K]; fp32 [1] or [G]."""
    dim = 3 if isinstance(x, torch.Tensor) and x.dim() == 3 else 2
    _tensor(x, "x", tuple(_FLOATS), dim)
    _need(x.numel() > 0, f"x is empty: {tuple(x.shape)}")
    G = x.shape[0] if dim == 3 else 1
    with _On(x.device, stream) as s:
        g = torch.empty(G, dtype=torch.float32, device=x.device)
        _check(_operators().moe_fp4_scale(G, x.numel() // G, _FLOATS[x.dtype], x.data_ptr(), g.data_ptr(), s))
    return g


def quantize_fp4(x, wdtype, *, g=None, groups=None, stream=None):
    """x in 4 bits (moe_quantize_fp4).  Without groups: x [N, K] or a stack [G, N, K], g fp32 [1] or [G].  With
    groups: x [T, K], and the result holds row order[i] // k of x at grouped row i.  K a multiple of 32; g only
    for "nvfp4" (None = 1)."""
    _need(wdtype in FP4_BLOCK, f"wdtype must be 'nvfp4' or 'mxfp4', is {wdtype!r}")
    dim = 2 if groups is not None or not isinstance(x, torch.Tensor) or x.dim() != 3 else 3
    _tensor(x, "x", tuple(_FLOATS), dim)
    dev, K = x.device, x.shape[-1]
    _need(K > 0 and K % 32 == 0, f"K must be a multiple of 32, is {K}")
    _need(x.data_ptr() % 16 == 0, "x must be 16-byte aligned")
    _need(g is None or wdtype == "nvfp4", "only nvfp4 takes a matrix scale g")
    G, N = (x.shape[0], x.shape[1]) if dim == 3 else (1, x.shape[0])
    gp, gn = _scale_arg(g, "g", (1, G), dev)
    if groups is not None:
        groups._checked(dev)
        _need(groups.place.shape[0] == N, f"x has {N} rows, groups hold {groups.place.shape[0]} tokens")
        N = groups.P
        nt, shape = _grouped_tiles(N, groups.E), (N, K // 2)
    else:
        nt, shape = G * -(-N // 128), (*x.shape[:-1], K // 2)
    with _On(dev, stream) as s:
        codes = torch.empty(shape, dtype=torch.uint8, device=dev)
        scales = torch.empty((nt, _block_groups(wdtype, K), 512), dtype=torch.uint8, device=dev)
        if groups is None:
            rest = (0, 0, None, None, None)
        else:
            rest = (groups.E, groups.k, groups.offsets.data_ptr(), groups.tiles.data_ptr(), groups.order.data_ptr())
        _check(_operators().moe_quantize_fp4(G, N, K, _FLOATS[x.dtype], x.data_ptr(), DTYPES[wdtype], gp, gn, *rest,
                                             codes.data_ptr(), scales.data_ptr(), s))
    return FP4Rows(codes, scales, wdtype, g, groups)


def dequantize_fp4(q, *, out_dtype=torch.bfloat16, stream=None):
    """The values that q stands for, in q.shape; rows that no pair fills are zero (moe_dequantize_fp4)."""
    _need(isinstance(q, FP4Rows), f"q must be FP4Rows, is {type(q)}")
    q._checked("q", (2,) if q.groups is not None else (2, 3))
    _need(out_dtype in _FLOATS, f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    dev = q.codes.device
    G, N = q._stack()
    gp, gn = _scale_arg(q.g, "q.g", (1, G), dev)
    rest = (0, None, None)
    if q.groups is not None:
        q.groups._checked(dev)
        _need(q.groups.P == N, f"q has {N} rows, its groups hold {q.groups.P} pairs")
        rest = (q.groups.E, q.groups.offsets.data_ptr(), q.groups.tiles.data_ptr())
    with _On(dev, stream) as s:
        out = torch.empty(q.shape, dtype=out_dtype, device=dev)
        _check(_operators().moe_dequantize_fp4(G, N, q.K, DTYPES[q.wdtype], q.codes.data_ptr(), q.scales.data_ptr(),
                                               gp, gn, *rest, _FLOATS[out_dtype], out.data_ptr(), s))
    return out


def _product_args(groups, E, N, act, out_dtype, dev):
    _need(isinstance(groups, ExpertGroups), f"groups must be ExpertGroups, is {type(groups)}")
    groups._checked(dev)
    _need(groups.E == E, f"w holds {E} experts, groups {groups.E}")
    _need(act in ACTS, f"act must be 'none' or 'swiglu', is {act!r}")
    _need(out_dtype in _FLOATS, f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    if ACTS[act]:
        _need(N % 32 == 0, f"swiglu needs w rows a multiple of 32, got {N}")
        return N // 2
    return N


def grouped_matmul(x, w, groups, *, act="none", gather=False, out_dtype=torch.bfloat16, stream=None):
    """Row i of expert e: x[i] @ w[e].T, w [E, N, K] bf16, x bf16 [P, K] in expert order, or with gather=True
    [T, K] and grouped row i reads x[order[i] // k].  act="swiglu": w holds gate rows, then up rows, and the
    result has N/2 columns.  K a multiple of 8 (moe_grouped_matmul).  Rows that no pair fills are undefined."""
    _tensor(x, "x", (torch.bfloat16,), 2)
    dev = x.device
    _tensor(w, "w", (torch.bfloat16,), 3, dev)
    E, N, K = w.shape
    cols = _product_args(groups, E, N, act, out_dtype, dev)
    _need(N > 0 and K > 0 and K % 8 == 0, f"w must be [E, N, K] with K a multiple of 8, is {tuple(w.shape)}")
    rows = groups.place.shape[0] if gather else groups.P
    _need(tuple(x.shape) == (rows, K), f"x must be {(rows, K)}, is {tuple(x.shape)}")
    _need(x.data_ptr() % 16 == 0 and w.data_ptr() % 16 == 0, "x and w must be 16-byte aligned")
    with _On(dev, stream) as s:
        out = torch.empty((groups.P, cols), dtype=out_dtype, device=dev)
        _check(_operators().moe_grouped_matmul(
            groups.P, E, N, K, x.data_ptr(), rows, groups.order.data_ptr() if gather else None, groups.k, w.data_ptr(),
            groups.offsets.data_ptr(), groups.tiles.data_ptr(), ACTS[act], _FLOATS[out_dtype], out.data_ptr(), s))
    return out


def grouped_matmul_fp4(x, w, groups, *, act="none", quantize=False, g_out=None, out_dtype=torch.bfloat16, stream=None):
    """grouped_matmul of 4-bit rows x (FP4Rows in expert order) and 4-bit weights w (FP4Rows [E, N, K]) of one
    format.  quantize=True (act="swiglu" only): the result as FP4Rows of that format with the matrix scale g_out
    [1] (None = 1; "nvfp4" only), rounded from the fp32 values (moe_grouped_matmul_fp4)."""
    _need(isinstance(x, FP4Rows) and isinstance(w, FP4Rows), "x and w must be FP4Rows")
    w._checked("w", (3,))
    dev = w.codes.device
    E, N, K = w.shape
    cols = _product_args(groups, E, N, act, out_dtype, dev)
    _need(x.groups is not None and x.groups.E == E and N > 0, "x must hold rows in the expert order of w's experts")
    x._checked("x", (2,), dev)
    _need(x.wdtype == w.wdtype, f"x is {x.wdtype}, w is {w.wdtype}")
    _need(x.shape == (groups.P, K), f"x must be {(groups.P, K)}, is {x.shape}")
    _need(not quantize or (ACTS[act] and cols % 32 == 0), "quantize needs act='swiglu' and w rows a multiple of 64")
    _need(g_out is None or (quantize and x.wdtype == "nvfp4"), "g_out goes with quantize=True and nvfp4")
    gx, _ = _scale_arg(x.g, "x.g", (1,), dev)
    gw, gwn = _scale_arg(w.g, "w.g", (1, E), dev)
    go, _ = _scale_arg(g_out, "g_out", (1,), dev)
    with _On(dev, stream) as s:
        if quantize:
            out, op = None, None
            codes = torch.empty((groups.P, cols // 2), dtype=torch.uint8, device=dev)
            scales = torch.empty((_grouped_tiles(groups.P, E), _block_groups(x.wdtype, cols), 512), dtype=torch.uint8, device=dev)
            cp, sp = codes.data_ptr(), scales.data_ptr()
        else:
            out = torch.empty((groups.P, cols), dtype=out_dtype, device=dev)
            op, cp, sp = out.data_ptr(), None, None
        _check(_operators().moe_grouped_matmul_fp4(
            groups.P, E, N, K, DTYPES[x.wdtype], x.codes.data_ptr(), x.scales.data_ptr(), gx, w.codes.data_ptr(),
            w.scales.data_ptr(), gw, gwn, groups.offsets.data_ptr(), groups.tiles.data_ptr(), ACTS[act],
            _FLOATS[out_dtype], op, cp, sp, go, s))
    return FP4Rows(codes, scales, x.wdtype, g_out, groups) if quantize else out


def combine(y, groups, topk_w, *, out_dtype=torch.float32, stream=None):
    """out[t] = sum_j topk_w[t, j] * y[place[t, j]], y [P, N] bf16 or fp32 in expert order; pairs dropped from the
    groups contribute nothing (moe_combine)."""
    _tensor(y, "y", tuple(_FLOATS), 2)
    dev, N = y.device, y.shape[1]
    _need(isinstance(groups, ExpertGroups), f"groups must be ExpertGroups, is {type(groups)}")
    groups._checked(dev)
    _tensor(topk_w, "topk_w", (torch.float32,), 2, dev)
    _need(topk_w.shape == groups.place.shape, f"topk_w must be {tuple(groups.place.shape)}, is {tuple(topk_w.shape)}")
    _need(y.shape[0] == groups.P and N > 0, f"y must be [{groups.P}, N], is {tuple(y.shape)}")
    _need(out_dtype in _FLOATS, f"out_dtype must be float32 or bfloat16, is {out_dtype}")
    T, k = topk_w.shape
    with _On(dev, stream) as s:
        out = torch.empty((T, N), dtype=out_dtype, device=dev)
        _check(_operators().moe_combine(T, k, N, _FLOATS[y.dtype], y.data_ptr(), groups.place.data_ptr(),
                                        topk_w.data_ptr(), _FLOATS[out_dtype], out.data_ptr(), s))
    return out


def check_operators(stream=None):
    """Synchronise the stream; MoEError if a bounded wait inside an operator kernel ran out since the last check."""
    if stream is None:
        stream = torch.cuda.current_stream()
    _check(_operators().moe_operators_check(getattr(stream, "cuda_stream", stream)))
