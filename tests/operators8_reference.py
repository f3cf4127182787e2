"""The 8-bit operators and the end of a block written out in numpy, 64 bits unless a definition rounds (test infrastructure)."""
from __future__ import annotations

import numpy as np

from oracle.formats import E4M3_TABLE
from tests.operators_reference import combine
from workloads import f32_to_e4m3_codes

LEAST = 2.0 ** -100


def round24(v):
    """Nearest 24-bit value, ties to even, without fp32's limits of the exponent."""
    m, e = np.frexp(v)
    return np.ldexp(np.round(np.ldexp(m, 24)), e - 24)


def _blocks(x, high):
    """Padded with zeros: [row blocks, high, column blocks, 128]."""
    R, K = x.shape
    p = np.zeros((-(-R // high) * high, -(-K // 128) * 128))
    p[:R, :K] = x
    return p.reshape(-1, high, p.shape[1] // 128, 128)


def quantize(x, high):
    """Rows [R, K] in blocks of high x 128 -> codes [R, K] and scales [row blocks, column blocks] (fp32), by the definition's
    correctly rounded steps."""
    x = np.asarray(x, np.float32)
    R, K = x.shape
    b = _blocks(x.astype(np.float64), high)
    bad = ~np.isfinite(b).all(axis=(1, 3))
    b = np.where(bad[:, None, :, None], 0.0, b)
    a = np.maximum(np.abs(b).max(axis=(1, 3)), LEAST)
    q = (round24(448 * b) / a[:, None, :, None]).astype(np.float32)
    codes = f32_to_e4m3_codes(q).reshape(b.shape)
    codes = np.where(bad[:, None, :, None], 0, codes)
    scales = np.where(bad, np.float32(np.nan), a.astype(np.float32) * np.float32(1 / 448))
    return codes.reshape(b.shape[0] * high, -1)[:R, :K].astype(np.uint8), scales.astype(np.float32)


def values(codes, scales, high):
    r, k = np.arange(codes.shape[0]) // high, np.arange(codes.shape[1]) // 128
    return E4M3_TABLE[codes] * scales.astype(np.float64)[r][:, k]


def half_step(v):
    """Half the distance between e4m3 values around |v|."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    return 2.0 ** (e - 4)


def normed(x, weight, eps):
    return x / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps) * weight


def block_end(y, place, w, residual, shared=None, post=None, gate=None, scale=1.0, pre=None, eps=1e-6):
    """(h, z) in 64 bits, and for each how large its parts are before they are added."""
    c = np.zeros(residual.shape) if y is None else y.astype(np.float64) if place is None else combine(y.astype(np.float64), place, w.astype(np.float64))
    mag = np.zeros(residual.shape) if y is None else np.abs(c) if place is None else combine(np.abs(y.astype(np.float64)), place, np.abs(w).astype(np.float64))
    if shared is not None:
        c, mag = c + shared, mag + np.abs(shared)
    if post is not None:
        inv = 1 / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps)
        c, mag = c * inv * post, mag * inv * np.abs(post)
    if gate is not None:
        c, mag = c * gate, mag * np.abs(gate)
    h = scale * residual + c
    mag = mag + np.abs(scale * residual)
    if pre is None:
        return h, None, mag, None
    inv = 1 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return h, h * inv * pre, mag, mag * inv * np.abs(pre)
