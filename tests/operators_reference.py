"""The routed-expert operators written out in numpy, 64 bits unless a definition rounds (test infrastructure)."""
from __future__ import annotations

import numpy as np

from oracle.formats import E2M1_TABLE, E4M3_TABLE, e8m0_codes_to_f64
from workloads import f32_to_e2m1_codes, f32_to_e4m3_codes

BLOCK = {"nvfp4": 16, "mxfp4": 32}


def route(logits, k, scoring="softmax", bias=None, n_group=1, topk_group=1, renorm=True, scale=1.0):
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    ids = np.empty((T, k), np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        l = np.where(np.isposinf(z[t]), float(np.finfo(np.float32).max), z[t])
        nan = np.isnan(l)
        if scoring == "softmax":
            live = ~nan & ~np.isneginf(l)
            p = np.zeros(E)
            if live.any():
                p[live] = np.exp(l[live] - l[live].max())
            pick = l.copy()
        else:
            with np.errstate(over="ignore"):
                p = np.where(nan, 0.0, 1 / (1 + np.exp(-np.where(nan, 0, l))))
            pick = p + (0 if bias is None else np.asarray(bias, np.float64))
        pick = np.where(nan, -np.inf, pick)
        rank = np.where(nan, -1, 0)          # NaN below -inf
        alive = np.ones(E, bool)
        if n_group > 1:
            gs = E // n_group
            score = [np.sort(pick[g * gs:(g + 1) * gs])[::-1][:2].sum() for g in range(n_group)]
            best = sorted(range(n_group), key=lambda g: (-score[g], g))[:topk_group]
            alive = np.isin(np.arange(E) // gs, best)
        order = sorted(np.flatnonzero(alive), key=lambda e: (-rank[e], -pick[e], e))[:k]
        ids[t] = order
        w[t] = p[order]
        if renorm or scoring == "softmax":
            d = w[t].sum() if renorm else p.sum()
            w[t] = w[t] / d if d > 0 else 0.0
    return ids, w * scale


def groups(ids, E):
    flat = np.asarray(ids).reshape(-1)
    order, offsets, tiles = [], [0], [0]
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        order += mine.tolist()
        offsets.append(offsets[-1] + mine.size)
        tiles.append(tiles[-1] + -(-mine.size // 128))
    place = np.full(flat.size, -1)
    place[order] = np.arange(len(order))
    order += [-1] * (flat.size - len(order))
    return np.array(offsets), np.array(tiles), np.array(order, np.int64), place.reshape(np.shape(ids))


def quantize(x, wdtype, g=1.0):
    """Rows [R, K] float32, g scalar or [R] -> codes [R, K] and scale codes [R, K / block], by the definition's
    correctly rounded 32-bit steps."""
    x = np.asarray(x, np.float32)
    R, K = x.shape
    B = BLOCK[wdtype]
    xb = x.reshape(R, K // B, B)
    g = np.broadcast_to(np.asarray(g, np.float32).reshape(-1, 1), (R, 1))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        nan = np.isnan(xb).any(axis=2)
        amax = np.where(nan, np.float32(0), np.abs(np.where(np.isnan(xb), np.float32(0), xb)).max(axis=2))
        if wdtype == "nvfp4":
            t = (amax * np.float32(1 / 6) / g).astype(np.float32)
            sc = f32_to_e4m3_codes(np.minimum(t, np.float32(448)))
            step = (E4M3_TABLE[sc].astype(np.float32) * g).astype(np.float32)
            m = np.where(step[:, :, None] > 0, xb / np.where(step > 0, step, np.float32(1))[:, :, None], np.float32(0))
            sc = np.where(nan, 0x7F, sc)
        else:
            ex = np.where(np.isinf(amax), 128, np.frexp(np.where(np.isinf(amax), 1, amax))[1] - 1)
            X = np.where(amax > 0, np.clip(ex - 2, -127, 127), 0)
            m = (xb.astype(np.float64) * np.ldexp(1.0, -X)[:, :, None]).astype(np.float32)
            sc = np.where(nan, 255, X + 127)
        codes = f32_to_e2m1_codes(np.where(nan[:, :, None], np.float32(0), m))
    return codes.reshape(R, K), sc.astype(np.uint8)


def values(codes, sc, wdtype, g=1.0):
    B = BLOCK[wdtype]
    s = E4M3_TABLE[sc] if wdtype == "nvfp4" else e8m0_codes_to_f64(sc)
    g = np.asarray(g, np.float64).reshape(-1, 1)
    return E2M1_TABLE[codes] * np.repeat(s * g, B, axis=1)


def unpack(packed):
    p = np.asarray(packed)
    out = np.empty((p.shape[0], p.shape[1] * 2), np.uint8)
    out[:, 0::2], out[:, 1::2] = p & 15, p >> 4
    return out


def untile(tiles, rows, blocks):
    """Scale tiles [n, groups, 512] -> scales of padded rows `rows`, [len(rows), blocks]."""
    t = np.asarray(tiles)
    r, b = np.asarray(rows)[:, None], np.arange(blocks)[None, :]
    return t[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def tile(sc, rows, n_tiles):
    """Scales [R, blocks] of padded rows `rows` -> scale tiles, padding 0."""
    sc = np.asarray(sc)
    ng = -(-sc.shape[1] // 4)
    out = np.zeros((n_tiles, ng, 512), np.uint8)
    r, b = np.asarray(rows)[:, None], np.arange(sc.shape[1])[None, :]
    out[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = sc
    return out


def padded_rows(offsets, tiles):
    return np.concatenate([128 * t + np.arange(b - a) for a, b, t in zip(offsets, offsets[1:], tiles)] or [np.empty(0, int)]).astype(np.int64)


def product(x, w, offsets):
    """(x [P, K] times w[e].T, the sum of absolute products): 64 bits."""
    y = np.zeros((x.shape[0], w.shape[1]))
    mag = np.zeros_like(y)
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        y[a:b] = x[a:b] @ w[e].T
        mag[a:b] = np.abs(x[a:b]) @ np.abs(w[e]).T
    return y, mag


def swiglu(y):
    n = y.shape[1] // 2
    with np.errstate(over="ignore"):
        return y[:, :n] / (1 + np.exp(-y[:, :n])) * y[:, n:]


def combine(y, place, w):
    out = np.zeros((place.shape[0], y.shape[1]))
    for t in range(place.shape[0]):
        for j in range(place.shape[1]):
            if place[t, j] >= 0:
                out[t] += w[t, j] * y[place[t, j]]
    return out
