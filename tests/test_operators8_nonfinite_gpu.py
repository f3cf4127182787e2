"""Blocks of a requantised 8-bit result that hold a NaN or an infinity: scale NaN and codes 0, as the quantiser has them, and no other block changed."""
import numpy as np
import pytest
import torch

from tests.test_operators8_gpu import codes_of, operands, whole
from tests.test_operators_gpu import host
from tests.test_operators_many_items_gpu import grouping

pytestmark = pytest.mark.gpu
N, K = 640, 272                     # two blocks of 128 features and one of 64: a tile's two halves, and a tile that has one half only


@pytest.fixture(scope="module")
def moe():
    import serving_layer_moe_gb300 as m
    return m


def poison(kind, xc, xs, wc, ws):
    """Changes the operands; returns the blocks [P, 3] that are not finite any more, as a function of (row, its expert)."""
    n = N // 2
    if kind == "first_half":         # an up row's code
        wc[0, n + 3, 5] = 0x7F
        return lambda i, e: [e == 0, False, False]
    if kind == "second_half":        # a gate row's
        wc[-1, 200, 271] = 0xFF
        return lambda i, e: [False, e == wc.shape[0] - 1, False]
    if kind == "last_half":
        wc[0, 300, 0] = 0x7F
        return lambda i, e: [False, False, e == 0]
    if kind == "row_nan":
        xc[3, 200] = 0x7F
        return lambda i, e: [i == 3] * 3
    if kind == "row_infinite":       # sums of infinities, or NaN
        xs[1, 4] = np.inf
        return lambda i, e: [i == 4] * 3
    xs[:, 2] *= 2.0 ** 80            # gates and ups are finite, the products with positive gates are past 2^128
    return lambda i, e: [i == 2] * 3


@pytest.mark.parametrize("kind", ["first_half", "second_half", "last_half", "row_nan", "row_infinite", "row_overflows"])
@pytest.mark.parametrize("counts", [[40, 0, 5, 30], [1700]])
def test_blocks_that_are_not_finite(moe, counts, kind):
    """Single CTAs, and pairs of them (one expert's rows)."""
    rng = np.random.default_rng(len(counts))
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    xs = xs / 8
    call = lambda **kw: moe.grouped_matmul_fp8(*operands(moe, xc, xs, wc, ws), gr, act="swiglu", **kw)  # noqa: E731
    clean = call(quantize=True)
    expert = np.searchsorted(offsets[1:], np.arange(P), side="right")
    where = poison(kind, xc, xs, wc, ws)
    bad = np.array([where(i, e) for i, e in enumerate(expert)])
    assert bad.any() and not bad.all() or E == 1
    got, h = call(quantize=True), host(call(out_dtype=torch.float32))
    assert np.array_equal(np.add.reduceat(~np.isfinite(h), [0, 128, 256], axis=1) > 0, bad)
    codes, scales, wide = codes_of(got), host(got.scales).T, np.repeat(bad, 128, axis=1)[:, :N // 2]
    assert np.isnan(scales[bad]).all() and np.array_equal(scales[~bad], host(clean.scales).T[~bad])
    assert not codes[wide].any(), np.unique(codes[wide])
    assert np.array_equal(codes[~wide], codes_of(clean)[~wide])
    same = moe.quantize_fp8(torch.from_numpy(h).cuda())
    assert np.array_equal(codes_of(same)[wide], codes[wide]) and np.array_equal(np.isnan(host(same.scales).T), bad)
