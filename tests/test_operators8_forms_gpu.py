"""Each form of the 8-bit products where a unit takes several tiles of several slices: pairs of CTAs, and single ones of every tile.

What only shows from a unit's second tile on: the carry of the ring, the accumulators and the groups of scales from one tile to the next, the
boxes that TMA stores under the next tile's products, and the turns in which two warps exchange their rows' maxima.  The form
that a call runs is asked of the library, so that a rule that moves past a case fails its test."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_operators8_gpu import check_quantized, operands, product, swiglu_within, whole
from tests.test_operators_gpu import bf16, dev, host
from tests.test_operators_many_items_gpu import grouping

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import serving_layer_moe_gb300 as m
    return m


def form(P, E, N, K, act="none", quant=False):
    """(CTAs a tile, weight rows of a tile, stages, accumulators, SMs)."""
    from serving_layer_moe_gb300.operators import _operators
    out, sms = (ctypes.c_int32 * 4)(), torch.cuda.get_device_properties(0).multi_processor_count
    _operators().moe_product8_form(P, E, N, K, int(act == "swiglu"), int(quant), sms, out)
    return (*out, sms)


def tiles(counts, N, rows, tile=256):
    return sum(-(-c // rows) for c in counts) * -(-N // tile)


def near(rng, E, lo, hi):
    """lo to hi rows an expert, on both sides of whole tiles and of a warp's 32 rows, one expert without rows and one with a few."""
    counts = rng.integers(lo, hi + 1, E)
    counts[:4] = hi - hi % 256, hi - hi % 256 + 1, hi - hi % 32, hi - hi % 32 + 31
    return [0, 33, *counts.tolist()]


# rows an expert, experts (and two more with few rows), N, K: several tiles a pair of several slices each
PLAIN_PAIRS = {"whole_rows": (860, 1100, 10, 1920, 1040), "odd_rows": (860, 1100, 10, 1901, 1040), "rows_of_fp32_whole": (860, 1100, 10, 1892, 1296),
               "short_K": (470, 700, 16, 2048, 400), "one_slice": (470, 700, 16, 1800, 112), "eight_slices": (860, 1100, 10, 1288, 2000)}


@pytest.mark.parametrize("name", PLAIN_PAIRS)
def test_pairs(moe, name):
    lo, hi, E, N, K = PLAIN_PAIRS[name]
    rng = np.random.default_rng(N + K)
    counts = near(rng, E, lo, hi)
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    ctas, _, _, _, sms = form(P, E, N, K)
    assert ctas == 2 and tiles(counts, N, 256) >= 3 * (sms // 2)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    y = product(xc, xs, wc, ws, offsets)
    x, w = operands(moe, xc, xs, wc, ws)
    assert np.array_equal(host(moe.grouped_matmul_fp8(x, w, gr, out_dtype=torch.float32)), y)
    assert np.array_equal(host(moe.grouped_matmul_fp8(x, w, gr)), bf16(y))
    moe.check_operators()


# cols = N / 2 of 960: seven tiles of 128 features and one of 64
SWIGLU_PAIRS = {"K_400": (1880, 2300, 8, 1920, 400), "K_1040": (1880, 2300, 8, 1920, 1040), "whole_tiles": (1880, 2300, 8, 2048, 272), "long_K": (850, 1000, 10, 1920, 4112),
                "one_expert": (1 << 14, 1 << 14, 0, 1920, 272), "one_slice": (1880, 2300, 8, 1920, 128)}


@pytest.mark.parametrize("name", SWIGLU_PAIRS)
def test_pairs_with_swiglu(moe, name):
    lo, hi, E, N, K = SWIGLU_PAIRS[name]
    rng = np.random.default_rng(N + K)
    counts = near(rng, E, lo, hi) if E else [lo + 77]
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    ctas, _, _, _, sms = form(P, E, N, K, "swiglu")
    assert ctas == 2 and form(P, E, N, K, "swiglu", True)[0] == 2 and tiles(counts, N, 256) >= 3 * (sms // 2)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    xs = xs / 64
    y = product(xc, xs, wc, ws, offsets).astype(np.float64)
    x, w = operands(moe, xc, xs, wc, ws)
    for out in (torch.float32, torch.bfloat16):
        swiglu_within(host(moe.grouped_matmul_fp8(x, w, gr, act="swiglu", out_dtype=out)), y, out)
    q = moe.grouped_matmul_fp8(x, w, gr, act="swiglu", quantize=True)
    check_quantized(q, y)
    for _ in range(4):       # the same bits again
        r = moe.grouped_matmul_fp8(x, w, gr, act="swiglu", quantize=True)
        assert torch.equal(r.codes.view(torch.uint8), q.codes.view(torch.uint8)) and torch.equal(r.scales, q.scales)
    moe.check_operators()


def test_pairs_of_many_experts(moe):
    """As many experts as there may be, most without rows: the table leaves the fewest stages, and pairs take the ones that have some."""
    rng = np.random.default_rng(4096)
    counts = [0] * 4096
    for e, n in ((0, 60000), (17, 8191), (2048, 31), (4095, 257)):
        counts[e] = n
    N, K = 256, 400
    used = np.array(counts) > 0
    P = sum(counts) + 384 * 4096           # pairs without an expert, behind the last one's rows
    ids = np.repeat(np.arange(4097), [*counts, 384 * 4096]).astype(np.int32)[:, None]
    rng.shuffle(ids)
    gr = moe.group_pairs(dev(ids), 4096)
    ctas, _, stages, accs, _ = form(P, 4096, N, K)
    assert ctas == 2 and stages < accs + 2
    xc, xs, few, scales = whole(rng, sum(counts), int(used.sum()), N, K)
    y = product(xc, xs, few, scales, np.concatenate([[0], np.cumsum(np.array(counts)[used])]))
    wc, ws = np.zeros((4096, *few.shape[1:]), np.uint8), np.ones((4096, *scales.shape[1:]), scales.dtype)
    wc[used], ws[used] = few, scales
    xc, xs = np.pad(xc.astype(np.uint8), ((0, P - len(xc)), (0, 0))), np.pad(xs, ((0, 0), (0, P - xs.shape[1])), constant_values=1)
    x, w = operands(moe, xc, xs, wc, ws)
    got = moe.grouped_matmul_fp8(x, w, gr, out_dtype=torch.float32)
    assert np.array_equal(host(got[:len(y)]), y)
    moe.check_operators()


# one matrix or few experts, rows of each, N, K, the tile's weight rows
FEW_TILES = [([1], 640, 2000, 64), ([70], 300, 1296, 64), ([2, 5, 0, 9], 1000, 1040, 64), ([1], 12000, 400, 128), ([128, 1], 3000, 656, 64), ([300, 128], 3200, 272, 128), ([1], 24000, 272, 256),
             ([400, 3], 5000, 1040, 256)]


@pytest.mark.parametrize("counts,N,K,tile", FEW_TILES)
def test_single_ctas_of_every_tile(moe, counts, N, K, tile):
    """Few tiles: 64, 128 and 256 weight rows each, results without SwiGLU and with it."""
    rng = np.random.default_rng(N + K)
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    assert form(P, E, N, K)[:2] == (1, tile)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    x, w = operands(moe, xc, xs, wc, ws)
    y = product(xc, xs, wc, ws, offsets)
    for out in (torch.float32, torch.bfloat16):
        assert np.array_equal(host(moe.grouped_matmul_fp8(x, w, gr, out_dtype=out)), y if out == torch.float32 else bf16(y))
    N -= N % 128
    if form(P, E, N, K, "swiglu")[:2] == (1, tile):
        xc, xs, wc, ws = whole(rng, P, E, N, K)
        xs = xs / 64
        x, w = operands(moe, xc, xs, wc, ws)
        y = product(xc, xs, wc, ws, offsets).astype(np.float64)
        for out in (torch.float32, torch.bfloat16):
            swiglu_within(host(moe.grouped_matmul_fp8(x, w, gr, act="swiglu", out_dtype=out)), y, out)
        check_quantized(moe.grouped_matmul_fp8(x, w, gr, act="swiglu", quantize=True), y)
    moe.check_operators()
