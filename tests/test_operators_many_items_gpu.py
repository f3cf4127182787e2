"""Products of many experts and many tiles, so that every unit of the persistent kernels takes several in turn.

What only shows from the second tile of a unit on: the carry of the ring, the accumulators and the scale slots from one tile to
the next, the schedules, and the search over many experts.  Operands are small whole or half numbers: all partial sums
are exact in the accumulators, so results without SwiGLU are compared bit for bit.
"""
import numpy as np
import pytest
import torch

from tests import operators_reference as ref
from tests.test_operators_gpu import BF16, EPS, bf16, dev, host, make_ids

pytestmark = pytest.mark.gpu

# rows an expert, on both sides of 16, 32, 64, 128, 192 and 256
EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 160, 191, 192, 193, 224, 255, 256, 257, 300, 511, 513, 0]


@pytest.fixture(scope="module")
def moe():
    import serving_layer_moe_gb300 as m
    return m


def many(rng, E):
    """Prompt-sized: the edges and 60 to 139 rows for the other experts, in any order."""
    return rng.permutation(EDGES + list(rng.integers(60, 140, E - len(EDGES)))).tolist()


def few(rng, E, most):
    """Decode-sized: 0 to `most` rows an expert."""
    return rng.integers(0, most + 1, E).tolist()


def items(counts, cols, act, pairs):
    """Tiles of the call: token tiles times weight blocks."""
    rows, block = (256, 128 if act else 256) if pairs else (128, 64 if act else 128)
    return sum(-(-c // rows) for c in counts) * -(-cols // block)


def enough(counts, cols, act, pairs):
    """At least three tiles for each unit that a GPU can have: CTAs, or pairs of them."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, units = items(counts, cols, act, pairs), sms // 2 if pairs else sms
    assert n >= 3 * units, (n, units)


def grouping(moe, rng, counts, k=1):
    P, E = sum(counts), len(counts)
    while P % k:
        k -= 1
    ids = make_ids(rng, counts, P // k, k)
    return moe.group_pairs(dev(ids), E), ref.groups(ids, E), P, E, k


def swiglu(y):
    """SwiGLU of exact y, and how far two approximate functions (2 units each), an exponent rounded by |gate| units
    and six further roundings may take it; a unit is 2^-23."""
    h = ref.swiglu(y)
    return h, (np.abs(y[:, :y.shape[1] // 2]) + 10) * 2 * EPS * np.abs(h)


def same_or_within(got, y, act, out):
    """bf16: the rounded value, or with SwiGLU a half unit (relative 2^-8) and the error before it; fp32 without SwiGLU: the value."""
    if not act:
        assert np.array_equal(got, bf16(y) if out == torch.bfloat16 else y.astype(np.float32))
        return
    h, tol = swiglu(y)
    bad = np.abs(got - h) > tol + (BF16 * (np.abs(h) + tol) if out == torch.bfloat16 else EPS * np.abs(h)) + 1e-30
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], h[bad][:5])


# counts, N, K, act, out, gathered, pairs of CTAs (four rows an expert and a bf16 result)
BF16_CASES = {
    "pairs": (many, 70, 4096, 328, "none", torch.bfloat16, False, True),
    "pairs_gathered_swiglu": (many, 40, 4096, 200, "swiglu", torch.bfloat16, True, True),
    "pairs_odd_columns": (many, 60, 3001, 72, "none", torch.bfloat16, True, True),
    "singles": (few, 250, 1000, 136, "none", torch.bfloat16, False, False),
    "singles_gathered_swiglu": (few, 200, 1024, 328, "swiglu", torch.bfloat16, True, False),
    "singles_fp32_runs": (few, 40, 2000, 600, "none", torch.float32, True, False),
    "singles_fp32": (many, 40, 2000, 328, "none", torch.float32, False, False),
    "singles_fp32_swiglu": (many, 40, 2048, 328, "swiglu", torch.float32, True, False),
    "pairs_most_experts": (few, 4096, 1100, 40, "none", torch.bfloat16, False, True),
}


@pytest.mark.parametrize("name", BF16_CASES)
def test_bf16_products_of_many_items(moe, name):
    make, E, N, K, act, out, gather, pairs = BF16_CASES[name]
    rng = np.random.default_rng(len(name) + N)
    counts = make(rng, E) if make is many else few(rng, E, {250: 6, 200: 6, 40: 60, 4096: 10}[E])
    if make is few and E in (250, 200):
        counts = [min(c, 5) if i % 2 else 0 if c < 5 else 1 for i, c in enumerate(counts)]      # below four rows an expert
    gr, (offsets, _, order, _), P, E, k = grouping(moe, rng, counts, 6 if gather else 1)
    assert (P >= 4 * E and out == torch.bfloat16) == pairs
    enough(counts, N // 2 if act == "swiglu" else N, act == "swiglu", pairs)
    x = rng.integers(-2, 3, (P // k if gather else P, K)).astype(np.float32)
    w = rng.integers(-2, 3, (E, N, K)).astype(np.float32)
    if act == "swiglu":
        w *= 0.125                                                 # gates up to about 10
    got = host(moe.grouped_matmul(dev(x, torch.bfloat16), dev(w, torch.bfloat16), gr, act=act, gather=gather, out_dtype=out))
    y, _ = product(x[order // k] if gather else x, w, offsets)
    same_or_within(got.astype(np.float64), y, act == "swiglu", out)
    moe.check_operators()


def product(x, w, offsets):
    """x [P, K] times w[e].T in fp32, which holds these sums exactly."""
    y = np.zeros((x.shape[0], w.shape[1]))
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if b > a:
            y[a:b] = x[a:b] @ w[e].T
    return y, None


def half_numbers(rng, wdtype, R, K):
    """Codes of 0 to 2 with either sign and block scales of 1 and 1/2, and the values they stand for."""
    codes = rng.integers(0, 5, (R, K)).astype(np.uint8) | (rng.integers(0, 2, (R, K)) << 3).astype(np.uint8)
    sc = rng.integers(0, 2, (R, K // ref.BLOCK[wdtype]))
    sc = ((7 - sc) << 3 if wdtype == "nvfp4" else 127 - sc).astype(np.uint8)
    return codes, sc, ref.values(codes, sc, wdtype).astype(np.float32)


def fp4_operands(moe, rng, wdtype, counts, N, K, gx, gw):
    gr, (offsets, tiles, _, _), P, E, _ = grouping(moe, rng, counts)
    rows, wt = ref.padded_rows(offsets, tiles), -(-N // 128)
    w_rows = (np.arange(E * N) // N) * (wt * 128) + np.arange(E * N) % N
    xc, xs, xv = half_numbers(rng, wdtype, P, K)
    wc, ws, wv = half_numbers(rng, wdtype, E * N, K)
    pack = lambda c: c[:, 0::2] | (c[:, 1::2] << 4)  # noqa: E731
    one = lambda g: dev(np.array([g], np.float32))  # noqa: E731
    x = moe.FP4Rows(dev(pack(xc)), dev(ref.tile(xs, rows, (P + 127 * min(P, E)) // 128)), wdtype, one(gx), gr)
    w = moe.FP4Rows(dev(pack(wc).reshape(E, N, K // 2)), dev(ref.tile(ws, w_rows, E * wt)), wdtype, one(gw))
    y, _ = product(xv, wv.reshape(E, N, K), offsets)
    return x, w, gr, y * gx * gw, rows, P, E


# counts, experts, N, K, act, out (None: requantised), pairs of CTAs (64 rows an expert)
FP4_CASES = {
    "pairs": (many, 72, 4096, 544, "none", torch.bfloat16, True),
    "pairs_swiglu": (many, 40, 4096, 800, "swiglu", torch.bfloat16, True),
    "pairs_swiglu_odd": (many, 40, 3104, 288, "swiglu", torch.bfloat16, True),
    "pairs_requantised": (many, 40, 4096, 544, "swiglu", None, True),
    "pairs_fp32": (many, 40, 3001, 544, "none", torch.float32, True),
    "singles": (few, 150, 1100, 544, "none", torch.bfloat16, False),
    "singles_swiglu": (few, 150, 1024, 288, "swiglu", torch.bfloat16, False),
    "singles_requantised": (few, 150, 1024, 544, "swiglu", None, False),
    "singles_fp32": (few, 150, 1000, 800, "none", torch.float32, False),
    "singles_most_experts": (few, 4096, 200, 96, "none", torch.bfloat16, False),
}


@pytest.mark.parametrize("wdtype", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("name", FP4_CASES)
def test_fp4_products_of_many_items(moe, name, wdtype):
    make, E, N, K, act, out, pairs = FP4_CASES[name]
    rng = np.random.default_rng(len(name) + N)
    counts = make(rng, E) if make is many else few(rng, E, 40 if E == 150 else 6)
    gx, gw = (0.25, 0.125) if act == "swiglu" else (0.5, 2.0)
    x, w, gr, y, rows, P, E = fp4_operands(moe, rng, wdtype, counts, N, K, gx, gw)
    assert (P >= 64 * E) == pairs
    enough(counts, N // 2 if act == "swiglu" else N, act == "swiglu", pairs)
    if out is not None:
        got = host(moe.grouped_matmul_fp4(x, w, gr, act=act, out_dtype=out)).astype(np.float64)
        same_or_within(got, y, act == "swiglu", out)
        moe.check_operators()
        return
    go = np.float32(2.0 ** -6) if wdtype == "nvfp4" else None
    q = moe.grouped_matmul_fp4(x, w, gr, act=act, quantize=True, g_out=None if go is None else dev(np.array([go])))
    moe.check_operators()
    h, tol = swiglu(y)
    g = 1.0 if go is None else go
    codes, sc = ref.quantize(h.astype(np.float32), wdtype, g)
    gsc = ref.untile(host(q.scales), rows, sc.shape[1])
    # a scale or a code is another one only where h's error, some 1e-6 of it, carries a value over a rounding edge
    assert np.abs(gsc.astype(int) - sc).max() <= 1 and (gsc != sc).mean() < 1e-3
    same = (gsc == sc).repeat(ref.BLOCK[wdtype], axis=1)
    got = ref.unpack(host(q.codes))
    assert (got != codes)[same].mean() < 1e-3
    step = ref.values(np.full(codes.shape, 2, np.uint8), gsc, wdtype, g)          # the code of 1
    m = np.where(step > 0, np.abs(h) / np.where(step > 0, step, 1), 0)
    half = np.where(m <= 2, 0.25, np.where(m <= 4, 0.5, 1.0)) * step
    over = np.maximum(np.abs(h) - 6 * step, 0)
    err = np.abs(ref.values(got, gsc, wdtype, g) - h)
    assert (err <= half * (1 + 1e-6) + over * (1 + 1e-6) + 2 * tol)[step > 0].all()
    pad = ref.untile(host(q.scales), rows, 4 * host(q.scales).shape[1])[:, sc.shape[1]:]
    assert not pad.any()
