"""8-bit blocks, their products and the end of a block on the GPU, against their definitions (tests/operators8_reference.py)."""
import numpy as np
import pytest
import torch

from oracle.formats import E4M3_TABLE
from tests import operators8_reference as ref8
from tests import operators_reference as ref
from tests.test_operators_gpu import BF16, EPS, bf16, dev, host, make_ids
from tests.test_operators_many_items_gpu import few, grouping, many

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def moe():
    import serving_layer_moe_gb300 as m
    return m


def codes_of(q):
    return q.codes.view(torch.uint8).cpu().numpy()


def to8(codes):
    return torch.from_numpy(np.ascontiguousarray(codes, np.uint8)).cuda().view(F8)


# ---------------------------------------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------------------------------------
def spread(rng, R, K):
    """Rows of very different sizes, with elements of very different sizes, zeros, and ties of the 8-bit grid."""
    x = rng.standard_normal((R, K)) * np.exp2(rng.integers(-20, 20, (R, 1))) * np.exp2(rng.integers(-9, 1, (R, K)))
    x[rng.random((R, K)) < 0.05] = 0
    if R > 2:
        x[2] = rng.integers(-448, 449, K) * 0.5          # a = 224 or near it: many quotients half way between codes
        x[2, ::128] = 224
    return x.astype(np.float32)


@pytest.mark.parametrize("T,K", [(1, 16), (1, 7168), (3, 144), (5, 128), (33, 400), (130, 1040), (700, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_rows(moe, T, K, dtype):
    x = spread(np.random.default_rng(T + K), T, K)
    x = bf16(x) if dtype == "bf16" else x
    q = moe.quantize_fp8(dev(x, torch.bfloat16 if dtype == "bf16" else None))
    codes, scales = ref8.quantize(x, 1)
    assert np.array_equal(codes_of(q), codes) and np.array_equal(host(q.scales), scales.T)
    v = ref8.values(codes, scales, 1)
    for out in (torch.float32, torch.bfloat16):
        got, want = host(moe.dequantize_fp8(q, out_dtype=out)), v.astype(np.float32)       # a product of 4 and 24 bits
        assert np.allclose(got, want if out == torch.float32 else bf16(want), rtol=0, atol=0), out


@pytest.mark.parametrize("G,N,K", [(1, 1, 16), (1, 128, 128), (2, 200, 208), (3, 129, 272), (None, 300, 1040), (5, 257, 128)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_weights(moe, G, N, K, dtype):
    n = G or 1
    w = spread(np.random.default_rng(N + K), n * N, K).reshape(n, N, K)
    w = bf16(w) if dtype == "bf16" else w
    q = moe.quantize_fp8_weights(dev(w if G else w[0], torch.bfloat16 if dtype == "bf16" else None))
    assert tuple(q.shape) == ((G, N, K) if G else (N, K))
    codes, scales, v = codes_of(q).reshape(n, N, K), host(q.scales).reshape(n, -(-N // 128), -(-K // 128)), host(moe.dequantize_fp8(q, out_dtype=torch.float32)).reshape(n, N, K)
    for g in range(n):
        c, s = ref8.quantize(w[g], 128)
        assert np.array_equal(codes[g], c) and np.array_equal(scales[g], s)
        assert np.array_equal(v[g], ref8.values(c, s, 128).astype(np.float32))


def test_special_blocks(moe):
    """Zeros and their signs, the smallest and the largest numbers, NaN and infinities: of each block its own."""
    x = np.ones((1, 13 * 128), np.float32)
    for i, v in enumerate([0.0, -0.0, 1e-45, -1e-38, 2.0 ** -100, 1e-30, 1e-24, 1.1e24, 3.4e38, -3.4e38]):
        x[0, 128 * i:128 * i + 128] = 0
        x[0, 128 * i:128 * i + 64] = v
        x[0, 128 * i + 64] = v / 3
    x[0, 10 * 128 + 5], x[0, 11 * 128 + 127], x[0, 12 * 128] = np.nan, np.inf, -np.inf
    codes, scales = ref8.quantize(x, 1)
    for q, s in ((moe.quantize_fp8(dev(x)), scales.T), (moe.quantize_fp8_weights(dev(x)), scales)):
        assert np.array_equal(codes_of(q), codes) and np.array_equal(host(q.scales), s, equal_nan=True)
    v = host(moe.dequantize_fp8(moe.quantize_fp8(dev(x)), out_dtype=torch.float32))
    assert np.isnan(v[0, 10 * 128:]).all() and np.isfinite(v[0, :10 * 128]).all()


@pytest.mark.parametrize("T,E,k,K", [(1, 8, 8, 256), (7, 4, 3, 144), (300, 60, 6, 1040), (33, 5, 1, 16)])
def test_quantize_rows_by_expert(moe, T, E, k, K):
    rng = np.random.default_rng(T)
    x = bf16(spread(rng, T, K))
    ids = rng.integers(-1, E + 1, (T, k)).astype(np.int32)          # some pairs have no expert
    gr = moe.group_pairs(dev(ids), E)
    q, one = moe.quantize_fp8(dev(x, torch.bfloat16), groups=gr), moe.quantize_fp8(dev(x, torch.bfloat16))
    offsets, _, order, _ = ref.groups(ids, E)
    n = offsets[-1]
    src = order[:n] // k
    assert q.shape == (T * k, K) and np.array_equal(codes_of(q)[:n], codes_of(one)[src]) and np.array_equal(host(q.scales)[:, :n], host(one.scales)[:, src])


# ---------------------------------------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------------------------------------
SMALL = np.array([0x00, 0x38, 0x40, 0x30, 0xB8, 0xC0, 0xB0, 0x44])       # 0, 1, 2, .5, -1, -2, -.5, 3


def whole(rng, P, E, N, K):
    """Codes of small numbers and scales that are powers of two: every partial sum is exact in 24 bits."""
    KB, NB = -(-K // 128), -(-N // 128)
    xc, wc = rng.choice(SMALL, (P, K)), rng.choice(SMALL, (E, N, K))
    xs = np.exp2(rng.integers(-1, 2, (KB, P))).astype(np.float32)
    ws = np.exp2(rng.integers(-1, 2, (E, NB, KB))).astype(np.float32)
    return xc, xs, wc, ws


def product(xc, xs, wc, ws, offsets, dtype=np.float32):
    """Exact: sums of multiples of 1/16 below 2^20 (in fp32), or of any numbers in 64 bits."""
    x = E4M3_TABLE[xc].astype(dtype) * np.repeat(xs.T, 128, axis=1)[:, :xc.shape[1]].astype(dtype)
    out = np.zeros((xc.shape[0], wc.shape[1]), dtype)
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if b > a:
            s = np.repeat(np.repeat(ws[e], 128, axis=0)[:wc.shape[1]], 128, axis=1)[:, :wc.shape[2]].astype(dtype)
            out[a:b] = x[a:b] @ (E4M3_TABLE[wc[e]].astype(dtype) * s).T
    return out


def operands(moe, xc, xs, wc, ws):
    return moe.FP8Rows(to8(xc), dev(xs)), moe.FP8Weights(to8(wc), dev(ws))


# rows an expert, N, K
PRODUCTS = [([1], 128, 128), ([0, 3, 0, 5], 25, 16), ([16, 17, 1, 0], 256, 144), ([2, 2, 2, 2, 2, 2, 2, 2], 384, 272), ([40, 0, 9], 300, 1040),
            ([100, 33, 64, 65], 264, 400), ([256, 257, 255], 640, 256), ([300, 513, 20, 0], 384, 2048), ([31, 32, 33, 63, 127, 128, 129], 250, 128)]


@pytest.mark.parametrize("counts,N,K", PRODUCTS)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_products_of_exact_sums(moe, counts, N, K, out):
    rng = np.random.default_rng(N + K)
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    y = product(xc, xs, wc, ws, offsets)
    got = host(moe.grouped_matmul_fp8(*operands(moe, xc, xs, wc, ws), gr, out_dtype=out))
    assert np.array_equal(got, y if out == torch.float32 else bf16(y))


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 7168, 256), (5, 129, 144), (16, 512, 2048), (77, 1000, 400), (300, 256, 1040), (1001, 130, 272)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_products_of_one_matrix(moe, M, N, K, out):
    rng = np.random.default_rng(M + N)
    xc, xs, wc, ws = whole(rng, M, 1, N, K)
    y = product(xc, xs, wc, ws, [0, M])
    got = host(moe.matmul_fp8(*operands(moe, xc, xs, wc[0], ws[0]), out_dtype=out))
    assert np.array_equal(got, y if out == torch.float32 else bf16(y))


def rough(y, h):
    """What SwiGLU may be off before bf16 and 8-bit roundings: |gate| + 10 units (2^-23).  Past exp(-gate) = 2^60 the exponential stays
    there: gate / (1 + 2^60) in place of gate / (1 + exp(-gate)) is |gate| 2^-60 off at most, |gate up| 2^-60 after the product."""
    gate, up = np.split(np.abs(y), 2, axis=1)
    return (gate + 10) * 2 * EPS * np.abs(h) + gate * up * 2.0 ** -60 * (gate > 41) + 1e-30


@pytest.mark.parametrize("counts,N,K", [([1, 0, 1, 1, 0, 1], 384, 2000), ([2, 5, 0, 9], 1000, 1040), ([1], 640, 7168), ([31, 1], 512, 2048), ([64], 300, 656), ([128], 260, 1296),
                                        ([0, 0, 3], 129, 512)])
def test_few_items_share_k(moe, counts, N, K):
    """Calls that leave most SMs idle: several CTAs an item, every form of result."""
    rng = np.random.default_rng(K)
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    y = product(xc, xs, wc, ws, offsets)
    x, w = operands(moe, xc, xs, wc, ws)
    for out in (torch.float32, torch.bfloat16):
        assert np.array_equal(host(moe.grouped_matmul_fp8(x, w, gr, out_dtype=out)), y if out == torch.float32 else bf16(y))
    if N % 128 == 0:
        y = (y / 64).astype(np.float64)
        x = moe.FP8Rows(x.codes, x.scales / 64)
        for out in (torch.float32, torch.bfloat16):
            swiglu_within(host(moe.grouped_matmul_fp8(x, w, gr, act="swiglu", out_dtype=out)), y, out)
        check_quantized(moe.grouped_matmul_fp8(x, w, gr, act="swiglu", quantize=True), y)
    moe.check_operators()


def swiglu_within(got, y, out):
    """fp32: silu within 11 half units and a product; bf16: what `rough` says, then half a bf16 step."""
    h = ref.swiglu(y)
    if out == torch.float32:
        bad = np.abs(got - h) > 13 * EPS * np.abs(h) + 1e-33
    else:
        tol = rough(y, h)
        bad = np.abs(got - h) > tol + BF16 * (np.abs(h) + tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], h[bad][:5])


@pytest.mark.parametrize("counts,N,K", [([1], 128, 128), ([0, 3, 0, 5], 256, 16), ([16, 17, 1, 0], 384, 144), ([100, 33, 64, 65], 640, 400), ([300, 513, 20, 0], 384, 2048)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, "fp8"])
def test_swiglu(moe, counts, N, K, out):
    rng = np.random.default_rng(N + K)
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    y = product(xc, xs / 8, wc, ws, offsets).astype(np.float64)
    x, w = operands(moe, xc, xs / 8, wc, ws)
    if out != "fp8":
        return swiglu_within(host(moe.grouped_matmul_fp8(x, w, gr, act="swiglu", out_dtype=out)), y, out)
    check_quantized(moe.grouped_matmul_fp8(x, w, gr, act="swiglu", quantize=True), y)


def check_quantized(q, y):
    """Scales from the largest of the block's values; every value within half a step of its code, and three units of products
    with reciprocals, and what SwiGLU may be off."""
    h, n = ref.swiglu(y), y.shape[1] // 2
    tol = rough(y, h)
    codes, scales = codes_of(q), host(q.scales).astype(np.float64).T
    pad = -n % 128
    hb, tb = (np.pad(v, ((0, 0), (0, pad))).reshape(-1, (n + pad) // 128, 128) for v in (np.abs(h), tol))
    a, at = hb.max(axis=2), tb.max(axis=2)
    assert scales.shape == a.shape
    assert (np.abs(scales * 448 - np.maximum(a, ref8.LEAST)) <= at + 4 * EPS * a + ref8.LEAST * 1e-6).all()
    s = np.repeat(scales, 128, axis=1)[:, :n]
    t = h / s
    off = np.abs(E4M3_TABLE[codes] - t) - (ref8.half_step(t) * (1 + 2.0 ** -10) + tol / s + 8 * EPS * np.abs(t))
    assert (off <= 0).all(), (off.max(), np.argwhere(off > 0)[:5])


CASES = {  # counts, E, N, K, act
    "pairs": (many, 70, 4096, 144, "none"), "pairs_swiglu": (many, 40, 4096, 272, "swiglu"), "pairs_odd": (many, 60, 3001, 16, "none"),
    "singles": (few, 250, 1000, 144, "none"), "singles_swiglu": (few, 200, 1024, 272, "swiglu")}


@pytest.mark.parametrize("name", CASES)
def test_products_of_many_tiles(moe, name):
    """Several tiles for every unit of the persistent kernel: what a unit carries from one to the next."""
    make, E, N, K, act = CASES[name]
    rng = np.random.default_rng(E)
    counts = make(rng, E) if make is many else make(rng, E, 9)
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    xs = xs / 8 if act == "swiglu" else xs
    y = product(xc, xs, wc, ws, offsets)
    x, w = operands(moe, xc, xs, wc, ws)
    for out in (torch.float32, torch.bfloat16):
        got = host(moe.grouped_matmul_fp8(x, w, gr, act=act, out_dtype=out))
        if act == "none":
            assert np.array_equal(got, y if out == torch.float32 else bf16(y))
        else:
            swiglu_within(got, y.astype(np.float64), out)
    if act == "swiglu":
        check_quantized(moe.grouped_matmul_fp8(x, w, gr, act=act, quantize=True), y.astype(np.float64))
    moe.check_operators()


@pytest.mark.parametrize("counts", [[70, 80, 75, 75], [3, 1, 2, 4]])
@pytest.mark.parametrize("K", [272, 7168])
def test_any_scales_add_up(moe, counts, K):
    """Scales of any size and mantissa.  A block's four additions truncate, by half a unit each on average, of a sum that grows to
    its size: 4 * 0.75 * 2^-24; the product of the scales and each addition over K round: 2^-24 each, whose errors add like their
    squares or slower.  Together below 5e-7 of the result's norm."""
    rng = np.random.default_rng(K)
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    N, KB = 200, -(-K // 128)
    x, w = rng.standard_normal((P, K)), rng.standard_normal((E, N, K))
    xc, _ = ref8.quantize(x, 1)
    wc = np.stack([ref8.quantize(v, 128)[0] for v in w])
    xs, ws = (np.exp(rng.standard_normal(s)).astype(np.float32) for s in ((KB, P), (E, 2, KB)))
    y = product(xc, xs, wc, ws, offsets, np.float64)
    got = host(moe.grouped_matmul_fp8(*operands(moe, xc, xs, wc, ws), gr, out_dtype=torch.float32))
    assert np.linalg.norm(got - y) < 5e-7 * np.linalg.norm(y)


def test_a_nan_stays_where_it_is(moe):
    """A NaN code or scale reaches the results that it is a part of, and no others."""
    rng = np.random.default_rng(3)
    counts, N, K = [40, 5, 30], 256, 400
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    y = product(xc, xs, wc, ws, offsets)
    xc[7, 399], xs[1, 42] = 0x7F, np.nan
    wc[1, 3, 5], ws[2, 1, 3] = 0xFF, np.nan
    y[7], y[42], y[40:45, 3], y[45:, 128:] = np.nan, np.nan, np.nan, np.nan
    assert np.array_equal(host(moe.grouped_matmul_fp8(*operands(moe, xc, xs, wc, ws), gr, out_dtype=torch.float32)), y, equal_nan=True)


def test_rows_behind_the_last_expert_stay(moe):
    """Pairs without an expert: their rows of out, codes and scales are not written."""
    from serving_layer_moe_gb300.operators import _operators
    lib, s = _operators(), torch.cuda.current_stream().cuda_stream
    rng = np.random.default_rng(5)
    E, P, N, K = 3, 100, 256, 144
    ids = rng.integers(0, E + 2, (P, 1)).astype(np.int32)
    gr, (offsets, _, _, _) = moe.group_pairs(dev(ids), E), ref.groups(ids, E)
    n = offsets[-1]
    assert 0 < n < P
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    x, w = operands(moe, xc, xs, wc, ws)
    y = product(xc, xs, wc, ws, offsets)
    out = torch.full((P, N), 7.0, device="cuda")
    args = (x.codes.data_ptr(), x.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(), gr.offsets.data_ptr())
    assert lib.moe_grouped_matmul_fp8(P, E, N, K, *args, 0, 0, out.data_ptr(), None, None, s) == 0
    assert np.array_equal(host(out)[:n], y[:n]) and (host(out)[n:] == 7).all()
    codes, scales = torch.full((P, N // 2), 9, dtype=torch.uint8, device="cuda"), torch.full((1, P), 7.0, device="cuda")
    assert lib.moe_grouped_matmul_fp8(P, E, N, K, *args, 1, 1, None, codes.data_ptr(), scales.data_ptr(), s) == 0
    assert (host(codes)[n:] == 9).all() and (host(scales)[:, n:] == 7).all() and not (host(scales)[:, :n] == 7).all()


# ---------------------------------------------------------------------------------------------------------
# the end of a block
# ---------------------------------------------------------------------------------------------------------
def end_within(got, want, mag, k, N, dtype, normed):
    """fp32 before the last rounding: k + 3 operations on parts that add up to mag, and with a norm a mean of N squares (each
    addition of its tree rounds: 2 log2 N + 8), a reciprocal root (two units, halved by the root) and two products."""
    ops = k + 5 + normed * (2 * np.log2(max(N, 2)) + 16 + N / 1024)
    tol = ops * EPS * mag + 1e-37
    if dtype == torch.bfloat16:
        tol = tol + BF16 * (np.abs(want) + tol)
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)


TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)]


@pytest.mark.parametrize("yt,rt", TYPES)
@pytest.mark.parametrize("T,E,k,N", [(1, 256, 8, 7168), (3, 4, 2, 1), (33, 8, 3, 257), (5, 60, 6, 2048), (2, 3, 1, 8200), (320, 16, 4, 1000), (400, 8, 2, 77),
                                     (310, 8, 2, 7168), (2, 4, 2, 32768), (2, 4, 2, 32767), (3, 4, 2, 15000)])
def test_combine_norm(moe, T, E, k, N, yt, rt):
    rng = np.random.default_rng(T + N)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[0, 0] = E                                                # a pair without an expert
    if T > 2:
        ids[2] = -1                                              # a token without any
    gr, (_, _, _, place) = moe.group_pairs(dev(ids), E), ref.groups(ids, E)
    r = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    t = lambda a, d: (bf16(a) if d == torch.bfloat16 else a)  # noqa: E731
    y, w, res, sh = t(r(T * k, N), yt), r(T, k), t(r(T, N), rt), t(r(T, N), yt)
    y[ref.groups(ids, E)[0][-1]:] = np.nan                       # rows that nobody fills
    post, pre, gate, gate_t = 1 + r(N) / 8, bf16(1 + r(N) / 8), r(N), r(T, 1)
    for i, kw in enumerate([dict(), dict(pre=pre), dict(shared=sh, post=post, gate=gate, scale=0.7, pre=pre), dict(post=pre, gate=gate_t, pre=post, eps=0.5),
                            dict(shared=sh, gate=gate, scale=-2.0), dict(post=post)]):
        h, z, mh, mz = ref8.block_end(y, place, w, res, **kw)
        on = {n: dev(v, (yt if n == "shared" else torch.bfloat16 if v is pre else None)) if isinstance(v, np.ndarray) else v for n, v in kw.items()}
        on["residual_scale"] = on.pop("scale", 1.0)
        zt = torch.float32 if i % 2 else torch.bfloat16
        got = moe.combine_norm(dev(y, yt), gr, dev(w), dev(res, rt), out_dtype=zt, **on)
        gh, gz = got if z is not None else (got, None)
        assert gh.dtype == rt
        end_within(host(gh), h, mh, k, N, rt, kw.get("post") is not None)
        if z is not None:
            assert gz.dtype == zt
            end_within(host(gz), z, mz + np.abs(z), k, N, zt, 2)


@pytest.mark.parametrize("T,N", [(1, 7168), (4, 3), (700, 256), (333, 1001)])
def test_residual_norm_and_rms_norm(moe, T, N):
    rng = np.random.default_rng(N)
    y, res = bf16(rng.standard_normal((T, N))), rng.standard_normal((T, N)).astype(np.float32) * 3
    post, pre = (1 + rng.standard_normal((2, N)) / 8).astype(np.float32)
    h, z, mh, mz = ref8.block_end(y, None, None, res, post=post, pre=pre, scale=0.5, eps=1e-5)
    gh, gz = moe.residual_norm(dev(y, torch.bfloat16), dev(res), post=dev(post), pre=dev(pre), residual_scale=0.5, eps=1e-5, out_dtype=torch.float32)
    end_within(host(gh), h, mh, 1, N, torch.float32, 1)
    end_within(host(gz), z, mz + np.abs(z), 1, N, torch.float32, 2)
    _, z, _, mz = ref8.block_end(None, None, None, res, pre=pre)
    end_within(host(moe.rms_norm(dev(res), dev(pre))), z, mz, 1, N, torch.bfloat16, 1)


def test_norms_of_zeros_and_of_huge_rows(moe):
    x = np.zeros((6, 64), np.float32)
    x[1], x[2], x[3, 5], x[4, 7], x[5] = 1e-30, 1e18, np.nan, np.inf, 3e19
    one = dev(np.ones(64, np.float32))
    got = host(moe.rms_norm(dev(x), one, out_dtype=torch.float32))
    assert not got[0].any() and np.allclose(got[1], 1e-30 / np.sqrt(1e-6), rtol=1e-5) and np.allclose(got[2], 1, rtol=1e-5)
    assert np.isnan(got[3]).all() and np.isnan(got[4, 7]) and not got[5].any()
    assert not got[4, :7].any()


# ---------------------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------------------
def block(moe, T, E, k, H, I, seed=0):
    """A block of experts with a shared one, from bf16 weights; call(x, h) -> (h, z)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).bfloat16()  # noqa: E731
    wide = {"gu": normal(E, 2 * I, H, std=H ** -0.5), "dn": normal(E, H, I, std=I ** -0.5), "sgu": normal(2 * I, H, std=H ** -0.5), "sdn": normal(H, I, std=I ** -0.5)}
    w8 = {n: moe.quantize_fp8_weights(w) for n, w in wide.items()}
    pre, post = (1 + torch.randn(2, H, generator=gen, device="cuda") / 8)
    logits, x, h = torch.randn(T, E, generator=gen, device="cuda"), normal(T, H), normal(T, H)

    def call():
        _, w, gr = moe.route(logits, k, groups=True)
        a = moe.grouped_matmul_fp8(moe.quantize_fp8(x, groups=gr), w8["gu"], gr, act="swiglu", quantize=True)
        y = moe.grouped_matmul_fp8(a, w8["dn"], gr)
        s = moe.matmul_fp8(moe.matmul_fp8(moe.quantize_fp8(x), w8["sgu"], act="swiglu", quantize=True), w8["sdn"])
        return moe.combine_norm(y, gr, w, h, shared=s, post=post, residual_scale=0.5, pre=pre)

    def plain():
        def mlp(v, gu, dn):
            a = v @ gu.double().T
            return (torch.nn.functional.silu(a[:, :I]) * a[:, I:]) @ dn.double().T
        p = torch.softmax(logits.double(), 1)
        w, ids = p.topk(k, 1)
        w, v = w / w.sum(1, keepdim=True), x.double()
        c = mlp(v, wide["sgu"], wide["sdn"])
        for e in range(E):
            hit = (ids == e).double() * w
            c = c + hit.sum(1, keepdim=True) * mlp(v, wide["gu"][e], wide["dn"][e])
        norm = lambda v, g: v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * g.double()  # noqa: E731
        out = 0.5 * h.double() + norm(c, post)
        return out, norm(out, pre)
    return call, plain, (logits, x, h)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 128), (37, 8, 3, 400, 192), (600, 16, 4, 512, 256)])
def test_a_block_of_experts(moe, T, E, k, H, I):
    """Four roundings to 8 bits (x, its products' input, both weights) on each way through: each is off by 2^-4 / sqrt(3) of a
    step's half on average, at most 2^-4 relative; together with bf16's well below sqrt(4) * 2^-4 of the block's part of h."""
    call, plain, _ = block(moe, T, E, k, H, I)
    (h, z), (ph, pz) = call(), plain()
    assert ((h.double() - ph).norm() / ph.norm()).item() < 0.125 and ((z.double() - pz).norm() / pz.norm()).item() < 0.125
    moe.check_operators()


@pytest.mark.parametrize("T", [1, 3, 300])
def test_a_block_in_a_graph_and_on_a_stream(moe, T):
    call, _, (logits, x, h) = block(moe, T, 8, 2, 256, 128)
    other, _, (l2, x2, h2) = block(moe, T, 8, 2, 256, 128, seed=1)
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for a, b in ((logits, l2), (x, x2), (h, h2)):
        a.copy_(b)
    graph.replay()
    now = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, now)) and not torch.equal(out[0], want[0])


def test_large_calls_give_the_same_bits_again(moe):
    call, _, _ = block(moe, 3000, 64, 8, 1024, 384)
    want = call()
    assert all(t.isfinite().all() for t in want)
    for _ in range(9):
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
    moe.check_operators()


@pytest.mark.parametrize("E", [0, 4])
def test_no_tokens(moe, E):
    x = torch.zeros(0, 256, device="cuda", dtype=torch.bfloat16)
    gr = moe.group_pairs(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), E) if E else None
    q = moe.quantize_fp8(x, groups=gr)
    assert q.shape == (0, 256) and moe.dequantize_fp8(q).shape == (0, 256)
    w = moe.quantize_fp8_weights(torch.ones(*((E,) if E else ()), 256, 256, device="cuda"))
    f = (lambda **kw: moe.grouped_matmul_fp8(q, w, gr, **kw)) if E else (lambda **kw: moe.matmul_fp8(q, w, **kw))
    assert f().shape == (0, 256) and f(act="swiglu", quantize=True).shape == (0, 128)
    one = torch.ones(256, device="cuda")
    if E:
        h, z = moe.combine_norm(x, gr, torch.zeros(0, 2, device="cuda"), x, pre=one)
    else:
        h, z = moe.residual_norm(x, x, pre=one)
    assert h.shape == z.shape == moe.rms_norm(x, one).shape == (0, 256)


@pytest.mark.parametrize("act,quant", [("none", False), ("swiglu", False), ("swiglu", True)])
def test_a_rows_result_does_not_depend_on_the_rows_beside_it(moe, act, quant):
    """The same row alone, in small calls and in large ones, whose tiles differ."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    K, N = 1040, 512
    x, w = torch.randn(3000, K, generator=gen, device="cuda").bfloat16(), moe.quantize_fp8_weights(torch.randn(N, K, generator=gen, device="cuda").bfloat16())

    def rows(n):
        r = moe.matmul_fp8(moe.quantize_fp8(x[:n]), w, act=act, quantize=quant)
        return r.codes.view(torch.uint8) if quant else r
    want = rows(3000)
    for n in (1, 16, 40, 128, 129, 700):
        assert torch.equal(rows(n), want[:n]), n


def test_the_example_runs(moe):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import routed_layer
    r = routed_layer.run(tokens=300, hidden=512, inter=256, experts=16, top_k=4, fmt="fp8")
    assert np.isfinite(r["distance"]) and r["chunk_ms"] > 0 and r["token_ms"] > 0
