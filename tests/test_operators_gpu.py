"""The routed-expert operators on the GPU against their definitions in 64 bits (tests/operators_reference.py)."""
import numpy as np
import pytest
import torch

from tests import operators_reference as ref

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24         # half a unit in the last place of fp32, relative
BF16 = 2.0 ** -8         # the same of bf16: eight significant bits


@pytest.fixture(scope="module")
def moe():
    import serving_layer_moe_gb300 as m
    return m


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def host(t):
    return (t.float() if t.dtype == torch.bfloat16 else t).cpu().numpy()


def bf16(a):
    """Rounded to bf16, as fp32."""
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().float().numpy()


def make_ids(rng, counts, T, k):
    """ids [T, k] whose pairs hold `counts[e]` of expert e (repeats within a token allowed), shuffled."""
    flat = np.repeat(np.arange(len(counts)), counts)
    assert flat.size == T * k
    return rng.permutation(flat).reshape(T, k).astype(np.int32)


# ---------------------------------------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,E,k,dtype,renorm,scale", [
    (1, 128, 8, "f32", True, 1.0), (5, 1, 1, "f32", True, 1.0), (33, 60, 6, "bf16", False, 2.5), (300, 300, 4, "f32", True, 1.0),
    (64, 8, 8, "f32", False, 1.0), (7, 1000, 40, "f32", True, 0.5), (3, 4096, 8, "bf16", True, 1.0), (2500, 128, 8, "f32", True, 1.0)])
def test_softmax_route_and_groups(moe, T, E, k, dtype, renorm, scale):
    rng = np.random.default_rng(T * 1000 + E)
    z = bf16(rng.standard_normal((T, E)))          # rounded: ties are there
    ids, w, gr = moe.route(dev(z, torch.bfloat16 if dtype == "bf16" else None), k, renormalize=renorm, scale=scale, groups=True)
    rid, rw = ref.route(z, k, renorm=renorm, scale=scale)
    assert np.array_equal(host(ids), rid)
    # a term is exp to 2 ulp of a difference rounded once (|l - max| < 16: 8 ulp in the exponential), sums of
    # k or E positive terms, one division, one product
    assert np.allclose(host(w), rw, rtol=(E + 32) * 2 * EPS, atol=1e-30)
    check_groups(gr, rid, E)


def check_groups(gr, ids, E):
    offsets, tiles, order, place = ref.groups(ids, E)
    assert np.array_equal(host(gr.offsets), offsets) and np.array_equal(host(gr.tiles), tiles)
    assert np.array_equal(host(gr.order), order) and np.array_equal(host(gr.place), place)


def test_route_rows_that_leave_nothing(moe):
    inf, nan = np.inf, np.nan
    z = np.zeros((8, 6), np.float32)
    z[0] = -inf
    z[1] = nan
    z[2] = [nan, -inf, 1, nan, -inf, 0]
    z[3] = [inf, 0, inf, 1, 2, 3]
    z[4] = np.finfo(np.float32).min
    z[5] = [0.0, -0.0, 0.0, -0.0, -1, 1]
    z[6] = [1e30, -1e30, 0, 0, 0, 0]
    z[7] = [-inf, -inf, -inf, -inf, -inf, 5]
    for scoring in ("softmax", "sigmoid"):
        ids, w = moe.route(dev(z), 4, scoring=scoring)
        rid, rw = ref.route(z, 4, scoring=scoring)
        assert np.array_equal(host(ids), rid), scoring
        assert np.isfinite(host(w)).all()
        assert np.allclose(host(w), rw, rtol=64 * EPS, atol=1e-37)


@pytest.mark.parametrize("T,E,k,n_group,topk_group,bias", [
    (40, 256, 8, 8, 4, True), (1, 256, 8, 8, 4, True), (17, 60, 6, 4, 2, True), (9, 32, 5, 32, 7, False),
    (600, 96, 6, 3, 2, True), (30, 128, 8, 1, 1, True), (30, 20, 2, 5, 1, False)])
def test_sigmoid_route_with_groups(moe, T, E, k, n_group, topk_group, bias):
    rng = np.random.default_rng(T + 7 * E)
    # scores on a grid of 2^-12 with exact sums: no choice hangs on the last bit of a sigmoid
    grid = np.stack([rng.permutation(4095)[:E] + 1 for _ in range(T)]) / 4096.0
    z = np.log(grid / (1 - grid)).astype(np.float32)
    b = (rng.integers(-512, 512, E) / 4096 + np.arange(E) / 2.0 ** 21).astype(np.float32) if bias else None
    pick = grid + (0 if b is None else b)
    if n_group > 1:
        s = np.sort(np.sort(pick.reshape(T, n_group, -1), axis=2)[:, :, ::-1][:, :, :2].sum(axis=2), axis=1)
        ok = (np.diff(s, axis=1) > 1e-5).all(axis=1)
        z, T = z[ok], int(ok.sum())
        assert T > 0
    ids, w, gr = moe.route(dev(z), k, scoring="sigmoid", bias=None if b is None else dev(b), n_group=n_group,
                           topk_group=topk_group, scale=2.5, groups=True)
    rid, rw = ref.route(z, k, "sigmoid", b, n_group, topk_group, scale=2.5)
    s = np.sort(1 / (1 + np.exp(-z.astype(np.float64))) + (0 if b is None else b), axis=1)
    clear = (np.diff(s, axis=1) > 1e-6).all(axis=1)
    assert clear.any() and np.array_equal(host(ids)[clear], rid[clear])
    assert np.allclose(host(w)[clear], rw[clear], rtol=(k + 32) * 2 * EPS)
    check_groups(gr, host(ids), E)


@pytest.mark.parametrize("E", [32, 64, 96, 128, 256, 384, 512, 1024, 2048, 4096])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("skip", [0, 1])
def test_route_widths_and_where_the_picks_lie(moe, E, dtype, skip):
    """Whole and partial lanes, rows that start off 16 bytes, and picks that lie together, apart, or are equal."""
    rng = np.random.default_rng(E)
    k = min(E, 40)
    z = bf16(rng.standard_normal((14, E)))
    z[0] = np.maximum(-np.arange(E), -255) / 4                     # the first ones in order: exact in bf16
    z[1] = z[0, ::-1]                                              # the last ones
    z[2] = 0.5
    z[3] = np.repeat(rng.permutation(E // 2) % 16, 2)              # equal neighbours
    z[4, ::3], z[4, 1] = np.nan, np.inf
    z[5] = np.nan
    z[6] = -np.inf
    z[7], z[7, E // 2:E // 2 + 3] = -np.inf, [1, np.nan, 1]
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.empty(z.size + skip, dtype=t, device="cuda")[skip:].view(z.shape)
    x.copy_(dev(z, t))
    ids, w, gr = moe.route(x, k, groups=True)
    rid, rw = ref.route(z, k)
    assert np.array_equal(host(ids), rid)
    # as above; picks lie within 10 of the largest, or their terms below 1e-30 come from a row of -inf
    assert np.allclose(host(w), rw, rtol=(k + 32) * 2 * EPS, atol=1e-30)
    check_groups(gr, rid, E)


@pytest.mark.parametrize("E,n_group", [(256, 8), (256, 32), (64, 2), (60, 6), (160, 8), (512, 16)])
def test_sigmoid_groups_with_equal_and_missing_scores(moe, E, n_group):
    rng = np.random.default_rng(E + n_group)
    z = rng.choice(np.array([-np.inf, 0, np.inf], np.float32), (24, E))    # scores 0, 0.5 and 1
    z[rng.random(z.shape) < 0.05] = np.nan
    gs, keep = E // n_group, max(1, n_group // 2)
    z[:, ::gs], z[:, 1::gs] = 0, 0                                         # no group is short of two scores, but for
    z[0:8, gs:2 * gs] = np.nan                                             # one that has none
    z[8] = np.nan
    ids, w = moe.route(dev(z), 4, scoring="sigmoid", n_group=n_group, topk_group=keep)
    rid, rw = ref.route(z, 4, "sigmoid", None, n_group, keep)
    assert np.array_equal(host(ids), rid)
    assert np.allclose(host(w), rw, rtol=64 * EPS)


@pytest.mark.parametrize("T,E,k", [(0, 4, 2), (1, 1, 1), (3, 5, 2), (100, 7, 3), (33, 4096, 4), (5000, 256, 8), (20000, 3, 2), (1300, 1024, 1)])
def test_group_pairs_drops_foreign_ids(moe, T, E, k):
    rng = np.random.default_rng(T + E)
    ids = rng.integers(-2, E + 2, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.3] = E // 2      # one crowded expert
    check_groups(moe.group_pairs(dev(ids), E), ids, E)


# ---------------------------------------------------------------------------------------------------------
# 4-bit quantisation
# ---------------------------------------------------------------------------------------------------------
def special_rows(K):
    x = np.zeros((9, K), np.float32)
    x[1] = 1e-40
    x[2, ::3] = np.inf
    x[3, 5] = np.nan
    x[4] = np.finfo(np.float32).max
    x[5] = np.resize([0.25, -0.75, 1.25, -1.75, 2.5, -3.5, 5.0, 6.0], K)      # ties
    x[6] = np.resize([-0.0, 1e-30, 3e38, -2.0], K)
    x[7] = np.resize([-0.0, 1.0, 0.0, -0.5], K)
    x[8] = np.resize([-3e37, 2.0, -1e30, 1e37], K)                            # far past the largest scale, both signs
    return x


@pytest.mark.parametrize("wdtype", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,N,K", [(1, 1, 32), (1, 5, 96), (3, 130, 160), (2, 128, 64), (1, 300, 1440), (5, 1, 224)])
def test_quantize_stack_bit_for_bit(moe, wdtype, dtype, G, N, K):
    rng = np.random.default_rng(G * N + K)
    x = (rng.standard_normal((G * N, K)) * np.exp(rng.standard_normal((G * N, 1)) * 3)).astype(np.float32)
    x[: min(9, G * N)] = special_rows(K)[: min(9, G * N)]
    if dtype == torch.bfloat16:
        x = bf16(x)
    g = np.exp(rng.standard_normal(G) - 6).astype(np.float32) if wdtype == "nvfp4" else None
    q = moe.quantize_fp4(dev(x.reshape(G, N, K), dtype), wdtype, g=None if g is None else dev(g))
    gr = 1.0 if g is None else np.repeat(g, N)
    codes, sc = ref.quantize(x, wdtype, gr)
    rows = (np.arange(G * N) // N) * (-(-N // 128) * 128) + np.arange(G * N) % N
    assert np.array_equal(ref.untile(host(q.scales), rows, sc.shape[1]), sc)
    nan = np.repeat(sc == (0x7F if wdtype == "nvfp4" else 255), ref.BLOCK[wdtype], axis=1)
    got = ref.unpack(host(q.codes).reshape(G * N, K // 2))
    assert np.array_equal(got[~nan], codes[~nan])
    # blocks past the end pad with 0
    B4 = 4 * host(q.scales).shape[1]
    assert not ref.untile(host(q.scales), rows, B4)[:, sc.shape[1]:].any()
    # back: e2m1 times a step of 32 bits, a value of 32 bits (6 * 2^126 is its infinity)
    v = moe.dequantize_fp4(q, out_dtype=torch.float32)
    with np.errstate(over="ignore"):
        want = ref.values(codes, sc, wdtype, gr).astype(np.float32)
    got = host(v).reshape(G * N, K)
    assert np.array_equal(np.isnan(got), nan)
    assert np.allclose(got[~nan], want[~nan], rtol=2 * EPS, atol=2.0 ** -149)
    assert torch.equal(moe.dequantize_fp4(q).nan_to_num(), v.bfloat16().nan_to_num())


def test_quantize_is_the_bank_layouts_conversion(moe):
    """Codes, block scales and matrix scales of the generator's NVFP4 and MXFP4 experts, byte for byte."""
    from workloads import _mxfp4, _nvfp4
    rng = np.random.default_rng(5)
    w = (rng.standard_normal((200, 256)) * 0.02).astype(np.float32)
    packed, sc, g = _nvfp4(w)
    got = moe.fp4_scale(dev(w))
    assert host(got)[0] == np.abs(w).max() * np.float32(1 / 2688)
    q = moe.quantize_fp4(dev(w), "nvfp4", g=dev(np.array([g])))
    assert np.array_equal(host(q.codes), packed)
    assert np.array_equal(ref.untile(host(q.scales), np.arange(200), 16), sc)
    packed, sc = _mxfp4(w)
    q = moe.quantize_fp4(dev(w), "mxfp4")
    assert np.array_equal(host(q.codes), packed) and np.array_equal(ref.untile(host(q.scales), np.arange(200), 8), sc)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,count", [(1, 7), (3, 4096), (2, 123457), (70, 33)])
def test_fp4_scale(moe, dtype, G, count):
    rng = np.random.default_rng(count)
    x = bf16(rng.standard_normal((G, 1, count)))
    x[0] = 0
    if G > 1:
        x[1, 0, count // 2] = -np.inf
    got = host(moe.fp4_scale(dev(x, dtype)))
    want = (np.abs(x).max(axis=(1, 2)) * np.float32(1 / 2688)).astype(np.float32)
    want[0] = 1
    assert np.array_equal(got, want)


@pytest.mark.parametrize("wdtype", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,E,k,K", [(1, 128, 8, 64), (77, 60, 6, 1440), (300, 4, 2, 96), (40, 9, 3, 2048)])
def test_quantize_rows_by_expert(moe, wdtype, T, E, k, K):
    rng = np.random.default_rng(T + K)
    x = bf16(rng.standard_normal((T, K)))
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)
    gr = moe.group_pairs(dev(ids), E)
    offsets, tiles, order, _ = ref.groups(ids, E)
    n = offsets[-1]
    g = np.array([0.01], np.float32) if wdtype == "nvfp4" else None
    q = moe.quantize_fp4(dev(x, torch.bfloat16), wdtype, g=None if g is None else dev(g), groups=gr)
    codes, sc = ref.quantize(x[order[:n] // k], wdtype, 1.0 if g is None else g[0])
    assert np.array_equal(ref.unpack(host(q.codes)[:n]), codes)
    assert np.array_equal(ref.untile(host(q.scales), ref.padded_rows(offsets, tiles), sc.shape[1]), sc)
    v = host(moe.dequantize_fp4(q, out_dtype=torch.float32))
    assert np.allclose(v[:n], ref.values(codes, sc, wdtype, 1.0 if g is None else g[0]), rtol=2 * EPS)
    assert not v[n:].any()


# ---------------------------------------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------------------------------------
COUNTS = [
    ([1], 1), ([0, 1, 0], 1), ([8] * 8, 8), ([0, 129, 0, 3, 128, 127, 257, 0], 4), ([1, 2, 3, 4, 5, 6, 7, 8], 6),
    ([700, 0, 0, 20], 8), ([16, 15, 17, 33, 31, 32, 64, 48], 8), ([513], 3), ([256, 256, 512], 2)]


def rounded_within(got, want, tol, out):
    """Each value within tol of what it should be, and its own rounding: a bf16's half unit, relative."""
    bound = tol + (BF16 * (np.abs(want) + tol) if out == torch.bfloat16 else EPS * np.abs(want))
    bad = np.abs(got - want) > bound
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], bound[bad][:5])


def swiglu_tolerance(y, tol):
    """SwiGLU of values that are off by tol: |silu'| <= 1.1, silu in fp32 to 8 units."""
    n = y.shape[1] // 2
    g, u, tg, tu = y[:, :n], y[:, n:], tol[:, :n], tol[:, n:]
    s = np.abs(g / (1 + np.exp(-g)))
    return 1.1 * tg * (np.abs(u) + tu) + s * tu + 16 * EPS * s * np.abs(u)


@pytest.mark.parametrize("counts,k", COUNTS)
@pytest.mark.parametrize("N,K,act,out,gather", [
    (64, 64, "none", torch.bfloat16, True), (96, 72, "swiglu", torch.bfloat16, False), (37, 8, "none", torch.float32, True),
    (1, 200, "none", torch.bfloat16, False), (416, 264, "swiglu", torch.float32, True), (300, 1032, "none", torch.float32, False)])
def test_grouped_matmul(moe, counts, k, N, K, act, out, gather):
    P, E = sum(counts), len(counts)
    while P % k:
        k -= 1
    T = P // k
    rng = np.random.default_rng(P + N + K)
    ids = make_ids(rng, counts, T, k)
    gr = moe.group_pairs(dev(ids), E)
    offsets, _, order, _ = ref.groups(ids, E)
    x = bf16(rng.standard_normal((T if gather else P, K)))
    w = bf16(rng.standard_normal((E, N, K)) * 0.1)
    got = host(moe.grouped_matmul(dev(x, torch.bfloat16), dev(w, torch.bfloat16), gr, act=act, gather=gather, out_dtype=out))
    xr = x[order // k] if gather else x
    y, mag = ref.product(xr.astype(np.float64), w.astype(np.float64), offsets)
    tol = 4 * K * EPS * mag      # exact products; K fp32 additions, each off by at most two units of the running sum
    if act == "swiglu":
        y, tol = ref.swiglu(y), swiglu_tolerance(y, tol)
    rounded_within(got.astype(np.float64), y, tol, out)


def make_fp4(moe, rng, wdtype, shape, gr=None, rows=None, n_tiles=None):
    """Quantised random rows [R, K] in the library's layout, and their exact values."""
    R, K = shape
    x = (rng.standard_normal((R, K)) * np.exp(rng.standard_normal((R, 1)))).astype(np.float32)
    g = np.float32(0.02)
    codes, sc = ref.quantize(x, wdtype, g if wdtype == "nvfp4" else 1.0)
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    tiles = ref.tile(sc, rows, n_tiles)
    # what pads a tile beyond the rows is never used: NaN scales there must not show
    fill = np.full_like(tiles, 0x7F if wdtype == "nvfp4" else 255)
    keep = ref.tile(np.ones((R, 4 * tiles.shape[1]), np.uint8), rows, n_tiles).astype(bool)
    tiles = np.where(keep, tiles, fill)
    return packed, tiles, (g if wdtype == "nvfp4" else None), ref.values(codes, sc, wdtype, g if wdtype == "nvfp4" else 1.0)


def fp4_case(moe, rng, wdtype, counts, k, N, K):
    P, E = sum(counts), len(counts)
    while P % k:
        k -= 1
    ids = make_ids(rng, counts, P // k, k)
    gr = moe.group_pairs(dev(ids), E)
    offsets, tiles, _, _ = ref.groups(ids, E)
    nt = (P + 127 * min(P, E)) // 128
    xc, xt, xg, xv = make_fp4(moe, rng, wdtype, (P, K), rows=ref.padded_rows(offsets, tiles), n_tiles=nt)
    wt = -(-N // 128)
    rows = (np.arange(E * N) // N) * (wt * 128) + np.arange(E * N) % N
    wc, wtl, wg, wv = make_fp4(moe, rng, wdtype, (E * N, K), rows=rows, n_tiles=E * wt)
    one = lambda g: None if g is None else dev(np.array([g], np.float32))  # noqa: E731
    x = moe.FP4Rows(dev(xc), dev(xt), wdtype, one(xg), gr)
    w = moe.FP4Rows(dev(wc.reshape(E, N, K // 2)), dev(wtl), wdtype, one(wg))
    y, mag = ref.product(xv, wv.reshape(E, N, K), offsets)
    return x, w, gr, y, mag, offsets, tiles


@pytest.mark.parametrize("wdtype", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("counts,k", COUNTS)
@pytest.mark.parametrize("N,K,act,out", [
    (128, 256, "none", torch.bfloat16), (37, 32, "none", torch.float32), (96, 160, "swiglu", torch.bfloat16),
    (300, 1056, "none", torch.float32), (320, 544, "swiglu", torch.float32)])
def test_grouped_matmul_fp4(moe, wdtype, counts, k, N, K, act, out):
    rng = np.random.default_rng(sum(counts) + N + K)
    x, w, gr, y, mag, _, _ = fp4_case(moe, rng, wdtype, counts, k, N, K)
    got = host(moe.grouped_matmul_fp4(x, w, gr, act=act, out_dtype=out))
    tol = (4 * K + 8) * EPS * mag
    if act == "swiglu":
        y, tol = ref.swiglu(y), swiglu_tolerance(y, tol)
    rounded_within(got.astype(np.float64), y, tol, out)


@pytest.mark.parametrize("wdtype", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("counts,k", COUNTS)
@pytest.mark.parametrize("N,K", [(64, 96), (320, 544), (448, 256)])
def test_grouped_matmul_fp4_to_fp4(moe, wdtype, counts, k, N, K):
    rng = np.random.default_rng(sum(counts) + N + K)
    x, w, gr, y, mag, offsets, tiles = fp4_case(moe, rng, wdtype, counts, k, N, K)
    go = np.float32(0.05) if wdtype == "nvfp4" else None
    q = moe.grouped_matmul_fp4(x, w, gr, act="swiglu", quantize=True, g_out=None if go is None else dev(np.array([go])))
    h, tol = ref.swiglu(y), swiglu_tolerance(y, (4 * K + 8) * EPS * mag)
    codes, sc = ref.quantize(h.astype(np.float32), wdtype, 1.0 if go is None else go)
    rows = ref.padded_rows(offsets, tiles)
    gsc = ref.untile(host(q.scales), rows, sc.shape[1])
    # a scale differs only where h's error can carry the block's largest value over a rounding edge
    assert np.abs(gsc.astype(int) - sc).max() <= 1 and (gsc != sc).mean() < 0.01
    B = ref.BLOCK[wdtype]
    g = 1.0 if go is None else go
    got = ref.unpack(host(q.codes))
    step = np.repeat(ref.values(np.full((len(rows), sc.shape[1] * B), 2, np.uint8), gsc, wdtype, g), 1, axis=1)
    with np.errstate(divide="ignore", invalid="ignore"):
        m = np.where(step > 0, np.abs(h) / step, 0.0)
    half = np.where(m <= 2, 0.25, np.where(m <= 4, 0.5, 1.0)) * step
    over = np.maximum(np.abs(h) - 6 * step, 0)
    err = np.abs(ref.values(got, gsc, wdtype, g) - h)
    assert (err <= half * (1 + 1e-6) + over * 1.000001 + 2 * tol)[step > 0].all()
    same = (gsc == sc).repeat(B, axis=1)
    assert (got != codes)[same].mean() < 0.01
    # blocks past the end pad with 0
    pad = ref.untile(host(q.scales), rows, 4 * host(q.scales).shape[1])[:, sc.shape[1]:]
    assert not pad.any()


# ---------------------------------------------------------------------------------------------------------
# combine
# ---------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("yd", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("od", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,N", [(1, 8, 8, 2048), (33, 60, 6, 1000), (5, 3, 2, 37), (700, 16, 4, 72), (2, 1, 1, 1)])
def test_combine(moe, yd, od, T, E, k, N):
    rng = np.random.default_rng(T + N)
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)
    if T > 1:
        ids[0] = -1                                     # a token with no expert here
    gr = moe.group_pairs(dev(ids), E)
    place = ref.groups(ids, E)[3]
    y = bf16(rng.standard_normal((T * k, N)))
    n = int((place >= 0).sum())
    y[n:] = np.nan                                       # rows that no pair fills
    w = rng.random((T, k)).astype(np.float32)
    w[place < 0] = np.nan
    got = host(moe.combine(dev(y, yd), gr, dev(w), out_dtype=od))
    want = ref.combine(y.astype(np.float64), place, w.astype(np.float64))
    mag = ref.combine(np.abs(y).astype(np.float64), place, np.abs(w).astype(np.float64))
    rounded_within(got.astype(np.float64), want, 2 * k * EPS * mag, od)


# ---------------------------------------------------------------------------------------------------------
# use: streams, graphs, repeats, the whole layer
# ---------------------------------------------------------------------------------------------------------
def layer(moe, x, logits, gu, down, k, gx, gh, stream=None):
    ids, w, gr = moe.route(logits, k, groups=True, stream=stream)
    xq = moe.quantize_fp4(x, "nvfp4", g=gx, groups=gr, stream=stream)
    h = moe.grouped_matmul_fp4(xq, gu, gr, act="swiglu", quantize=True, g_out=gh, stream=stream)
    y = moe.grouped_matmul_fp4(h, down, gr, stream=stream)
    return moe.combine(y, gr, w, stream=stream)


@pytest.fixture(scope="module")
def small_layer(moe):
    torch.manual_seed(3)
    E, H, I = 16, 256, 192
    gu = torch.randn(E, 2 * I, H, device="cuda") * 0.05
    dn = torch.randn(E, H, I, device="cuda") * 0.05
    gu = moe.quantize_fp4(gu, "nvfp4", g=moe.fp4_scale(gu))
    dn = moe.quantize_fp4(dn, "nvfp4", g=moe.fp4_scale(dn))
    one = torch.full((1,), 0.002, device="cuda")
    return E, H, I, gu, dn, one


@pytest.mark.parametrize("T", [1, 50, 777])
def test_layer_is_its_parts(moe, small_layer, T):
    E, H, I, gu, dn, g = small_layer
    k = 4
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    logits = torch.randn(T, E, device="cuda", generator=gen)
    out = layer(moe, x, logits, gu, dn, k, g, g)
    ids, w = ref.route(host(logits), k)
    offsets, _, order, place = ref.groups(ids, E)
    gv = float(host(g)[0])
    xr = ref.values(*ref.quantize(host(x)[order // k], "nvfp4", np.float32(gv)), "nvfp4", np.float32(gv))
    wgu = host(moe.dequantize_fp4(gu, out_dtype=torch.float32)).astype(np.float64)
    wdn = host(moe.dequantize_fp4(dn, out_dtype=torch.float32)).astype(np.float64)
    h = ref.swiglu(ref.product(xr, wgu, offsets)[0])
    hr = ref.values(*ref.quantize(h.astype(np.float32), "nvfp4", np.float32(gv)), "nvfp4", np.float32(gv))
    want = ref.combine(ref.product(hr, wdn, offsets)[0], place, w)
    # y is rounded to bf16 before the sum; a code of h may flip at an edge
    err = np.linalg.norm(host(out) - want) / np.linalg.norm(want)
    assert err < 2 * BF16, err


def test_same_bits_on_another_stream_and_from_a_graph(moe, small_layer):
    E, H, I, gu, dn, g = small_layer
    T, k = 200, 4
    x = torch.randn(T, H, device="cuda").bfloat16()
    logits = torch.randn(T, E, device="cuda")
    want = layer(moe, x, logits, gu, dn, k, g, g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = layer(moe, x, logits, gu, dn, k, g, g, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(moe, x, logits, gu, dn, k, g, g)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    x2 = torch.randn(T, H, device="cuda").bfloat16()
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, layer(moe, x2, logits, gu, dn, k, g, g)) and not torch.equal(out, want)
    moe.check_operators()


def test_no_tokens(moe, small_layer):
    E, H, I, gu, dn, g = small_layer
    x = torch.empty(0, H, device="cuda", dtype=torch.bfloat16)
    out = layer(moe, x, torch.empty(0, E, device="cuda"), gu, dn, 4, g, g)
    assert out.shape == (0, H)
    gr = moe.group_pairs(torch.empty(0, 4, dtype=torch.int32, device="cuda"), E)
    assert not gr.offsets.any() and not gr.tiles.any()


def test_every_pair_dropped(moe, small_layer):
    E, H, I, gu, dn, g = small_layer
    ids = torch.full((9, 4), -1, dtype=torch.int32, device="cuda")
    gr = moe.group_pairs(ids, E)
    x = torch.randn(9, H, device="cuda").bfloat16()
    xq = moe.quantize_fp4(x, "nvfp4", g=g, groups=gr)
    h = moe.grouped_matmul_fp4(xq, gu, gr, act="swiglu", quantize=True, g_out=g)
    y = moe.grouped_matmul_fp4(h, dn, gr)
    out = moe.combine(y, gr, torch.rand(9, 4, device="cuda"))
    assert not out.any()


def test_binding_refusals(moe, small_layer):
    E, H, I, gu, dn, g = small_layer
    x = torch.randn(6, H, device="cuda").bfloat16()
    logits = torch.randn(6, E, device="cuda")
    _, w, gr = moe.route(logits, 4, groups=True)
    xq = moe.quantize_fp4(x, "nvfp4", g=g, groups=gr)
    mx = moe.quantize_fp4(x, "mxfp4", groups=gr)
    wb = torch.zeros(E, 64, H, device="cuda", dtype=torch.bfloat16)
    for word, call in [
        ("top_k", lambda: moe.route(logits, E + 1)), ("scoring", lambda: moe.route(logits, 2, scoring="max")),
        ("softmax", lambda: moe.route(logits, 2, bias=logits[0])), ("E = 16", lambda: moe.route(logits, 2, scoring="sigmoid", bias=logits[0, :3].contiguous())),
        ("n_group", lambda: moe.route(logits, 4, scoring="sigmoid", n_group=8, topk_group=1)),
        ("multiple of 32", lambda: moe.quantize_fp4(x[:, :40].contiguous(), "nvfp4")),
        ("only nvfp4", lambda: moe.quantize_fp4(x, "mxfp4", g=g)), ("rows", lambda: moe.quantize_fp4(x[:5].contiguous(), "nvfp4", groups=gr)),
        ("g must hold", lambda: moe.quantize_fp4(x, "nvfp4", g=torch.ones(3, device="cuda"))),
        ("act", lambda: moe.grouped_matmul(x, wb, gr, act="gelu", gather=True)), ("x must be", lambda: moe.grouped_matmul(x, wb, gr)),
        ("experts", lambda: moe.grouped_matmul(x, wb[:3].contiguous(), gr, gather=True)),
        ("16-byte", lambda: moe.grouped_matmul(torch.zeros(6 * H + 1, device="cuda", dtype=torch.bfloat16)[1:].view(6, H), wb, gr, gather=True)),
        ("mxfp4", lambda: moe.grouped_matmul_fp4(mx, gu, gr)), ("x must be", lambda: moe.grouped_matmul_fp4(xq, dn, gr)),
        ("quantize needs", lambda: moe.grouped_matmul_fp4(xq, gu, gr, quantize=True)),
        ("g_out", lambda: moe.grouped_matmul_fp4(xq, gu, gr, act="swiglu", g_out=g)),
        ("scales must be", lambda: moe.grouped_matmul_fp4(xq, moe.FP4Rows(gu.codes, gu.scales[:1], "nvfp4", gu.g), gr)),
        ("topk_w", lambda: moe.combine(x, gr, w[:3])), ("y must be", lambda: moe.combine(x, gr, w)),
        ("on cpu", lambda: moe.combine(torch.zeros(24, 8, device="cuda"), gr, w.cpu())),
    ]:
        with pytest.raises(ValueError, match=word):
            call()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_example_layer(fmt):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import routed_layer
    r = routed_layer.run(tokens=300, hidden=512, inter=256, experts=16, top_k=4, fmt=fmt)
    # a 4-bit value is up to 1/6 of its block's largest off; three of them multiply up to a result
    assert 0.01 < r["distance"] < 0.4, r
