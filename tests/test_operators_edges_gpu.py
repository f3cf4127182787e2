"""The routed-expert operators on the GPU: refusals, special values and sizes, one case each."""
import numpy as np
import pytest
import torch

from tests import operators_reference as ref
from tests.test_operators_gpu import EPS, bf16, dev, host, make_ids

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import serving_layer_moe_gb300 as m
    return m


def test_quantize_takes_no_integers_for_groups(moe):
    x = torch.zeros(2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="ExpertGroups"):
        moe.quantize_fp4(x, "mxfp4", groups=(0, 8, 4, 2, 2, 4096, 8192, 12288, 16384))


def small_case(moe):
    gen = torch.Generator(device="cuda").manual_seed(1)
    T, E, k, H = 40, 8, 2, 64
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    w = moe.quantize_fp4(torch.randn(E, 96, H, device="cuda", generator=gen).bfloat16(), "mxfp4")
    ids, gates, gr = moe.route(torch.randn(T, E, device="cuda", generator=gen), k, groups=True)
    return x, w, ids, gates, gr, moe.quantize_fp4(x, "mxfp4", groups=gr)


def test_copies_are_used_where_they_are(moe):
    """A copy's results do not hang on the memory of what it was copied from."""
    import copy
    x, w, ids, gates, gr, q = small_case(moe)
    want = moe.combine(moe.grouped_matmul_fp4(q, w, gr), gr, gates)
    q2, w2, gr2 = copy.deepcopy((q, w, gr))
    for t in (q.codes, q.scales, w.codes, w.scales, gr.offsets, gr.tiles, gr.order, gr.place):
        t.zero_()
    assert torch.equal(moe.combine(moe.grouped_matmul_fp4(q2, w2, gr2), gr2, gates), want)
    assert not torch.equal(moe.dequantize_fp4(w2), moe.dequantize_fp4(w))
    assert torch.equal(gr2.order.sort().values, torch.arange(gr2.P, device="cuda", dtype=torch.int32))


def test_resized_tensors_are_found_or_refused(moe):
    x, w, ids, gates, gr, q = small_case(moe)
    want = moe.combine(moe.grouped_matmul_fp4(q, w, gr), gr, gates)
    ids.resize_(1 << 20)                                   # whatever this moves, the groups go with it
    torch.cuda.synchronize()
    junk = [torch.full((1 << 20,), -1, device="cuda", dtype=torch.int32) for _ in range(4)]
    assert torch.equal(moe.combine(moe.grouped_matmul_fp4(q, w, gr), gr, gates), want)
    del junk
    codes = w.codes.clone()
    v = moe.FP4Rows(codes, w.scales, "mxfp4")
    codes.resize_(2, 96, 32)
    with pytest.raises(ValueError, match="experts"):       # it holds two of eight now
        moe.grouped_matmul_fp4(q, v, gr)
    order = gr.order.clone()
    held = moe.ExpertGroups(gr.offsets, gr.tiles, order, gr.place)
    order.set_(torch.empty(0, dtype=torch.int32, device="cuda"))
    y = torch.zeros(gr.P, 8, device="cuda")
    with pytest.raises(ValueError, match="resized"):
        moe.combine(y, held, gates)


@pytest.mark.parametrize("T,E,k", [(40, 200, 2), (2000, 256, 8)])
def test_results_keep_their_own_memory_only(moe, T, E, k):
    """No result of route or group_pairs keeps the grouping's scratch; ids and gates of many pairs
    do not keep the groups."""
    ids, w, gr = moe.route(torch.randn(T, E, device="cuda"), k, groups=True)
    P, four = T * k, 4 * 2 * (E + 1 + T * k)
    most = {ids: 8 * P, w: 8 * P, gr.order: four} if P > 256 else {ids: 8 * P + four, w: 8 * P + four, gr.order: 8 * P + four}
    for t, n in most.items():
        assert t.untyped_storage().nbytes() == n, (tuple(t.shape), t.untyped_storage().nbytes(), n)
    assert moe.group_pairs(ids, E).order.untyped_storage().nbytes() == four


# ---------------------------------------------------------------------------------------------------------
# fp32 results
# ---------------------------------------------------------------------------------------------------------
def distance(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("K", [1944, 7168])
@pytest.mark.parametrize("counts", [[70, 80, 75, 75], [3, 1, 2, 4]])
def test_fp32_results_of_bf16_products_add_up(moe, counts, K):
    """An accumulator that truncates, by half a unit (2^-24 of the sum or less) on average, takes 16 additions to a sum that grows
    to its size: 16 * 0.75 * 2^-24 * 2/3 = 4.8e-7 of it.  All of K = 1944 in one, 122 additions: 3.6e-6."""
    rng = np.random.default_rng(K)
    ids = make_ids(rng, counts, sum(counts), 1)
    gr, (offsets, _, _, _) = moe.group_pairs(dev(ids), len(counts)), ref.groups(ids, len(counts))
    x, w = bf16(rng.standard_normal((sum(counts), K))), bf16(rng.standard_normal((len(counts), 96, K)))
    y, _ = ref.product(x.astype(np.float64), w.astype(np.float64), offsets)
    got = host(moe.grouped_matmul(dev(x, torch.bfloat16), dev(w, torch.bfloat16), gr, out_dtype=torch.float32))
    assert distance(got, y) < 5e-7


def rows_of_uneven_blocks(rng, wdtype, R, K, rows, tiles):
    """Rows whose blocks' sizes differ by a factor of e^2 (one standard deviation), 4-bit: packed codes, tiles, g, values."""
    B = ref.BLOCK[wdtype]
    size = np.repeat(np.exp(2 * rng.standard_normal((R, K // B))), B, axis=1)
    x = (rng.standard_normal((R, K)) * size).astype(np.float32)
    g = np.float32(np.abs(x).max() / 2688) if wdtype == "nvfp4" else np.float32(1)
    codes, sc = ref.quantize(x, wdtype, g)
    return dev(codes[:, 0::2] | (codes[:, 1::2] << 4)), dev(ref.tile(sc, rows, tiles)), g, ref.values(codes, sc, wdtype, g)


@pytest.mark.parametrize("wdtype", ["nvfp4", "mxfp4"])
def test_fp32_results_of_4bit_products_add_up(moe, wdtype):
    """Few large blocks and many small ones: once a sum is large, each addition to it is truncated.  16 of them take 16 * 0.75 * 2^-24
    = 7.2e-7 of it at most on average, all 112 of K = 7168 seven times that."""
    rng = np.random.default_rng(11)
    counts, N, K = [70, 80, 75, 75], 96, 7168
    P, E = sum(counts), len(counts)
    ids = make_ids(rng, counts, P, 1)
    gr, (offsets, tiles, _, _) = moe.group_pairs(dev(ids), E), ref.groups(ids, E)
    xc, xs, xg, xv = rows_of_uneven_blocks(rng, wdtype, P, K, ref.padded_rows(offsets, tiles), (P + 127 * E) // 128)
    wc, ws, wg, wv = rows_of_uneven_blocks(rng, wdtype, E * N, K, np.arange(E * N) // N * 128 + np.arange(E * N) % N, E)
    one = lambda g: dev(np.array([g])) if wdtype == "nvfp4" else None  # noqa: E731
    got = host(moe.grouped_matmul_fp4(moe.FP4Rows(xc, xs, wdtype, one(xg), gr), moe.FP4Rows(wc.view(E, N, K // 2), ws, wdtype, one(wg)), gr,
                                      out_dtype=torch.float32))
    y, _ = ref.product(xv, wv.reshape(E, N, K), offsets)
    assert distance(got, y) < 1e-6


@pytest.mark.parametrize("kind", ["bf16", "nvfp4", "mxfp4"])
def test_fp32_swiglu(moe, kind):
    """Of exact sums: silu within ten half units, one more for the product with up."""
    from tests.test_operators_many_items_gpu import fp4_operands, product
    rng = np.random.default_rng(4)
    counts, N, K = [5, 9, 100, 64], 512, 544
    if kind == "bf16":
        P, E = sum(counts), len(counts)
        ids = make_ids(rng, counts, P, 1)
        gr, (offsets, _, _, _) = moe.group_pairs(dev(ids), E), ref.groups(ids, E)
        x, w = rng.integers(-2, 3, (P, K)).astype(np.float32), rng.integers(-2, 3, (E, N, K)).astype(np.float32) * 0.5
        y, _ = product(x, w, offsets)
        got = moe.grouped_matmul(dev(x, torch.bfloat16), dev(w, torch.bfloat16), gr, act="swiglu", out_dtype=torch.float32)
    else:
        x, w, gr, y, _, _, _ = fp4_operands(moe, rng, kind, counts, N, K, 1.0, 0.5)
        got = moe.grouped_matmul_fp4(x, w, gr, act="swiglu", out_dtype=torch.float32)
    assert y.min() < -40 and y.max() > 40
    h = ref.swiglu(y)
    bad = np.abs(host(got) - h) > 12 * EPS * np.abs(h) + 1e-33      # a gate below -87 leaves less than 1e-36 of itself
    assert not bad.any(), (y[:, :N // 2][bad][:5], host(got)[bad][:5], h[bad][:5])


# ---------------------------------------------------------------------------------------------------------
# NaN in the router
# ---------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("E", [8, 64, 100, 256])
@pytest.mark.parametrize("renorm", [True, False])
def test_a_nan_score_has_no_gate(moe, E, renorm):
    """Three experts of finite score, k = 5: the other two picks have NaN for a bias, or for a logit, and weigh nothing."""
    z, b = np.full((2, E), -1, np.float32), np.full(E, np.nan, np.float32)
    good = [1, 3, E - 1]
    b[good] = [0.5, 0.25, 0.0]
    z[1, good[0]] = np.nan                                 # in the second row only two are left
    ids, w = moe.route(dev(z), 5, scoring="sigmoid", bias=dev(b), renormalize=renorm)
    rest = [e for e in range(E) if e not in good]
    assert host(ids)[0].tolist() == good + rest[:2]
    assert host(ids)[1].tolist() == good[1:] + sorted(rest + good[:1])[:3]
    s = 1 / (1 + np.exp(1.0))
    want = np.array([[s] * 3 + [0] * 2, [s] * 2 + [0] * 3])
    if renorm:
        want /= want.sum(axis=1, keepdims=True)
    assert np.allclose(host(w), want, rtol=16 * EPS, atol=0)


@pytest.mark.parametrize("size", [2, 3, 8, 32])
def test_a_nan_adds_nothing_to_its_groups_score(moe, size):
    """Eight groups: one of a single number and NaN, one of NaN alone, the others of numbers; three compete."""
    E = 8 * size
    z = np.full((1, 8, size), -3, np.float32)
    z[0, 2] = np.nan
    z[0, 4], z[0, 4, size - 1] = np.nan, 3                  # scores sigmoid(3) = 0.95
    z[0, 5] = 0                                            # 1
    z[0, 7] = -0.5                                         # 0.76
    ids, w = moe.route(dev(z.reshape(1, E)), 3, scoring="sigmoid", n_group=8, topk_group=3)
    assert host(ids)[0].tolist() == [4 * size + size - 1, 5 * size, 5 * size + 1]
    # with one group more, and all of their experts picked, the NaN of group 4 come after the numbers
    ids, w = moe.route(dev(z.reshape(1, E)), 4 * size, scoring="sigmoid", n_group=8, topk_group=4, renormalize=False)
    numbers = 3 * size + 1
    nan = [4 * size + i for i in range(size - 1)]
    assert host(ids)[0, numbers:].tolist() == nan and not host(w)[0, numbers:].any() and host(w)[0, :numbers].all()
    # all eight: the group of NaN alone is in
    ids, _ = moe.route(dev(z.reshape(1, E)), E, scoring="sigmoid", n_group=8, topk_group=8)
    assert host(ids)[0, E - size - len(nan):].tolist() == list(range(2 * size, 3 * size)) + nan


def test_rows_of_other_groups_are_refused(moe):
    """The rows of one routing under the groups of another, of the same sizes: their scales lie elsewhere."""
    x, w, ids, gates, gr, q = small_case(moe)
    want = moe.grouped_matmul_fp4(q, w, gr)
    other = moe.group_pairs((ids + 1) % gr.E, gr.E)
    with pytest.raises(ValueError, match="other groups"):
        moe.grouped_matmul_fp4(q, w, other)
    same = moe.ExpertGroups(gr.offsets, gr.tiles, gr.order, gr.place)
    assert torch.equal(moe.grouped_matmul_fp4(q, w, same), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_combine_refuses_rows_off_16_bytes_as_a_value(moe, dtype):
    x, w, ids, gates, gr, q = small_case(moe)
    room = torch.randn(gr.P * 16 + 1, device="cuda").to(dtype)
    with pytest.raises(ValueError, match="16-byte aligned"):
        moe.combine(room[1:].view(gr.P, 16), gr, gates)
    odd = room[1:gr.P * 9 + 1].view(gr.P, 9)               # rows of nine start anywhere
    assert torch.equal(moe.combine(odd, gr, gates), moe.combine(odd.clone(), gr, gates))


def test_too_many_matrices_are_refused_as_values(moe):
    x = torch.zeros(65536, 1, 32, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="65535"):
        moe.quantize_fp4(x, "mxfp4")
    assert torch.equal(moe.fp4_scale(x), torch.ones(65536, device="cuda"))        # no stack of 4-bit matrices
    q = moe.quantize_fp4(x[:65535], "mxfp4")
    assert q.shape == (65535, 1, 32) and not moe.dequantize_fp4(q).any()


@pytest.mark.parametrize("g", [1e-39, 2e-45, 1.0])
def test_requantised_zeros_under_a_subnormal_matrix_scale(moe, g):
    """1 / g is infinite below 2^-128, 0 / g is not: a block of zeros has scale and codes 0."""
    E, H, I = 2, 64, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn(E, 2 * I, H, device="cuda", generator=gen).bfloat16()
    w[:, I:I + 32] = 0                                     # the first 32 features of every result are zero
    gr = moe.group_pairs(torch.tensor([[0], [1], [1]], dtype=torch.int32, device="cuda"), E)
    x = moe.quantize_fp4(torch.randn(3, H, device="cuda", generator=gen).bfloat16(), "nvfp4", groups=gr)
    g = torch.tensor([g], device="cuda")
    q = moe.grouped_matmul_fp4(x, moe.quantize_fp4(w, "nvfp4"), gr, act="swiglu", quantize=True, g_out=g)
    v = host(moe.dequantize_fp4(q, out_dtype=torch.float32))
    assert not v[:, :32].any() and np.isfinite(v).all()


@pytest.mark.parametrize("T,k", [(16, 8), (32, 8), (33, 7), (64, 4), (65, 3), (128, 2), (256, 1), (257, 1)])
@pytest.mark.parametrize("E", [60, 1024])
def test_route_and_group_pairs_of_about_256_pairs(moe, T, k, E):
    """On both sides of the limits of the one-block forms, 32 tokens and 256 pairs."""
    z = np.random.default_rng(T * E).permutation(T * E).reshape(T, E).astype(np.float32) / (T * E)      # no two alike
    ids, w, gr = moe.route(dev(z), k, groups=True)
    assert np.array_equal(host(ids), np.argsort(-z, axis=1)[:, :k])
    want = ref.groups(host(ids), E)
    for g in (gr, moe.group_pairs(ids, E)):
        assert all(np.array_equal(host(a), b) for a, b in zip((g.offsets, g.tiles, g.order, g.place), want))


# ---------------------------------------------------------------------------------------------------------
# long and repeated calls, and the cache behind the router
# ---------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,E,k,scoring", [(8193, 96, 4, "softmax"), (20000, 64, 6, "sigmoid"), (70001, 8, 2, "softmax")])
def test_route_of_several_tokens_a_warp(moe, T, E, k, scoring):
    """Past 8192 tokens a counting block takes more than eight.  Logits of a row are exact steps of 1/64: no two alike."""
    rng = np.random.default_rng(T)
    z = (np.argsort(rng.random((T, E)), axis=1) / 64).astype(np.float32)
    ids, w, gr = moe.route(dev(z), k, scoring=scoring, groups=True)
    rid = np.argsort(-z, axis=1)[:, :k]
    assert np.array_equal(host(ids), rid)
    zt = np.take_along_axis(z, rid, axis=1).astype(np.float64)
    p = np.exp(zt) if scoring == "softmax" else 1 / (1 + np.exp(-zt))
    # a term within 4 units, k additions, a division
    assert np.allclose(host(w), p / p.sum(axis=1, keepdims=True), rtol=(k + 16) * 2 * EPS)
    want = ref.groups(rid, E)
    for g in (gr, moe.group_pairs(ids, E)):
        assert all(np.array_equal(host(a), b) for a, b in zip((g.offsets, g.tiles, g.order, g.place), want))


def test_large_calls_give_the_same_bits_again(moe):
    """A 4-bit layer and a bf16 one of 3000 tokens and 128 experts, ten times each."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    T, E, k, H, I = 3000, 128, 8, 512, 384
    gu = (torch.randn(E, 2 * I, H, device="cuda", generator=gen) * 0.05).bfloat16()
    dn = (torch.randn(E, H, I, device="cuda", generator=gen) * 0.05).bfloat16()
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    logits = torch.randn(T, E, device="cuda", generator=gen)
    gu4, dn4 = (moe.quantize_fp4(w, "nvfp4", g=moe.fp4_scale(w)) for w in (gu, dn))
    g = torch.full((1,), 0.002, device="cuda")

    def layer4(out):
        _, w, gr = moe.route(logits, k, groups=True)
        h = moe.grouped_matmul_fp4(moe.quantize_fp4(x, "nvfp4", g=g, groups=gr), gu4, gr, act="swiglu", quantize=True, g_out=g)
        return moe.combine(moe.grouped_matmul_fp4(h, dn4, gr, out_dtype=out), gr, w)

    def layer16(out):
        _, w, gr = moe.route(logits, k, groups=True)
        h = moe.grouped_matmul(x, gu, gr, act="swiglu", gather=True)
        return moe.combine(moe.grouped_matmul(h, dn, gr, out_dtype=out), gr, w)

    for layer in (layer4, layer16):
        for out in (torch.bfloat16, torch.float32):
            want = layer(out)
            assert want.isfinite().all() and want.any()
            for _ in range(9):
                assert torch.equal(layer(out), want)
    moe.check_operators()


def test_the_cache_decodes_what_the_router_picks(moe):
    """route's ids and gates as they are, into MoECache.decode: slot maps equal the oracle's, outputs within its tolerance."""
    from oracle.cache import SlotCache
    from oracle.ffn import ExpertStore, combine, pair_outputs, relative_max_error
    from tests.harness import TOL, build_pool, make_cache, torch_act
    from workloads import activations, config
    cfg = config("tiny")
    s = cfg.shape
    arena, offs, pool = build_pool(cfg)
    bw = cfg.bw_mbps
    cache, K = make_cache(cfg, pool, offs, None, bw)
    ora = SlotCache(s.L, s.E, cfg.capacity, K, bw[0], bw[1])
    store = ExpertStore(arena, offs, s.wdtype, s.H, s.I, s.blob_bytes)
    gen = torch.Generator(device="cuda").manual_seed(9)
    out = torch.empty(cfg.T, s.H, device="cuda")
    slots = torch.empty(cfg.T, s.k, dtype=torch.int32, device="cuda")
    for step in range(12):
        logits = torch.randn(cfg.T, s.E, device="cuda", generator=gen).bfloat16()
        ids, gates, _ = moe.route(logits, s.k, groups=True) if step % 2 else (*moe.route(logits, s.k), None)
        plan = ora.decode(0, host(ids))
        x = activations(cfg, step, 0)
        y = pair_outputs(store, 0, s.E, x, s.adtype, host(ids))
        cpu = dev(np.where(plan.slot_map[..., None] < 0, y, np.nan).astype(np.float32))
        cache.decode(0, torch_act(x, "cuda"), ids, gates, out, cpu_part=cpu, slot_map=slots)
        assert np.array_equal(host(slots), plan.slot_map)
        assert relative_max_error(host(out), combine(host(gates), y, plan.slot_map, y)) <= TOL
    cache.close()


def test_fp32_swiglu_of_huge_and_infinite_gates(moe):
    big = float(torch.finfo(torch.bfloat16).max)
    gates = np.array([big, np.inf, 2.0 ** 100, 2.0 ** 127, -big, -2.0 ** 100, np.nan, 128, 129, -128, -129, 88, -88, 1, 0, -0.0], np.float32)
    with np.errstate(over="ignore"):
        want = gates / (1 + np.exp(-gates.astype(np.float64)))
    # products that are these gates, and ones for up: the first element of K times one, the others zeros
    w, x = np.zeros((2, 32, 64), np.float32), np.zeros((6, 64), np.float32)
    w[:, :16, 0], w[:, 16:, 0], x[:, 0] = gates, 1, 1
    gr = moe.group_pairs(torch.tensor([[0], [1], [1], [0], [1], [0]], dtype=torch.int32, device="cuda"), 2)
    for row in host(moe.grouped_matmul(dev(x, torch.bfloat16), dev(w, torch.bfloat16), gr, act="swiglu", out_dtype=torch.float32)):
        assert np.array_equal(np.isnan(row), np.isnan(want)), row
        ok = ~np.isnan(want)
        assert np.array_equal(np.isinf(row), np.isinf(want)) and np.allclose(row[ok], want[ok], rtol=12 * EPS, atol=1e-33), row


# ---------------------------------------------------------------------------------------------------------
# groups that are none
# ---------------------------------------------------------------------------------------------------------
class Guarded:
    """Memory for an output with as much again on both sides, which has to stay as it is."""

    def __init__(self, n):
        self.room, self.n = torch.full((n + (2 << 20),), 0x5A, dtype=torch.uint8, device="cuda"), n
        self.at = self.room.data_ptr() + (1 << 20)
        assert self.at % 16 == 0

    def kept(self):
        return bool((self.room[:1 << 20] == 0x5A).all()) and bool((self.room[(1 << 20) + self.n:] == 0x5A).all())


def strange_groups(kind, P, E, rng):
    i32 = np.iinfo(np.int32)
    if kind == "random":
        return [rng.integers(i32.min, i32.max, n, dtype=np.int64).astype(np.int32) for n in (E + 1, E + 1, P, P)]
    if kind == "larger":      # a grouping, of four times the rows
        ids = rng.integers(0, E, (4 * P, 1))
        off, tiles, order, place = ref.groups(ids, E)
        return [np.asarray(a, np.int32) for a in (off, tiles, order[:P], place.reshape(-1)[:P])]
    if kind == "falling":
        off = np.linspace(P, 0, E + 1).astype(np.int32)
        return [off, off, np.arange(P, dtype=np.int32)[::-1].copy(), np.full(P, P, np.int32)]
    edge = np.array([i32.min, -1, 0, P - 1, P, i32.max])
    return [rng.choice(edge, n).astype(np.int32) for n in (E + 1, E + 1, P, P)]


@pytest.mark.parametrize("kind", ["random", "larger", "falling", "edges"])
@pytest.mark.parametrize("P,E", [(96, 40), (1200, 6), (640, 5)])
def test_no_groups_lead_outside_the_arrays(moe, kind, P, E):
    """Offsets, tiles, orders and places that are no grouping: wrong results, nothing read or written elsewhere, and the next call right."""
    from serving_layer_moe_gb300.operators import _operators
    lib, s = _operators(), torch.cuda.current_stream().cuda_stream
    rng = np.random.default_rng(P + E)
    k, N, K = 2, 256, 128
    T = P // k
    off, tiles, order, place = (dev(a) for a in strange_groups(kind, P, E, rng))
    x, w = torch.randn(P, K, device="cuda").bfloat16(), torch.randn(E, N, K, device="cuda").bfloat16()
    y, gates = torch.randn(P, N, device="cuda"), torch.rand(T, k, device="cuda")
    n_tiles = lib.moe_grouped_tiles(P, E)
    p = lambda t: t.data_ptr()  # noqa: E731
    outs = []

    def out(n):
        outs.append(Guarded(n))
        return outs[-1].at

    def done(status):
        assert status == 0, lib.moe_last_error()

    done(lib.moe_combine(T, k, N, 0, p(y), p(place), p(gates), 0, out(T * N * 4), s))
    for act in (0, 1):
        for gathered in (False, True):
            for od, size in ((0, 4), (1, 2)):
                need = lib.moe_grouped_matmul_workspace(P, E, K, gathered)
                done(lib.moe_grouped_matmul(P, E, N, K, p(x), T if gathered else P, p(order) if gathered else None, p(place) if gathered else None, k, p(w),
                                            p(off), p(tiles), act, od, out(P * N // (1 + act) * size), out(need) if need else None, need, s))
    for fmt, code in (("nvfp4", 3), ("mxfp4", 4)):
        groups = -(-K // (64 if fmt == "nvfp4" else 128))
        codes, scales = out(P * K // 2), out(n_tiles * groups * 512)
        done(lib.moe_quantize_fp4(1, P, K, 1, p(x), code, None, 0, E, k, p(off), p(tiles), p(place), codes, scales, s))
        done(lib.moe_dequantize_fp4(1, P, K, code, codes, scales, None, 0, E, p(off), p(tiles), 1, out(P * K * 2), s))
        w4 = moe.quantize_fp4(w, fmt)
        for act, od, size in ((0, 1, 2), (0, 0, 4), (1, 1, 2), (1, 0, 4)):
            done(lib.moe_grouped_matmul_fp4(P, E, N, K, code, codes, scales, None, p(w4.codes), p(w4.scales), None, 0, p(off), p(tiles), act, od,
                                            out(P * N // (1 + act) * size), None, None, None, s))
        og = -(-N // 2 // (64 if fmt == "nvfp4" else 128))
        done(lib.moe_grouped_matmul_fp4(P, E, N, K, code, codes, scales, None, p(w4.codes), p(w4.scales), None, 0, p(off), p(tiles), 1, 1, None,
                                        out(P * N // 4), out(n_tiles * og * 512), None, s))
    torch.cuda.synchronize()
    assert all(o.kept() for o in outs)
    moe.check_operators()
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    gr, (_, _, right, _) = moe.group_pairs(dev(ids), E), ref.groups(ids, E)
    got = host(moe.grouped_matmul(x[:T].contiguous(), w, gr, gather=True, out_dtype=torch.float32))
    want = np.einsum("pk,pnk->pn", host(x)[right // k].astype(np.float64), host(w).astype(np.float64)[ids.reshape(-1)[right]])
    assert distance(got, want) < 1e-6
