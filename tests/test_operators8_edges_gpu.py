"""The 8-bit operators and the end of a block on the GPU: many experts, strange groups, other streams, odd memory, one case each."""
import copy

import numpy as np
import pytest
import torch

from tests import operators8_reference as ref8
from tests import operators_reference as ref
from tests.test_operators8_gpu import block, check_quantized, codes_of, end_within, operands, product, swiglu_within, to8, whole
from tests.test_operators_edges_gpu import Guarded, strange_groups
from tests.test_operators_gpu import bf16, dev, host
from tests.test_operators_many_items_gpu import grouping

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import serving_layer_moe_gb300 as m
    return m


@pytest.mark.parametrize("E,most,N,K", [(255, 3, 128, 144), (256, 9, 256, 272), (257, 9, 256, 272), (1000, 3, 128, 144), (4096, 1, 128, 128), (300, 700, 128, 128)])
def test_many_experts(moe, E, most, N, K):
    """On both sides of 256 experts, and as many as there may be; the last one with pairs of CTAs."""
    rng = np.random.default_rng(E)
    counts = rng.integers(0, most + 1, E)
    counts[rng.integers(0, E)] = 300
    if most == 700:
        counts += 384
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts.tolist())
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    xs = xs / 8
    y = product(xc, xs, wc, ws, offsets)
    x, w = operands(moe, xc, xs, wc, ws)
    assert np.array_equal(host(moe.grouped_matmul_fp8(x, w, gr, out_dtype=torch.float32)), y)
    assert np.array_equal(host(moe.grouped_matmul_fp8(x, w, gr)), bf16(y))
    y = y.astype(np.float64)
    swiglu_within(host(moe.grouped_matmul_fp8(x, w, gr, act="swiglu")), y, torch.bfloat16)
    check_quantized(moe.grouped_matmul_fp8(x, w, gr, act="swiglu", quantize=True), y)
    moe.check_operators()


@pytest.mark.parametrize("E,counts,N,K", [(1500, [1] * 60 + [0] * 1380 + [3] * 60, 512, 2048), (4096, [0] * 4040 + [2] * 56, 256, 1040), (1500, [0] * 1492 + [300] * 8, 640, 1936)])
def test_many_experts_and_many_slices(moe, E, counts, N, K):
    """The experts' table leaves room for three stages, an odd number, for two warps, and the weights come from memory."""
    rng = np.random.default_rng(E + N)
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    used = np.array(counts) > 0
    xc, xs, few, scales = whole(rng, P, int(used.sum()), N, K)
    xs = xs / 8
    y = product(xc, xs, few, scales, np.concatenate([[0], np.cumsum(np.array(counts)[used])]))
    wc, ws = np.zeros((E, *few.shape[1:]), few.dtype), np.ones((E, *scales.shape[1:]), scales.dtype)
    wc[used], ws[used] = few, scales
    x, w = operands(moe, xc, xs, wc, ws)
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(8):
        big.zero_()   # the weights are in memory, not in the cache
        assert np.array_equal(host(moe.grouped_matmul_fp8(x, w, gr, out_dtype=torch.float32)), y)
    check_quantized(moe.grouped_matmul_fp8(x, w, gr, act="swiglu", quantize=True), y.astype(np.float64))
    moe.check_operators()


@pytest.mark.parametrize("N", [7, 24, 130, 136, 257, 1000])
@pytest.mark.parametrize("counts", [[900, 1], [5, 0, 31]])
def test_widths_of_results(moe, N, counts):
    """Rows of results that start on 16 bytes or anywhere, whole and ragged tiles of tokens, both kinds of tiles."""
    rng = np.random.default_rng(N)
    K = 272
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    y = product(xc, xs, wc, ws, offsets)
    x, w = operands(moe, xc, xs, wc, ws)
    for out in (torch.float32, torch.bfloat16):
        assert np.array_equal(host(moe.grouped_matmul_fp8(x, w, gr, out_dtype=out)), y if out == torch.float32 else bf16(y))


@pytest.mark.parametrize("kind", ["random", "larger", "falling", "edges"])
@pytest.mark.parametrize("P,E", [(96, 40), (4800, 3), (640, 300)])
def test_no_groups_lead_outside_the_arrays(moe, kind, P, E):
    """Offsets and places that are no grouping: wrong results, nothing read or written elsewhere, and the next call right."""
    from serving_layer_moe_gb300.operators import _operators
    lib, s = _operators(), torch.cuda.current_stream().cuda_stream
    rng = np.random.default_rng(P + E)
    k, N, K = 2, 256, 144
    T = P // k
    off, _, _, place = (dev(a) for a in strange_groups(kind, P, E, rng))
    x, y, res, gates = torch.randn(T, K, device="cuda").bfloat16(), torch.randn(P, N, device="cuda"), torch.randn(T, N, device="cuda"), torch.rand(T, k, device="cuda")
    pre = torch.ones(N, device="cuda")
    w = moe.quantize_fp8_weights(torch.randn(E, N, K, device="cuda").bfloat16())
    outs = []

    def out(n):
        outs.append(Guarded((n + 15) // 16 * 16))
        return outs[-1].at

    p = lambda t: t.data_ptr()  # noqa: E731
    codes, scales = out(P * K), out(P * 2 * 4)
    done = lambda st: (_ for _ in ()).throw(AssertionError(lib.moe_last_error())) if st else None  # noqa: E731
    done(lib.moe_quantize_fp8(T, K, 1, p(x), k, p(place), codes, scales, s))
    for act in (0, 1):
        for od, size in ((0, 4), (1, 2)):
            done(lib.moe_grouped_matmul_fp8(P, E, N, K, codes, scales, p(w.codes), p(w.scales), p(off), act, od, out(P * N // (1 + act) * size), None, None, s))
    done(lib.moe_grouped_matmul_fp8(P, E, N, K, codes, scales, p(w.codes), p(w.scales), p(off), 1, 1, None, out(P * N // 2), out(P * 4), s))
    done(lib.moe_combine_norm(T, k, N, 0, p(y), p(place), p(gates), None, 0, None, 0, None, 1.0, 0, p(res), 0, p(pre), 1e-6, out(T * N * 4), 1, out(T * N * 2), s))
    torch.cuda.synchronize()
    assert all(o.kept() for o in outs)
    moe.check_operators()
    counts = [P // E] * E
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    assert np.array_equal(host(moe.grouped_matmul_fp8(*operands(moe, xc, xs, wc, ws), gr, out_dtype=torch.float32)), product(xc, xs, wc, ws, offsets))


@pytest.mark.parametrize("T,k,N", [(310, 30, 256), (310, 31, 256), (310, 40, 264), (5, 40, 256), (320, 2, 8), (320, 1, 4096), (305, 2, 4104), (305, 3, 8192), (305, 3, 8200)])
def test_combine_norm_on_both_sides_of_its_forms(moe, T, k, N):
    """30 rows and 8192 columns are what the form for many tokens takes."""
    rng = np.random.default_rng(T + k + N)
    E = 16
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)
    gr, (_, _, _, place) = moe.group_pairs(dev(ids), E), ref.groups(ids, E)
    r = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    for yt, rt in ((torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
        y, w, res, sh = bf16(r(T * k, N)), r(T, k), bf16(r(T, N)), bf16(r(T, N))
        post, pre, gate = 1 + r(N) / 8, 1 + r(N) / 8, r(N)
        for kw in (dict(pre=pre), dict(shared=sh, post=post, gate=gate, pre=pre), dict(post=post), dict()):
            h, z, mh, mz = ref8.block_end(y, place, w, res, **kw)
            got = moe.combine_norm(dev(y, yt), gr, dev(w), dev(res, rt), out_dtype=torch.float32, **{n: dev(v, yt if n == "shared" else None) for n, v in kw.items()})
            gh, gz = got if z is not None else (got, None)
            end_within(host(gh), h, mh, k, N, rt, "post" in kw)
            if z is not None:
                end_within(host(gz), z, mz + np.abs(z), k, N, torch.float32, 2)


@pytest.mark.parametrize("T,N", [(304, 8), (310, 2056), (350, 7168), (306, 8192), (303, 2048)])
def test_many_dense_rows(moe, T, N):
    """A row a token, as many tokens as the form for many of them takes and one fewer, with and without each part."""
    rng = np.random.default_rng(T + N)
    r = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    y, res, post, pre, gate, gate_t = bf16(r(T, N)), bf16(r(T, N)), 1 + r(N) / 8, bf16(1 + r(N) / 8), r(N), r(T, 1)
    for yt, rt in ((torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
        for kw in (dict(post=post, gate=gate, pre=pre), dict(post=post, gate=gate_t, pre=pre), dict(post=post), dict(post=pre, pre=post), dict(gate=gate, pre=pre)):
            h, z, mh, mz = ref8.block_end(y, None, None, res, scale=0.5, **kw)
            got = moe.residual_norm(dev(y, yt), dev(res, rt), residual_scale=0.5, out_dtype=torch.float32, **{n: dev(v, torch.bfloat16 if v is pre else None) for n, v in kw.items()})
            gh, gz = got if z is not None else (got, None)
            end_within(host(gh), h, mh, 1, N, rt, "post" in kw)
            if z is not None:
                end_within(host(gz), z, mz + np.abs(z), 1, N, torch.float32, 2)


def test_the_stream_may_be_updated_in_place(moe):
    """The C call's h is the residual itself: rows of other tokens are read before or after, never half way."""
    from serving_layer_moe_gb300.operators import _operators
    lib, s = _operators(), torch.cuda.current_stream().cuda_stream
    for T, N in ((1, 7168), (1000, 2048), (700, 1001)):
        y, res, pre = torch.randn(T, N, device="cuda").bfloat16(), torch.randn(T, N, device="cuda"), torch.ones(N, device="cuda")
        h, z = moe.residual_norm(y, res, pre=pre)
        z2 = torch.empty_like(z)
        assert lib.moe_combine_norm(T, 1, N, 1, y.data_ptr(), None, None, None, 0, None, 0, None, 1.0, 0, res.data_ptr(), 0, pre.data_ptr(), 1e-6, res.data_ptr(), 1, z2.data_ptr(), s) == 0
        assert torch.equal(res, h) and torch.equal(z2, z)


def test_calls_on_a_stream_of_their_own(moe):
    """stream= and torch's current stream: everything of a call, its memory too, is that stream's."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, E, k, H, I = 50, 8, 2, 256, 128
    x, logits, res = torch.randn(T, H, device="cuda", generator=gen).bfloat16(), torch.randn(T, E, device="cuda", generator=gen), torch.randn(T, H, device="cuda", generator=gen)
    gu, dn = torch.randn(E, 2 * I, H, device="cuda", generator=gen).bfloat16(), torch.randn(E, H, I, device="cuda", generator=gen).bfloat16()
    one = torch.ones(H, device="cuda")

    def layer(**on):
        _, w, gr = moe.route(logits, k, groups=True, **on)
        g, d = moe.quantize_fp8_weights(gu, **on), moe.quantize_fp8_weights(dn, **on)
        a = moe.grouped_matmul_fp8(moe.quantize_fp8(x, groups=gr, **on), g, gr, act="swiglu", quantize=True, **on)
        h, z = moe.combine_norm(moe.grouped_matmul_fp8(a, d, gr, **on), gr, w, res, pre=one, **on)
        return h, z, moe.residual_norm(z, h, **on), moe.rms_norm(h, one, **on), moe.matmul_fp8(moe.quantize_fp8(z, **on), moe.FP8Weights(g.codes[0], g.scales[0]), **on), moe.dequantize_fp8(a, **on)

    want = layer()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for got in (layer(stream=s), layer(stream=s.cuda_stream)):
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(s):
        got = layer()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_captured_graphs_and_eager_calls_share_nothing(moe):
    """Replays on two streams at once, with eager calls beside them."""
    calls = [block(moe, T, 8, 2, 512, 256, seed=i)[0] for i, T in enumerate((3, 400, 64))]
    want = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = calls[2]()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for got, w in zip((*outs, eager), want) for a, b in zip(got, w))
    moe.check_operators()


def test_copies_resized_and_misaligned_blocks(moe):
    rng = np.random.default_rng(1)
    counts, N, K = [9, 30, 1], 256, 272
    gr, (offsets, _, _, _), P, E, _ = grouping(moe, rng, counts)
    xc, xs, wc, ws = whole(rng, P, E, N, K)
    x, w = operands(moe, xc, xs, wc, ws)
    want = moe.grouped_matmul_fp8(x, w, gr)
    x2, w2 = copy.deepcopy((x, w))
    x.codes.view(torch.uint8).zero_()
    w.scales.zero_()
    assert torch.equal(moe.grouped_matmul_fp8(x2, w2, gr), want)
    room = torch.zeros(P * K + 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="16-byte"):
        moe.FP8Rows(room[8:8 + P * K].view(P, K), x2.scales)
    with pytest.raises(ValueError, match="16-byte"):
        moe.quantize_fp8(torch.zeros(P * 32 + 8, device="cuda", dtype=torch.bfloat16)[4:4 + P * 32].view(P, 32))
    codes = to8(wc)
    v = moe.FP8Weights(codes, w2.scales)
    codes.resize_(2, N, K)
    with pytest.raises(ValueError, match="scales"):
        moe.grouped_matmul_fp8(x2, v, gr)
    with pytest.raises(ValueError, match="16-byte"):
        moe.rms_norm(torch.zeros(65, device="cuda")[1:].view(1, 64), torch.ones(64, device="cuda"))
    odd = torch.randn(64, device="cuda")[1:].view(1, 63)          # rows of 63 start anywhere
    assert torch.equal(moe.rms_norm(odd, torch.ones(63, device="cuda")), moe.rms_norm(odd.clone(), torch.ones(63, device="cuda")))


def test_small_results_share_memory_and_large_ones_do_not(moe):
    one = torch.ones(2048, device="cuda")
    h, z = moe.residual_norm(torch.ones(4, 2048, device="cuda"), torch.ones(4, 2048, device="cuda"), pre=one)
    assert h.untyped_storage().data_ptr() == z.untyped_storage().data_ptr() and h.is_contiguous() and z.is_contiguous()
    h, z = moe.residual_norm(torch.ones(400, 2048, device="cuda"), torch.ones(400, 2048, device="cuda"), pre=one)
    assert h.untyped_storage().nbytes() == 400 * 2048 * 4 and z.untyped_storage().nbytes() == 400 * 2048 * 2
