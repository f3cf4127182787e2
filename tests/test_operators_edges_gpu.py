"""The routed-expert operators on the GPU: refusals, special values and sizes, one case each."""
import numpy as np
import pytest
import torch

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
