"""The 8-bit operators and the end of a block on tensors of more than 2^31 elements: the last rows are those of a small call on them."""
import pytest
import torch

pytestmark = pytest.mark.gpu
T, N = 300_001, 8192                # 2.46e9 elements
LAST = slice(T - 5, T)


@pytest.fixture(scope="module")
def moe():
    import serving_layer_moe_gb300 as m
    return m


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def normal(*shape, dtype=torch.bfloat16):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.view(-1).split(1 << 28):
        part.normal_()
    return out


def bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def same_rows(moe, big, small, rows):
    """FP8Rows `small` are the rows `rows` of `big`."""
    assert torch.equal(bits(big.codes)[rows], bits(small.codes)) and torch.equal(big.scales[:, rows], small.scales)


def test_rows(moe):
    x = normal(T, N)
    q = moe.quantize_fp8(x)
    same_rows(moe, q, moe.quantize_fp8(x[LAST].contiguous()), LAST)
    del x
    small = moe.FP8Rows(q.codes[LAST].contiguous(), q.scales[:, LAST].contiguous())
    for t in (torch.bfloat16, torch.float32):
        assert torch.equal(moe.dequantize_fp8(q, out_dtype=t)[LAST], moe.dequantize_fp8(small, out_dtype=t))


def test_weights(moe):
    w = normal(40, N, N)
    q = moe.quantize_fp8_weights(w)
    last = moe.quantize_fp8_weights(w[39])
    assert torch.equal(bits(q.codes)[39], bits(last.codes)) and torch.equal(q.scales[39], last.scales)
    assert torch.equal(moe.dequantize_fp8(q)[39], moe.dequantize_fp8(last))


@pytest.mark.parametrize("form", ["one_matrix", "experts"])
def test_products(moe, form):
    """One matrix: pairs of CTAs.  1024 experts: single ones, and weights of 2^31 codes."""
    K, E = 256, 1 if form == "one_matrix" else 1024
    x, w = moe.quantize_fp8(normal(T, K)), moe.quantize_fp8_weights(normal(E, N, K))
    if E == 1:
        gr, expert, rows = None, 0, LAST
        wide = moe.FP8Weights(w.codes[0], w.scales[0])
    else:
        ids = torch.randint(0, E, (T, 1), device="cuda", dtype=torch.int32)
        ids[:5] = E - 1
        gr, expert, rows = moe.group_pairs(ids, E), E - 1, LAST
        wide = w
    last, one = moe.FP8Rows(x.codes[rows].contiguous(), x.scales[:, rows].contiguous()), moe.FP8Weights(w.codes[expert], w.scales[expert])

    def call(v, **kw):
        return moe.matmul_fp8(v, wide, **kw) if gr is None else moe.grouped_matmul_fp8(v, wide, gr, **kw)
    for t in (torch.bfloat16, torch.float32):
        assert torch.equal(call(x, out_dtype=t)[rows], moe.matmul_fp8(last, one, out_dtype=t))
    assert torch.equal(call(x, act="swiglu")[rows], moe.matmul_fp8(last, one, act="swiglu"))
    moe.check_operators()


def test_requantised_products(moe):
    x, w = moe.quantize_fp8(normal(T, 256)), moe.quantize_fp8_weights(normal(2 * N, 256))
    last = moe.FP8Rows(x.codes[LAST].contiguous(), x.scales[:, LAST].contiguous())
    same_rows(moe, moe.matmul_fp8(x, w, act="swiglu", quantize=True), moe.matmul_fp8(last, w, act="swiglu", quantize=True), LAST)
    moe.check_operators()


@pytest.mark.parametrize("width", [N, N - 1])
def test_the_end_of_a_block(moe, width):
    """Rows in shared memory's ring, and rows of any width; the last tokens' rows are anywhere among the pairs'.  A small call's means are
    summed in another order, by other threads, so this compares with 64 bits.  h: half a bf16 step and five roundings of parts below 10 in all (6e-7).
    z: those, and a mean whose sums round 2 log2 N + 24 times, 50 * 2^-24 = 3e-6 of z: below 1e-5 (1 + |z|)."""
    t, k = T // 2, 2
    ids = torch.randint(0, 64, (t, k), device="cuda", dtype=torch.int32)
    gr, y, w, h, pre = moe.group_pairs(ids, 64), normal(t * k, width), torch.rand(t, k, device="cuda"), normal(t, width), torch.rand(width, device="cuda")
    out, z = moe.combine_norm(y, gr, w, h, pre=pre, out_dtype=torch.float32)
    for rows in (slice(0, 5), slice(t - 5, t)):
        want = h[rows].double() + (w[rows, :, None].double() * y[gr.place[rows].long()].double()).sum(dim=1)
        assert torch.equal(out[rows], want.to(torch.bfloat16)) or ((out[rows].double() - want).abs() <= 2.0 ** -8 * want.abs() * (1 + 2.0 ** -10) + 1e-6).all()
        normed = want * (want.square().mean(dim=1, keepdim=True) + 1e-6).rsqrt() * pre.double()
        assert ((z[rows].double() - normed).abs() <= 1e-5 * (1 + normed.abs())).all()
    z = moe.rms_norm(out, pre, out_dtype=torch.float32)
    v = out[-5:].double()
    assert ((z[-5:].double() - v * (v.square().mean(dim=1, keepdim=True) + 1e-6).rsqrt() * pre.double()).abs() <= 1e-5 * (1 + v.abs())).all()
