"""Cases of the 8-bit operators and of the norms around a block: quantisation by blocks of 128, products of 8-bit rows and
weights (one matrix, or grouped by expert), and the combine with post-norm, gate, residual and the next block's norm.

Each case names one operator and its sizes; `run` computes it in a plain form (32-bit torch operations) or, with `own` set,
through this package's public functions.  Shapes are the package's own workloads (DeepSeek-V3-shaped: top-8, H 7168, I 2048;
Qwen3-30B-A3B-shaped: E 128, top-8, H 2048, I 768) and odd sizes around them.

Formats.  Rows [R, K] in e4m3 with one fp32 scale for each 128 consecutive elements of a row, scales [ceil(K/128), R].  Weights
[N, K] (or a stack of them) in e4m3 with one fp32 scale for each 128 x 128 elements, scales [ceil(N/128), ceil(K/128)].  A
block's scale is a / 448, a its largest |x| but at least 2^-100, and its codes are those of 448 x / a.
"""
import math
import types

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
TINY = 2.0 ** -100
OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoded token's activations on their way into the shared expert: the smallest call, all latency
        dict(name="quantize8_one_token", op="quantize", of="rows", T=1, E=0, k=0, K=7168, N=0),
        # a prompt chunk's activations, each row stored for its eight experts
        dict(name="quantize8_prompt", op="quantize", of="rows", T=4096, E=256, k=8, K=7168, N=0),
        # a layer's gate/up weights from a bf16 checkpoint, 32 experts, an odd K (its last block is short)
        dict(name="quantize8_weights", op="quantize", of="weights", T=0, E=32, k=0, K=2000, N=4096),
        # one decoded token's gate/up product and SwiGLU: eight experts' weights stream past one row each
        dict(name="matmul8_one_token", op="matmul", T=1, E=64, k=8, K=7168, N=4096, act="swiglu", out="bf16"),
        # sixteen decoded tokens' down product
        dict(name="matmul8_batch16", op="matmul", T=16, E=128, k=8, K=768, N=2048, act="none", out="bf16"),
        # a prompt chunk's gate/up product with the SwiGLU behind it, one GPU's 32 experts
        dict(name="matmul8_prompt", op="matmul", T=2048, E=32, k=8, K=7168, N=4096, act="swiglu", out="bf16"),
        # the shared expert's down product of a ragged batch, one matrix, fp32 results
        dict(name="matmul8_shared_odd", op="matmul", T=1001, E=0, k=0, K=2048, N=7168, act="none", out="f32"),
        # the end of a block for one decoded token: combine, residual, next norm
        dict(name="norm_one_token", op="norm", T=1, E=256, k=8, N=7168, y="bf16", res="bf16", shared=True, post=False, gate="none", scale=1.0),
        # the same for a prompt chunk, with every part: shared rows, post-norm, channel gate, scaled residual
        dict(name="norm_prompt", op="norm", T=4096, E=256, k=8, N=7168, y="bf16", res="bf16", shared=True, post=True, gate="channel", scale=0.7071),
        # the end of a block that is no mixture: one row a token, odd sizes, fp32 stream, a gate for each token
        dict(name="norm_dense_odd", op="norm", T=333, E=0, k=0, N=1001, y="f32", res="f32", shared=False, post=True, gate="token", scale=1.0),
        # the whole 8-bit layer, router to next norm: one decoded token, and a prompt chunk
        dict(name="layer8_one_token", op="layer", T=1, E=128, k=8, H=2048, I=768),
        dict(name="layer8_prompt", op="layer", T=8192, E=128, k=8, H=2048, I=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, lo, hi):
    return _log(rng, lo, hi) | 1


def draw(rng):
    """One more case: tokens from one to a prompt chunk, experts from one to 256 or one matrix, even and odd sizes."""
    op = rng.choice(("quantize", "matmul", "matmul", "norm", "layer"))
    T = rng.choice((1, 16, _odd(rng, 1, 8191), _odd(rng, 1, 8191)))
    E = rng.choice((0, 8, 128, _log(rng, 1, 256)))
    k = min(E, rng.choice((1, 2, 6, 8)))
    if op == "quantize":
        K = rng.choice((768, 2048, 7168, 16 * _odd(rng, 1, 447)))
        if rng.random() < 0.6:
            while T * max(1, k) * K > 4096 * 8 * 7168:
                T = (T // 2) | 1
            return dict(op=op, of="rows", T=T, E=E, k=k, K=K, N=0)
        N = rng.choice((768, 8 * _odd(rng, 1, 255), _odd(rng, 1, 4095)))
        return dict(op=op, of="weights", T=0, E=max(1, min(E, 250_000_000 // (N * K))), k=0, K=K, N=N)
    if op == "norm":
        N = rng.choice((2048, 7168, 8 * _odd(rng, 2, 895), _odd(rng, 16, 8191)))
        while T * (k + 4) * N > 4096 * 12 * 7168:
            T = (T // 2) | 1
        return dict(op=op, T=T, E=E, k=k, N=N, y=rng.choice(("bf16", "bf16", "f32")), res=rng.choice(("bf16", "f32")), shared=E > 0 and rng.random() < 0.5,
                    post=rng.random() < 0.5, gate=rng.choice(("none", "channel", "token")), scale=rng.choice((1.0, round(rng.uniform(0.1, 1.5), 3))))
    if op == "layer":
        H, I = rng.choice(((2048, 768), (128 * _odd(rng, 1, 31), 64 * _odd(rng, 1, 23))))
        E = max(1, min(E or 1, 300_000_000 // (3 * H * I)))
        k = max(1, min(E, k))
        while T * k * 3 * H * I > 65536 * 3 * 2048 * 768:
            T = (T // 2) | 1
        return dict(op=op, T=T, E=E, k=k, H=H, I=I)
    act = rng.choice(("none", "swiglu"))
    K = rng.choice((768, 2048, 7168, 16 * _odd(rng, 1, 447)))
    N = rng.choice((1536, 4096, 128 * _odd(rng, 1, 31))) if act == "swiglu" else rng.choice((2048, 8 * _odd(rng, 4, 511), _odd(rng, 24, 4095)))
    E = max(min(E, 1), min(E, 1_000_000_000 // (N * K)))
    k = min(E, k)
    while T * max(1, k) * N * K > 16384 * 4096 * 7168:
        T = (T // 2) | 1
    return dict(op=op, T=T, E=E, k=k, K=K, N=N, act=act, out=rng.choice(("bf16", "bf16", "f32")))


def work(case):
    """Bytes and operations of one pass: each input once, each output once, the weights of the experts that T
    tokens with k distinct experts out of E reach on average."""
    c = types.SimpleNamespace(**case)
    P = c.T * max(1, c.k)
    seen = c.E * (1 - (1 - c.k / c.E) ** c.T) if c.E and c.T else max(1, c.E)
    if c.op == "quantize":
        rows, src = (P, c.T) if c.of == "rows" else (c.E * c.N, c.E * c.N)
        return {"bytes": 2 * src * c.K + rows * c.K * (1 + 2), "flops": 6 * rows * c.K}
    if c.op == "norm":
        wy, wr = (2 if c.y == "bf16" else 4), (2 if c.res == "bf16" else 4)
        return {"bytes": P * c.N * wy + (c.T * c.N * wy if c.shared else 0) + 2 * c.T * c.N * wr + 2 * c.T * c.N + 8 * P + 8 * c.N,
                "flops": (2 * max(1, c.k) + 10) * c.T * c.N}
    if c.op == "layer":
        n = 3 * c.H * c.I
        return {"bytes": 4 * c.T * c.E + 2 * c.T * c.H * 2 + seen * n + 2 * c.T * c.H * 2, "flops": 2 * P * n}
    cols = c.N // 2 if c.act == "swiglu" else c.N
    return {"bytes": P * c.K + seen * c.N * c.K + P * cols * (2 if c.out == "bf16" else 4), "flops": 2 * P * c.N * c.K}


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV) * std


def _logits(gen, T, E):
    """Router logits: spread over experts, some experts favoured by every token."""
    return _randn(gen, T, E) + _randn(gen, 1, E, std=0.5)


def _groups(logits, k):
    """Experts of each token, and the (token, expert) pairs in expert order."""
    ids = logits.sort(dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)
    offsets, tiles, order, place = _plain_groups(ids, logits.shape[1])
    return types.SimpleNamespace(E=logits.shape[1], k=k, ids=ids, offsets=offsets, tiles=tiles, order=order, place=place, most=int(offsets.diff().max()))


def _weights(gen, E, N, K):
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
    for part in w.split(max(1, (1 << 27) // (N * K))):
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * 0.02)
    return w


def _weights8(gen, E, N, K):
    """8-bit weights of E experts as a checkpoint has them: codes [E, N, K] and scales [E, ceil(N/128), ceil(K/128)]."""
    codes, scales = torch.empty(E, N, K, dtype=F8, device=DEV), []
    step = max(1, (1 << 27) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        c, s = _plain_quantize_weights(_weights(gen, n, N, K))
        codes[e:e + n] = c
        scales.append(s)
    return types.SimpleNamespace(codes=codes, scales=torch.cat(scales), E=E, N=N, K=K)


def prepare(case, seed):
    c = types.SimpleNamespace(**case)
    gen = _gen(seed)
    s = types.SimpleNamespace(c=c, groups=None)
    if c.op == "quantize" and c.of == "weights":
        s.w = _weights(gen, c.E, c.N, c.K)
        return s
    if c.op == "layer":
        s.x, s.h = _randn(gen, c.T, c.H).bfloat16(), _randn(gen, c.T, c.H).bfloat16()
        s.logits = _logits(gen, c.T, c.E)
        s.gu, s.down = _weights8(gen, c.E, 2 * c.I, c.H), _weights8(gen, c.E, c.H, c.I)
        s.pre = 1 + _randn(gen, c.H, std=0.1)
        s.most = _groups(s.logits, c.k).most
        return s
    if c.E:
        s.groups = _groups(_logits(gen, c.T, c.E), c.k)
    P = c.T * max(1, c.k)
    if c.op == "quantize":
        s.x = _randn(gen, c.T, c.K).bfloat16()
    elif c.op == "matmul":
        codes, scales = _plain_quantize_rows(_randn(gen, P, c.K).bfloat16())
        s.x = types.SimpleNamespace(codes=codes, scales=scales)
        s.w = _weights8(gen, max(1, c.E), c.N, c.K)
    elif c.op == "norm":
        s.y = _randn(gen, P, c.N).to(OUT[c.y])
        s.h = _randn(gen, c.T, c.N, std=2.0).to(OUT[c.res])
        s.shared = _randn(gen, c.T, c.N).to(OUT[c.y]) if c.shared else None
        s.post = 1 + _randn(gen, c.N, std=0.1) if c.post else None
        s.pre = 1 + _randn(gen, c.N, std=0.1)
        s.gate = None if c.gate == "none" else _randn(gen, c.N, std=0.5) if c.gate == "channel" else torch.rand(c.T, 1, generator=gen, device=DEV)
        w = torch.rand(c.T, max(1, c.k), generator=gen, device=DEV) + 0.05
        s.topk_w = w / w.sum(dim=1, keepdim=True)
    return s


# ---------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------
def _plain_route(logits, k):
    ids = logits.sort(dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.exp(logits - logits.amax(dim=1, keepdim=True)).gather(1, ids)
    return ids.to(torch.int32), p / p.sum(dim=1, keepdim=True)


def _plain_groups(ids, E):
    """Pairs (token-major) in expert order: where each expert starts, its first 128-row tile, the pair at each grouped
    row, and the grouped row of each pair."""
    flat = ids.reshape(-1).long()
    count = torch.zeros(E, dtype=torch.int32, device=ids.device).scatter_add(0, flat, torch.ones_like(flat, dtype=torch.int32))
    zero = torch.zeros(1, dtype=torch.int32, device=ids.device)
    offsets = torch.cat([zero, count.cumsum(0).to(torch.int32)])
    tiles = torch.cat([zero, ((count + 127) // 128).cumsum(0).to(torch.int32)])
    order = flat.sort(stable=True).indices
    place = torch.empty_like(order).scatter(0, order, torch.arange(order.numel(), device=ids.device))
    return offsets, tiles, order.to(torch.int32), place.to(torch.int32).view(ids.shape)


def _plain_codes(blocks, a):
    return (blocks * 448 / a).to(F8)


def _padded(x, rows, cols):
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % cols, 0, -x.shape[-2] % rows))


def _plain_quantize_rows(x):
    """Rows [R, K] -> codes [R, K], scales [ceil(K/128), R]."""
    R, K = x.shape
    xb = _padded(x.float(), 1, 128).view(R, -1, 128)
    a = xb.abs().amax(dim=2, keepdim=True).clamp(min=TINY)
    codes = _plain_codes(xb, a).view(R, -1)[:, :K].contiguous()
    return codes, (a[:, :, 0] * (1 / 448)).T.contiguous()


def _plain_quantize_weights(w):
    """Matrices [E, N, K] -> codes [E, N, K], scales [E, ceil(N/128), ceil(K/128)]."""
    E, N, K = w.shape
    wp = _padded(w.float(), 128, 128)
    wb = wp.view(E, wp.shape[1] // 128, 128, wp.shape[2] // 128, 128)
    a = wb.abs().amax(dim=(2, 4), keepdim=True).clamp(min=TINY)
    codes = _plain_codes(wb, a).view(E, wp.shape[1], wp.shape[2])[:, :N, :K].contiguous()
    return codes, a[:, :, 0, :, 0] * (1 / 448)


def _plain_rows(codes, scales):
    return codes.float() * scales.T.repeat_interleave(128, dim=1)[:, :codes.shape[1]]


def _plain_matrices(codes, scales):
    s = scales.repeat_interleave(128, dim=2)[:, :, :codes.shape[2]].repeat_interleave(128, dim=1)[:, :codes.shape[1]]
    return codes.float() * s


def _plain_matmul(x, w, offsets, most):
    """Rows [P, K] in expert order times w [E, N, K] of their expert, in 32 bits."""
    P, E = x.shape[0], w.shape[0]
    at = torch.arange(P, device=DEV)
    e = torch.searchsorted(offsets[1:].contiguous(), at.to(torch.int32), right=True)
    if P <= E:  # few rows: each with its own expert's matrix
        return torch.bmm(w[e], x.unsqueeze(2)).squeeze(2)
    rows = (offsets[:-1, None] + torch.arange(most, device=DEV)).clamp(max=P - 1)
    y = torch.bmm(x[rows.long()], w.transpose(1, 2))
    return y[e, at - offsets[e].long()]


def _plain_product(x, w, groups):
    wide = _plain_matrices(w.codes, w.scales)
    rows = _plain_rows(x.codes, x.scales)
    return rows @ wide[0].T if groups is None else _plain_matmul(rows, wide, groups.offsets, groups.most)


def _plain_swiglu(y):
    a, b = y.chunk(2, dim=1)
    return a / (1 + torch.exp(-a)) * b


def _plain_normed(x, weight, eps=1e-6):
    return x / torch.sqrt((x * x).mean(dim=1, keepdim=True) + eps) * weight


def _plain_block_end(y, place, topk_w, shared, post, gate, scale, h, pre):
    c = y.float() if place is None else (y.float()[place.long()] * topk_w[:, :, None]).sum(dim=1)
    if shared is not None:
        c = c + shared.float()
    if post is not None:
        c = _plain_normed(c, post)
    if gate is not None:
        c = c * gate
    out = scale * h.float() + c
    return {"h": out.to(h.dtype), "z": _plain_normed(out, pre).bfloat16()}


def _plain_layer(s):
    c = s.c
    ids, w = _plain_route(s.logits, c.k)
    offsets, tiles, order, place = _plain_groups(ids, c.E)
    groups = types.SimpleNamespace(offsets=offsets, most=s.most)
    one = lambda codes, scales: types.SimpleNamespace(codes=codes, scales=scales)  # noqa: E731
    x = one(*_plain_quantize_rows(s.x[order.long() // c.k]))
    h = one(*_plain_quantize_rows(_plain_swiglu(_plain_product(x, s.gu, groups))))
    y = _plain_product(h, s.down, groups)
    return _plain_block_end(y, place, w, None, None, None, 1.0, s.h, s.pre)


def _plain(s):
    c = s.c
    if c.op == "quantize" and c.of == "weights":
        return _plain_matrices(*_plain_quantize_weights(s.w)).bfloat16()
    if c.op == "quantize":
        x = s.x if s.groups is None else s.x[s.groups.order.long() // c.k]
        return _plain_rows(*_plain_quantize_rows(x)).bfloat16()
    if c.op == "matmul":
        y = _plain_product(s.x, s.w, s.groups)
        return (_plain_swiglu(y) if c.act == "swiglu" else y).to(OUT[c.out])
    if c.op == "norm":
        return _plain_block_end(s.y, s.groups.place if s.groups else None, s.topk_w, s.shared, s.post, s.gate, c.scale, s.h, s.pre)
    return _plain_layer(s)


# ---------------------------------------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------------------------------------
def _own(s):
    import serving_layer_moe_gb300 as moe
    c = s.c
    if c.op == "layer":
        gu, down = moe.FP8Weights(s.gu.codes, s.gu.scales), moe.FP8Weights(s.down.codes, s.down.scales)
        _, w, gr = moe.route(s.logits, c.k, groups=True)
        x = moe.quantize_fp8(s.x, groups=gr)
        h = moe.grouped_matmul_fp8(x, gu, gr, act="swiglu", quantize=True)
        y = moe.grouped_matmul_fp8(h, down, gr)
        out, z = moe.combine_norm(y, gr, w, s.h, pre=s.pre)
        return {"h": out, "z": z}
    if c.op == "quantize" and c.of == "weights":
        return moe.dequantize_fp8(moe.quantize_fp8_weights(s.w))
    g = s.groups
    gr = moe.ExpertGroups(g.offsets, g.tiles, g.order, g.place) if g else None
    if c.op == "quantize":
        return moe.dequantize_fp8(moe.quantize_fp8(s.x, groups=gr))
    if c.op == "matmul":
        x = moe.FP8Rows(s.x.codes, s.x.scales)
        if gr is None:
            return moe.matmul_fp8(x, moe.FP8Weights(s.w.codes[0], s.w.scales[0]), act=c.act, out_dtype=OUT[c.out])
        return moe.grouped_matmul_fp8(x, moe.FP8Weights(s.w.codes, s.w.scales), gr, act=c.act, out_dtype=OUT[c.out])
    more = dict(post=s.post, gate=s.gate, residual_scale=c.scale, pre=s.pre)
    out, z = moe.residual_norm(s.y, s.h, **more) if gr is None else moe.combine_norm(s.y, gr, s.topk_w, s.h, shared=s.shared, **more)
    return {"h": out, "z": z}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------
def _exact_e4m3(v):
    """Nearest e4m3 value of |v| <= 448 in 64 bits, ties to even: three bits below the leading one, none below 2^-9."""
    m = v.abs()
    ulp = torch.exp2(torch.floor(torch.log2(m.clamp(min=2.0 ** -6))) - 3)
    return torch.round(m / ulp) * ulp * torch.sign(v)


def _exact_blocks(x, high):
    """[..., N, K] in 64 bits -> the 8-bit values of its blocks of `high` rows and 128 columns."""
    N, K = x.shape[-2:]
    out = torch.empty_like(x)
    for i in range(0, N, high):
        for j in range(0, K, 128):
            b = x[..., i:i + high, j:j + 128]
            a = b.abs().amax(dim=(-2, -1), keepdim=True).clamp(min=TINY)
            out[..., i:i + high, j:j + 128] = _exact_e4m3(b * 448 / a) * (a / 448)
    return out


def _exact_rows8(x):
    """Each row's blocks of 128 columns, several rows at a time."""
    out = torch.empty_like(x)
    for j in range(0, x.shape[1], 128):
        b = x[:, j:j + 128]
        a = b.abs().amax(dim=1, keepdim=True).clamp(min=TINY)
        out[:, j:j + 128] = _exact_e4m3(b * 448 / a) * (a / 448)
    return out


def _exact_values(bits):
    """The values of e4m3 codes, from their bits."""
    u = torch.arange(256, device=DEV)
    man, ex = (u & 7).double(), ((u >> 3) & 15).double()
    v = torch.where(ex > 0, (8 + man) * torch.exp2(ex - 10), man * 2.0 ** -9) * torch.where(u > 127, -1.0, 1.0)
    return v[bits.view(torch.uint8).long()]


def _exact_decode(codes, scales, high):
    """codes [N, K] with scales [ceil(N/high), ceil(K/128)] of their blocks."""
    r, k = torch.arange(codes.shape[0], device=DEV) // high, torch.arange(codes.shape[1], device=DEV) // 128
    return _exact_values(codes) * scales.double()[r][:, k]


def _exact_product(x, w, offsets):
    """x [P, K] in 64 bits; the weights' values in 64 bits, one expert at a time."""
    o = offsets if offsets is not None else [0, x.shape[0]]
    return torch.cat([x[a:b] @ _exact_decode(w.codes[e], w.scales[e], 128).T for e, (a, b) in enumerate(zip(o, o[1:])) if b > a])


def _exact_swiglu(y):
    n = y.shape[1] // 2
    return y[:, :n] * torch.sigmoid(y[:, :n]) * y[:, n:]


def _exact_order(ids, E):
    flat = ids.reshape(-1).tolist()
    by = [[] for _ in range(E)]
    for p, e in enumerate(flat):
        by[e].append(p)
    order = [p for b in by for p in b]
    place = [0] * len(flat)
    for i, p in enumerate(order):
        place[p] = i
    offsets = [0]
    for b in by:
        offsets.append(offsets[-1] + len(b))
    return offsets, torch.tensor(order, device=DEV), torch.tensor(place, device=DEV).view(ids.shape)


def _exact_normed(x, weight):
    return x * torch.rsqrt(x.square().mean(dim=1, keepdim=True) + 1e-6) * weight.double()


def _exact_end(c, post, gate, scale, h, pre):
    if post is not None:
        c = _exact_normed(c, post)
    if gate is not None:
        c = c * gate.double()
    out = scale * h.double() + c
    return {"h": out, "z": _exact_normed(out, pre)}


def exact(case, seed):
    s = prepare(case, seed)
    c = s.c
    if c.op == "quantize" and c.of == "weights":
        return torch.stack([_exact_blocks(w.double(), 128) for w in s.w])
    if c.op == "quantize":
        x = s.x.double() if s.groups is None else s.x.double()[s.groups.order.long() // c.k]
        return _exact_rows8(x)
    if c.op == "matmul":
        x = _exact_decode(s.x.codes, s.x.scales.T, 1)
        y = _exact_product(x, s.w, s.groups.offsets.tolist() if s.groups else None)
        return _exact_swiglu(y) if c.act == "swiglu" else y
    if c.op == "layer":
        p = torch.softmax(s.logits.double(), dim=1)
        ids = torch.argsort(-s.logits.double(), dim=1, stable=True)[:, :c.k]
        w = p.gather(1, ids)
        w = w / w.sum(dim=1, keepdim=True)
        offsets, order, place = _exact_order(ids, c.E)
        x = _exact_rows8(s.x.double()[order // c.k])
        h = _exact_rows8(_exact_swiglu(_exact_product(x, s.gu, offsets)))
        y = _exact_product(h, s.down, offsets)
        return _exact_end(torch.einsum("tk,tkn->tn", w, y[place]), None, None, 1.0, s.h, s.pre)
    if s.groups is None:
        sums = s.y.double()
    else:
        sums = torch.zeros(c.T, c.N, dtype=torch.float64, device=DEV)
        for j in range(c.k):
            sums += s.topk_w[:, j, None].double() * s.y[s.groups.place[:, j].long()].double()
    if s.shared is not None:
        sums = sums + s.shared.double()
    return _exact_end(sums, s.post, s.gate, c.scale, s.h, s.pre)
