"""Cases of the routed-expert operators: the router, 4-bit quantisation, expert-grouped products and the combine.

Each case names one operator and its sizes; `run` computes it in a plain form (32-bit torch operations) or,
with `own` set, through this package's public functions.  Shapes are the package's own workloads
(Qwen3-30B-A3B-shaped: E 128, top-8, H 2048, I 768; DeepSeek-V3-shaped: E 256, top-8, H 7168, I 2048) and odd
sizes around them.

Formats.  A 4-bit matrix is held as packed e2m1 codes [rows, K/2] (even element in the low nibble) and block
scales in tiles: rows in tiles of 128, blocks in groups of four, 512 bytes a (tile, group), the scale of row r,
block b at byte (r % 32) * 16 + (r / 32) * 4 + b of it.  NVFP4: one e4m3 scale per 16 elements and one fp32
scale per matrix; MXFP4: one e8m0 scale per 32 elements.  A ragged matrix starts each expert's rows on a new tile.
"""
import math
import types

import torch

own = False

DEV = "cuda"
BLOCK = {"nvfp4": 16, "mxfp4": 32}
F8 = torch.float8_e4m3fn
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoded token of the Qwen3-shaped model: the smallest call, all latency
        dict(name="route_one_token", op="route", T=1, E=128, k=8, scoring="softmax", groups=1, keep=1),
        # a prompt chunk through the DeepSeek-V3-shaped router: biased sigmoid scores, 4 of 8 expert groups
        dict(name="route_prompt_grouped", op="route", T=8192, E=256, k=8, scoring="sigmoid", groups=8, keep=4),
        # activations of a small ragged batch on their way into the 4-bit product, odd sizes, MX blocks
        dict(name="quantize_rows_odd", op="quantize", of="rows", fmt="mxfp4", T=77, E=60, k=6, K=1440, N=0),
        # a layer's gate/up weights from bf16 checkpoints to NVFP4, one matrix scale per expert
        dict(name="quantize_weights", op="quantize", of="weights", fmt="nvfp4", T=0, E=128, k=0, K=2048, N=1536),
        # one decoded token's gate/up product: eight experts' weights stream past one row each
        dict(name="matmul_one_token", op="matmul", T=1, E=128, k=8, K=2048, N=1536, act="none", out="bf16", gather=True),
        # a prompt chunk's gate/up product with the SwiGLU behind it, rows gathered by expert
        dict(name="matmul_prompt", op="matmul", T=8192, E=128, k=8, K=2048, N=1536, act="swiglu", out="bf16", gather=True),
        # sixteen decoded tokens' down product, 4-bit weights and activations
        dict(name="fp4_batch16", op="matmul_fp4", fmt="mxfp4", T=16, E=128, k=8, K=768, N=2048, act="none", out="bf16"),
        # a prompt chunk's gate/up product on one GPU's 32 of the DeepSeek-V3-shaped experts
        dict(name="fp4_prompt", op="matmul_fp4", fmt="nvfp4", T=2048, E=32, k=8, K=7168, N=4096, act="swiglu", out="bf16"),
        # odd sizes, fp32 out: the form whose output is the decode call's
        dict(name="combine_odd", op="combine", T=333, E=60, k=6, N=1000, out="f32"),
        # a prompt chunk at the DeepSeek-V3-shaped hidden size
        dict(name="combine_prompt", op="combine", T=4096, E=256, k=8, N=7168, out="bf16"),
        # the whole 4-bit layer, router to combine: one decoded token, and a prompt chunk
        dict(name="layer_one_token", op="layer", fmt="nvfp4", T=1, E=128, k=8, H=2048, I=768),
        dict(name="layer_prompt", op="layer", fmt="nvfp4", T=8192, E=128, k=8, H=2048, I=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, lo, hi):
    return _log(rng, lo, hi) | 1


def draw(rng):
    """One more case: tokens from one to a prompt chunk, experts from one to 256, even and odd sizes."""
    op = rng.choice(("route", "quantize", "matmul", "matmul_fp4", "combine", "layer"))
    T = rng.choice((1, 16, _odd(rng, 1, 8191), _odd(rng, 1, 8191)))
    E = rng.choice((8, 128, _log(rng, 1, 256)))
    k = min(E, rng.choice((1, 2, 6, 8)))
    fmt = rng.choice(("nvfp4", "mxfp4"))
    if op == "route":
        if rng.random() < 0.5:
            return dict(op=op, T=T, E=E, k=k, scoring="softmax", groups=1, keep=1)
        groups = rng.choice((1, 4, 8))
        E = groups * _log(rng, 2, 256 // groups)
        keep = rng.randint((groups + 1) // 2, groups)
        return dict(op=op, T=T, E=E, k=min(k, keep * (E // groups)), scoring="sigmoid", groups=groups, keep=keep)
    if op == "quantize":
        K = rng.choice((768, 2048, 32 * _odd(rng, 1, 223)))
        if rng.random() < 0.5:
            return dict(op=op, of="rows", fmt=fmt, T=T, E=E, k=k, K=K, N=0)
        N = rng.choice((768, 8 * _odd(rng, 1, 255), _odd(rng, 1, 2047)))
        E = max(1, min(E, 400_000_000 // (N * K)))
        return dict(op=op, of="weights", fmt=fmt, T=0, E=E, k=0, K=K, N=N)
    if op == "combine":
        N = rng.choice((2048, 8 * _odd(rng, 2, 895), _odd(rng, 16, 7167)))
        while T * k * N > 4096 * 8 * 7168:
            T = (T // 2) | 1
        return dict(op=op, T=T, E=E, k=k, N=N, out=rng.choice(("bf16", "f32")))
    if op == "layer":
        H, I = rng.choice(((2048, 768), (32 * _odd(rng, 3, 127), 32 * _odd(rng, 1, 47))))
        E = max(1, min(E, 300_000_000 // (3 * H * I)))
        k = min(E, k)
        while T * k * 3 * H * I > 65536 * 3 * 2048 * 768:
            T = (T // 2) | 1
        return dict(op=op, fmt=fmt, T=T, E=E, k=k, H=H, I=I)
    act = rng.choice(("none", "swiglu"))
    K = rng.choice((768, 2048, 32 * _odd(rng, 1, 127)))
    if op == "matmul":
        K = rng.choice((K, 8 * _odd(rng, 4, 511)))
    N = rng.choice((1536, 32 * _odd(rng, 1, 63))) if act == "swiglu" else rng.choice((2048, 8 * _odd(rng, 4, 255), _odd(rng, 24, 2047)))
    E = max(1, min(E, 400_000_000 // (N * K)))
    k = min(E, k)
    while T * k * N * K > 65536 * 1536 * 2048:
        T = (T // 2) | 1
    if op == "matmul":
        return dict(op=op, T=T, E=E, k=k, K=K, N=N, act=act, out=rng.choice(("bf16", "bf16", "f32")), gather=rng.random() < 0.5)
    return dict(op=op, fmt=fmt, T=T, E=E, k=k, K=K, N=N, act=act, out="bf16")


def work(case):
    """Bytes and operations of one pass: each input once, each output once, the weights of the experts that T
    tokens with k distinct experts out of E reach on average."""
    c = types.SimpleNamespace(**case)
    P = c.T * c.k
    seen = c.E * (1 - (1 - c.k / c.E) ** c.T) if c.T else c.E
    wide = {"nvfp4": 0.5 + 1 / 16, "mxfp4": 0.5 + 1 / 32}.get(getattr(c, "fmt", ""), 2)
    if c.op == "route":
        return {"bytes": 4 * c.T * c.E + 8 * P + 8 * P + 8 * (c.E + 1), "flops": 8 * c.T * c.E}
    if c.op == "quantize":
        rows, src = (P, c.T) if c.of == "rows" else (c.E * c.N, c.E * c.N)
        return {"bytes": 2 * src * c.K + wide * rows * c.K + 2 * rows * c.K, "flops": 6 * rows * c.K}
    if c.op == "combine":
        return {"bytes": 2 * P * c.N + 8 * P + c.T * c.N * (2 if c.out == "bf16" else 4), "flops": 2 * P * c.N}
    if c.op == "layer":
        n = 3 * c.H * c.I
        return {"bytes": 4 * c.T * c.E + 2 * c.T * c.H + seen * n * wide + 2 * c.T * c.H, "flops": 2 * P * n}
    cols = c.N // 2 if c.act == "swiglu" else c.N
    x = c.T * c.K * 2 if getattr(c, "gather", False) else P * c.K * wide
    return {"bytes": x + seen * c.N * c.K * wide + P * cols * (2 if c.out == "bf16" else 4), "flops": 2 * P * c.N * c.K}


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV) * std


def _sigmoid_margin(logits, bias, groups):
    """Least gap between any two biased scores of a row, and between any two group scores, in 64 bits."""
    s = torch.sigmoid(logits.double()) + bias.double()
    gap = s.sort(dim=1).values.diff(dim=1).amin(dim=1)
    if groups > 1:
        g = s.view(s.shape[0], groups, -1).topk(2, dim=2).values.sum(dim=2)
        gap = torch.minimum(gap, g.sort(dim=1).values.diff(dim=1).amin(dim=1))
    return gap


def _logits(gen, T, E):
    """Router logits: spread over experts, some experts favoured by every token."""
    return _randn(gen, T, E) + _randn(gen, 1, E, std=0.5)


def _groups(logits, k):
    """Experts of each token, and the (token, expert) pairs in expert order."""
    E = logits.shape[1]
    ids = logits.sort(dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)
    offsets, tiles, order, place = _plain_groups(ids, E)
    most = int(offsets.diff().max())
    return types.SimpleNamespace(E=E, k=k, ids=ids, offsets=offsets, tiles=tiles, order=order, place=place, most=most)


def _quantized(x, fmt, g, groups=None):
    """x [G, N, K] or ragged rows [P, K] as this package holds it: codes, scale tiles, and the matrix scales."""
    block, K = BLOCK[fmt], x.shape[-1]
    lead = x.shape[:-1]
    xb = x.reshape(-1, K // block, block)
    codes, scale = [], []
    for part in xb.split(max(1, (1 << 27) // K)):
        gp = g.reshape(1, 1) if g.numel() == 1 else None
        if gp is None:
            n = sum(c.shape[0] for c in scale)
            gp = g.repeat_interleave(x.shape[1])[n:n + part.shape[0], None]
        mag, step, sc = _plain_fp4(part.float(), fmt, gp)
        code = mag + 8 * torch.signbit(part).to(torch.uint8)
        code = code.view(part.shape[0], K)
        codes.append(code[:, 0::2] | (code[:, 1::2] << 4))
        scale.append(sc)
    codes, scale = torch.cat(codes), torch.cat(scale)
    nb = -(-(K // block) // 4)
    if groups is None:
        G = lead[0] if len(lead) > 1 else 1
        n = lead[-1]
        at = torch.arange(G * n, device=DEV)
        row = (at // n) * (-(-n // 128) * 128) + at % n
        nt = G * (-(-n // 128))
    else:
        P = lead[0]
        at = torch.arange(P, device=DEV)
        e = torch.searchsorted(groups.offsets[1:].contiguous(), at.to(torch.int32), right=True)
        row = groups.tiles[e].long() * 128 + at - groups.offsets[e]
        nt = (P + 127 * min(groups.E, P)) // 128
    pad = torch.zeros(nt * 128, nb * 4, dtype=torch.uint8, device=DEV)
    pad[row, : K // block] = scale
    tiles = pad.view(nt, 4, 32, nb, 4).permute(0, 3, 2, 1, 4).contiguous().view(nt, nb, 512)
    return codes.view(*lead, K // 2), tiles


def _weights(gen, E, N, K):
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
    for part in w.split(max(1, (1 << 27) // (N * K))):
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * 0.02)
    return w


def _weights_fp4(gen, fmt, E, N, K):
    """Quantised weights of E experts: codes, scale tiles, matrix scales."""
    codes, tiles, gs = [], [], []
    for e in range(0, E, max(1, (1 << 27) // (N * K))):
        w = _weights(gen, min(E - e, max(1, (1 << 27) // (N * K))), N, K)
        g = _plain_scale(w) if fmt == "nvfp4" else torch.ones(w.shape[0], device=DEV)
        c, t = _quantized(w, fmt, g)
        codes.append(c), tiles.append(t), gs.append(g)
    return types.SimpleNamespace(codes=torch.cat(codes), scales=torch.cat(tiles), g=torch.cat(gs), fmt=fmt, shape=(E, N, K))


def _calibrated(gen, top):
    """An activation's matrix scale as a model's calibration leaves it: the largest value seen, near `top`, onto 6 * 448."""
    return (top + torch.rand(1, generator=gen, device=DEV)) / 2688


def prepare(case, seed):
    c = types.SimpleNamespace(**case)
    gen = _gen(seed)
    s = types.SimpleNamespace(c=c)
    if c.op == "route":
        s.logits = _logits(gen, c.T, c.E)
        s.bias = None
        if c.scoring == "sigmoid":
            s.bias = _randn(gen, c.E, std=0.1)
            # rows whose order fp32 sigmoids cannot tell are drawn again: ids are compared as whole numbers
            for _ in range(6):
                close = _sigmoid_margin(s.logits, s.bias, c.groups) < 2e-6 if c.E > 1 else torch.zeros(c.T, dtype=torch.bool, device=DEV)
                s.logits = torch.where(close[:, None], _logits(gen, c.T, c.E), s.logits)
        return s
    if c.op == "quantize" and c.of == "weights":
        s.w = _weights(gen, c.E, c.N, c.K)
        return s
    if c.op == "layer":
        s.x = _randn(gen, c.T, c.H).bfloat16()
        s.logits = _logits(gen, c.T, c.E)
        s.gu = _weights_fp4(gen, c.fmt, c.E, 2 * c.I, c.H)
        s.down = _weights_fp4(gen, c.fmt, c.E, c.H, c.I)
        s.gx, s.gh = _calibrated(gen, 5.0), _calibrated(gen, 11.0)
        s.most = _groups(s.logits, c.k).most
        return s
    s.groups = _groups(_logits(gen, c.T, c.E), c.k)
    P = c.T * c.k
    if c.op == "quantize":
        s.x = _randn(gen, c.T, c.K).bfloat16()
        s.g = _calibrated(gen, 5.0) if c.fmt == "nvfp4" else torch.ones(1, device=DEV)
    elif c.op == "matmul":
        s.x = _randn(gen, c.T if c.gather else P, c.K).bfloat16()
        s.w = _weights(gen, c.E, c.N, c.K)
    elif c.op == "matmul_fp4":
        x = _randn(gen, P, c.K).bfloat16()
        g = _calibrated(gen, 5.0) if c.fmt == "nvfp4" else torch.ones(1, device=DEV)
        codes, tiles = _quantized(x, c.fmt, g, s.groups)
        s.x = types.SimpleNamespace(codes=codes, scales=tiles, g=g, fmt=c.fmt, shape=(P, c.K))
        s.w = _weights_fp4(gen, c.fmt, c.E, c.N, c.K)
    elif c.op == "combine":
        s.y = _randn(gen, P, c.N).bfloat16()
        w = torch.rand(c.T, c.k, generator=gen, device=DEV) + 0.05
        s.topk_w = w / w.sum(dim=1, keepdim=True)
    return s


# ---------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------
def _plain_route(logits, k, scoring, bias, groups, keep):
    logits = logits.float()
    if scoring == "softmax":
        pick, p = logits, torch.exp(logits - logits.amax(dim=1, keepdim=True))
    else:
        p = 1 / (1 + torch.exp(-logits))
        pick = p + bias
        if groups > 1:
            per = pick.view(pick.shape[0], groups, -1)
            score = per.sort(dim=2, descending=True).values[:, :, :2].sum(dim=2)
            best = score.sort(dim=1, descending=True, stable=True).indices[:, :keep]
            live = torch.zeros_like(score).scatter(1, best, 1.0) > 0
            pick = torch.where(live[:, :, None], per, torch.full_like(per, -math.inf)).view(pick.shape)
    ids = pick.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    return ids.to(torch.int32), w / w.sum(dim=1, keepdim=True)


def _plain_groups(ids, E):
    """Pairs (token-major) in expert order: where each expert starts, its first 128-row scale tile, the pair at
    each grouped row, and the grouped row of each pair."""
    flat = ids.reshape(-1).long()
    count = torch.zeros(E, dtype=torch.int32, device=ids.device).scatter_add(0, flat, torch.ones_like(flat, dtype=torch.int32))
    zero = torch.zeros(1, dtype=torch.int32, device=ids.device)
    offsets = torch.cat([zero, count.cumsum(0).to(torch.int32)])
    tiles = torch.cat([zero, ((count + 127) // 128).cumsum(0).to(torch.int32)])
    order = flat.sort(stable=True).indices
    place = torch.empty_like(order).scatter(0, order, torch.arange(order.numel(), device=ids.device))
    return offsets, tiles, order.to(torch.int32), place.to(torch.int32).view(ids.shape)


def _plain_scale(w):
    """The fp32 scale of each matrix of NVFP4 weights: the largest value onto 6 * 448."""
    top = w.float().abs().amax(dim=(1, 2))
    return torch.where(top > 0, top / 2688, torch.ones_like(top))


def _plain_fp4(xb, fmt, g):
    """Blocks [R, K/block, block] in 32 bits -> e2m1 magnitude codes, the value of one step, block scale codes."""
    top = xb.abs().amax(dim=2)
    if fmt == "nvfp4":
        sc = (top / 6 / g).clamp(max=448.0).to(F8)
        step = sc.float() * g
        bits = sc.view(torch.uint8)
    else:
        e = torch.where(top > 0, torch.frexp(top).exponent - 3, torch.zeros_like(top, dtype=torch.int32)).clamp(-127, 127)
        step = torch.ldexp(torch.ones_like(top), e)
        bits = (e + 127).to(torch.uint8)
    m = torch.where(step[:, :, None] > 0, xb / step[:, :, None], torch.zeros_like(xb)).abs()
    code = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5)
    return code, step, bits


def _plain_values(xb, fmt, g):
    """The 4-bit values that blocks [R, K/block, block] round to, as fp32 [R, K]."""
    code, step, _ = _plain_fp4(xb, fmt, g)
    table = torch.tensor(E2M1[:8], device=xb.device)
    return (table[code.int()] * torch.copysign(step[:, :, None], xb)).view(xb.shape[0], -1)


def _plain_untile(q, row):
    """Scale tiles -> the scale of each block of each row, as fp32."""
    nt, nb = q.scales.shape[:2]
    flat = q.scales.view(nt, nb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(nt * 128, nb * 4)
    K = q.codes.shape[-1] * 2
    bits = flat[row][:, : K // BLOCK[q.fmt]].contiguous()
    return bits.view(F8).float() if q.fmt == "nvfp4" else torch.ldexp(torch.ones_like(bits, dtype=torch.float32), bits.int() - 127)


def _plain_decode(q, row, g):
    """Codes [R, K/2] and tiled scales -> fp32 values [R, K]."""
    table = torch.tensor(E2M1, device=q.codes.device)
    codes = q.codes.reshape(-1, q.codes.shape[-1])
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], dim=2)
    sc = _plain_untile(q, row) * g
    return (v.view(codes.shape[0], -1, BLOCK[q.fmt]) * sc[:, :, None]).view(codes.shape[0], -1)


def _plain_decode_rows(q, offsets, tiles):
    at = torch.arange(q.codes.shape[0], device=DEV)
    e = torch.searchsorted(offsets[1:].contiguous(), at.to(torch.int32), right=True)
    return _plain_decode(q, tiles[e].long() * 128 + at - offsets[e], q.g.view(1, 1))


def _plain_decode_weights(q):
    E, N, K = q.shape
    at = torch.arange(E * N, device=DEV)
    row = (at // N) * (-(-N // 128) * 128) + at % N
    return _plain_decode(q, row, q.g.repeat_interleave(N)[:, None]).view(E, N, K)


def _plain_matmul(x, w, offsets, most):
    """Rows [P, K] in expert order times w [E, N, K] of their expert, in 32 bits."""
    P, E = x.shape[0], w.shape[0]
    at = torch.arange(P, device=DEV)
    e = torch.searchsorted(offsets[1:].contiguous(), at.to(torch.int32), right=True)
    if P <= E:  # few rows: each with its own expert's matrix
        return torch.bmm(w[e].float(), x.float().unsqueeze(2)).squeeze(2)
    rows = (offsets[:-1, None] + torch.arange(most, device=DEV)).clamp(max=P - 1)
    y = torch.bmm(x[rows.long()].float(), w.float().transpose(1, 2))
    return y[e, at - offsets[e].long()]


def _plain_swiglu(y):
    a, b = y.chunk(2, dim=1)
    return a / (1 + torch.exp(-a)) * b


def _plain_combine(y, place, topk_w):
    return (y.float()[place.long()] * topk_w[:, :, None]).sum(dim=1)


def _plain_layer(s):
    c = s.c
    ids, w = _plain_route(s.logits, c.k, "softmax", None, 1, 1)
    offsets, tiles, order, place = _plain_groups(ids, c.E)
    gx, gh = (s.gx, s.gh) if c.fmt == "nvfp4" else (torch.ones_like(s.gx), torch.ones_like(s.gh))
    x = s.x[order.long() // c.k].float()
    x = _plain_values(x.view(x.shape[0], -1, BLOCK[c.fmt]), c.fmt, gx.view(1, 1))
    h = _plain_swiglu(_plain_matmul(x, _plain_decode_weights(s.gu), offsets, s.most))
    h = _plain_values(h.view(h.shape[0], -1, BLOCK[c.fmt]), c.fmt, gh.view(1, 1))
    y = _plain_matmul(h, _plain_decode_weights(s.down), offsets, s.most)
    return _plain_combine(y, place, w).bfloat16()


def _plain(s):
    c = s.c
    if c.op == "route":
        ids, w = _plain_route(s.logits, c.k, c.scoring, s.bias, c.groups, c.keep)
        offsets, tiles, order, place = _plain_groups(ids, c.E)
        return {"ids": ids, "w": w, "offsets": offsets, "tiles": tiles, "order": order, "place": place}
    if c.op == "quantize":
        if c.of == "weights":
            g = _plain_scale(s.w) if c.fmt == "nvfp4" else torch.ones(c.E, device=DEV)
            v = _plain_values(s.w.float().view(-1, c.K // BLOCK[c.fmt], BLOCK[c.fmt]), c.fmt, g.repeat_interleave(c.N)[:, None])
            return v.bfloat16().view(c.E, c.N, c.K)
        x = s.x[s.groups.order.long() // c.k].float()
        return _plain_values(x.view(x.shape[0], -1, BLOCK[c.fmt]), c.fmt, s.g.view(1, 1)).bfloat16()
    if c.op == "combine":
        return _plain_combine(s.y, s.groups.place, s.topk_w).to(OUT[c.out])
    if c.op == "layer":
        return _plain_layer(s)
    if c.op == "matmul":
        x = s.x[s.groups.order.long() // c.k] if c.gather else s.x
        y = _plain_matmul(x, s.w, s.groups.offsets, s.groups.most)
    else:
        x = _plain_decode_rows(s.x, s.groups.offsets, s.groups.tiles)
        y = _plain_matmul(x, _plain_decode_weights(s.w), s.groups.offsets, s.groups.most)
    return (_plain_swiglu(y) if c.act == "swiglu" else y).to(OUT[c.out])


# ---------------------------------------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------------------------------------
def _own(s):
    import serving_layer_moe_gb300 as moe
    c = s.c
    if c.op == "route":
        ids, w, gr = moe.route(s.logits, c.k, scoring=c.scoring, bias=s.bias, n_group=c.groups, topk_group=c.keep, groups=True)
        return {"ids": ids, "w": w, "offsets": gr.offsets, "tiles": gr.tiles, "order": gr.order, "place": gr.place}
    if c.op == "layer":
        gx, gh = (s.gx, s.gh) if c.fmt == "nvfp4" else (None, None)
        gu = moe.FP4Rows(s.gu.codes, s.gu.scales, c.fmt, s.gu.g)
        down = moe.FP4Rows(s.down.codes, s.down.scales, c.fmt, s.down.g)
        _, w, gr = moe.route(s.logits, c.k, groups=True)
        x = moe.quantize_fp4(s.x, c.fmt, g=gx, groups=gr)
        h = moe.grouped_matmul_fp4(x, gu, gr, act="swiglu", quantize=True, g_out=gh)
        y = moe.grouped_matmul_fp4(h, down, gr)
        return moe.combine(y, gr, w, out_dtype=torch.bfloat16)
    if c.op == "quantize" and c.of == "weights":
        g = moe.fp4_scale(s.w) if c.fmt == "nvfp4" else None
        return moe.dequantize_fp4(moe.quantize_fp4(s.w, c.fmt, g=g))
    gr = moe.ExpertGroups(s.groups.offsets, s.groups.tiles, s.groups.order, s.groups.place)
    if c.op == "quantize":
        return moe.dequantize_fp4(moe.quantize_fp4(s.x, c.fmt, g=s.g if c.fmt == "nvfp4" else None, groups=gr))
    if c.op == "matmul":
        return moe.grouped_matmul(s.x, s.w, gr, act=c.act, gather=c.gather, out_dtype=OUT[c.out])
    if c.op == "matmul_fp4":
        x = moe.FP4Rows(s.x.codes, s.x.scales, c.fmt, s.x.g, gr)
        w = moe.FP4Rows(s.w.codes, s.w.scales, c.fmt, s.w.g)
        return moe.grouped_matmul_fp4(x, w, gr, act=c.act, out_dtype=OUT[c.out])
    return moe.combine(s.y, gr, s.topk_w, out_dtype=OUT[c.out])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------
def _exact_fp4(x, fmt, g):
    """[R, K] in 64 bits -> the 4-bit values of its rows; g: the matrix scale of each row, [R]."""
    grid = torch.tensor(E2M1[:8], dtype=torch.float64, device=DEV)
    out = torch.empty_like(x)
    for i in range(0, x.shape[0], 1 << 14):
        b = x[i:i + (1 << 14)].unflatten(1, (-1, BLOCK[fmt]))
        top = b.abs().amax(dim=2, keepdim=True)
        if fmt == "nvfp4":
            gd = g[i:i + (1 << 14), None, None]
            t = (top / (6 * gd)).clamp(max=448.0)
            # e4m3: three bits below the leading one, none below 2^-9
            ulp = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
            step = torch.round(t / ulp) * ulp * gd
        else:
            step = torch.exp2((torch.floor(torch.log2(top)) - 2).clamp(-127, 127))
            step = torch.where(top > 0, step, torch.ones_like(step))
        m = torch.where(step > 0, b.abs() / step, torch.zeros_like(b))
        # nearest value of the grid, ties to the even code: halves below 2, ones to 4, twos above
        ulp = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
        v = (torch.round(m / ulp) * ulp).clamp(max=float(grid[-1]))
        out[i:i + (1 << 14)] = (v * step * torch.sign(b)).flatten(1)
    return out


def _exact_decode(q, rows):
    """Each code by the table, each scale by its place in the tiles; rows: the padded row of each row."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    codes = q.codes.reshape(rows.numel(), -1)
    K = codes.shape[1] * 2
    b = torch.arange(K // BLOCK[q.fmt], device=DEV)
    nt, nb = q.scales.shape[:2]
    r = rows[:, None] % 128
    at = ((rows[:, None] // 128) * nb + b // 4) * 512 + (r % 32) * 16 + (r // 32) * 4 + b % 4
    bits = q.scales.reshape(-1)[at]
    if q.fmt == "nvfp4":
        man, ex = (bits & 7).double(), (bits >> 3).double()
        sc = torch.where(ex > 0, (8 + man) * torch.exp2(ex - 10), man * 2.0 ** -9)
    else:
        sc = torch.exp2(bits.double() - 127)
    v = torch.empty(codes.shape[0], K, dtype=torch.float64, device=DEV)
    v[:, 0::2], v[:, 1::2] = grid[(codes % 16).long()], grid[(codes // 16).long()]
    return v * sc.repeat_interleave(BLOCK[q.fmt], dim=1)


def _exact_product(x, weight, offsets):
    """x [P, K] in 64 bits, weight(e) -> [N, K] in 64 bits."""
    o = offsets.tolist()
    return torch.cat([x[a:b] @ weight(e).T for e, (a, b) in enumerate(zip(o, o[1:])) if b > a])


def _exact_weight(q):
    E, N, K = q.shape

    def weight(e):
        nt = -(-N // 128)
        one = types.SimpleNamespace(codes=q.codes[e], scales=q.scales[e * nt:(e + 1) * nt], fmt=q.fmt)
        return _exact_decode(one, torch.arange(N, device=DEV)) * q.g[e].double()
    return weight


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
    offsets, tiles = [0], [0]
    for b in by:
        offsets.append(offsets[-1] + len(b))
        tiles.append(tiles[-1] + -(-len(b) // 128))
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return whole(offsets), whole(tiles), whole(order), whole(place).view(ids.shape)


def _exact_route(logits, k, scoring, bias, groups, keep):
    z = logits.double()
    p = torch.softmax(z, dim=1) if scoring == "softmax" else torch.sigmoid(z)
    # fp32 logits order the softmax; equal ones go to the lower index
    pick = z if scoring == "softmax" else p + bias.double()
    if groups > 1:
        per = pick.unflatten(1, (groups, -1))
        score = per.topk(2, dim=2).values.sum(dim=2)
        cut = score.topk(keep, dim=1).values[:, -1:]
        pick = per.masked_fill((score < cut)[:, :, None], -math.inf).flatten(1)
    ids = torch.argsort(-pick, dim=1, stable=True)[:, :k]
    w = p.gather(1, ids)
    return ids.to(torch.int32), w / w.sum(dim=1, keepdim=True)


def exact(case, seed):
    s = prepare(case, seed)
    c = s.c
    if c.op == "route":
        ids, w = _exact_route(s.logits, c.k, c.scoring, s.bias, c.groups, c.keep)
        offsets, tiles, order, place = _exact_order(ids, c.E)
        return {"ids": ids, "w": w, "offsets": offsets, "tiles": tiles, "order": order, "place": place}
    if c.op == "quantize" and c.of == "weights":
        out = torch.empty(c.E, c.N, c.K, dtype=torch.float64, device=DEV)
        for e in range(c.E):
            w = s.w[e].double()
            # the matrix scale is held in 32 bits
            g = (w.abs().max() / 2688).float().double() if c.fmt == "nvfp4" else torch.ones((), dtype=torch.float64, device=DEV)
            out[e] = _exact_fp4(w, c.fmt, g.expand(c.N))
        return out
    if c.op == "layer":
        ids, w = _exact_route(s.logits, c.k, "softmax", None, 1, 1)
        offsets, _, order, place = _exact_order(ids, c.E)
        one = lambda g: (g if c.fmt == "nvfp4" else torch.ones_like(g)).double().expand(c.T * c.k)  # noqa: E731
        x = _exact_fp4(s.x.double()[order.long() // c.k], c.fmt, one(s.gx))
        h = _exact_fp4(_exact_swiglu(_exact_product(x, _exact_weight(s.gu), offsets)), c.fmt, one(s.gh))
        y = _exact_product(h, _exact_weight(s.down), offsets)
        return torch.einsum("tk,tkn->tn", w, y[place.long()])
    gr = s.groups
    if c.op == "quantize":
        return _exact_fp4(s.x.double()[gr.order.long() // c.k], c.fmt, s.g.double().expand(c.T * c.k))
    if c.op == "combine":
        out = torch.zeros(c.T, c.N, dtype=torch.float64, device=DEV)
        for j in range(c.k):
            out += s.topk_w[:, j, None].double() * s.y[gr.place[:, j].long()].double()
        return out
    if c.op == "matmul":
        x = s.x.double()[gr.order.long() // c.k] if c.gather else s.x.double()
        y = _exact_product(x, lambda e: s.w[e].double(), gr.offsets)
    else:
        o = gr.offsets.tolist()
        rows = torch.cat([torch.arange(b - a, device=DEV) + 128 * t for a, b, t in zip(o, o[1:], gr.tiles.tolist())])
        y = _exact_product(_exact_decode(s.x, rows) * s.x.g.double(), _exact_weight(s.w), gr.offsets)
    return _exact_swiglu(y) if c.act == "swiglu" else y
