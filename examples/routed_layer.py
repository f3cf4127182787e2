"""A 4-bit MoE layer from bf16 weights: quantise once, then route, multiply and combine prompt chunks and decoded tokens.

    python examples/routed_layer.py [--tokens 8192] [--hidden 2048] [--inter 768] [--experts 128] [--top-k 8] [--format nvfp4]
                                    [--rows bf16]

The layer is what a caller of MoECache.decode has for itself: a router in front (the ids and gates that decode takes), and,
for experts that all stay on the GPU, the whole layer on tensors it holds.  Prints how far the 4-bit layer is from the bf16 one
on the same weights, and the time of a prompt chunk and of one decoded token replayed from a CUDA graph.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import serving_layer_moe_gb300 as moe  # noqa: E402


class RoutedLayer:
    """One MoE layer: router [E, H] bf16, gate_up [E, 2 I, H] (gate rows, then up rows) and down [E, H, I] bf16.
    rows: the type of the experts' rows that combine adds up; fp32 rounds them less and moves twice the bytes."""

    def __init__(self, router, gate_up, down, top_k, fmt="nvfp4", rows=torch.bfloat16):
        self.router, self.gate_up, self.down, self.k, self.fmt, self.rows = router, gate_up, down, top_k, fmt, rows
        scale = moe.fp4_scale if fmt == "nvfp4" else (lambda w: None)
        self.gate_up4 = moe.quantize_fp4(gate_up, fmt, g=scale(gate_up))
        self.down4 = moe.quantize_fp4(down, fmt, g=scale(down))
        self.gx = self.gh = None

    def calibrate(self, x):
        """NVFP4: the matrix scales of the activations, from a sample of them."""
        if self.fmt != "nvfp4":
            return
        self.gx = moe.fp4_scale(x)
        _, _, groups = moe.route(x @ self.router.T, self.k, groups=True)
        h = moe.grouped_matmul(x, self.gate_up, groups, act="swiglu", gather=True)
        self.gh = moe.fp4_scale(h)

    def bf16(self, x):
        _, w, groups = moe.route(x @ self.router.T, self.k, groups=True)
        h = moe.grouped_matmul(x, self.gate_up, groups, act="swiglu", gather=True)
        return moe.combine(moe.grouped_matmul(h, self.down, groups, out_dtype=self.rows), groups, w, out_dtype=torch.bfloat16)

    def __call__(self, x):
        _, w, groups = moe.route(x @ self.router.T, self.k, groups=True)
        xq = moe.quantize_fp4(x, self.fmt, g=self.gx, groups=groups)
        h = moe.grouped_matmul_fp4(xq, self.gate_up4, groups, act="swiglu", quantize=True, g_out=self.gh)
        return moe.combine(moe.grouped_matmul_fp4(h, self.down4, groups, out_dtype=self.rows), groups, w, out_dtype=torch.bfloat16)


def milliseconds(call, n=20):
    for _ in range(3):
        call()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(n):
        call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def run(tokens=8192, hidden=2048, inter=768, experts=128, top_k=8, fmt="nvfp4", seed=0, rows="bf16"):
    """Build a layer with random weights, run it; {relative distance from bf16, ms a chunk, ms a token}."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(shape, generator=gen, device="cuda") * std).bfloat16()

    layer = RoutedLayer(normal(experts, hidden, std=hidden ** -0.5), normal(experts, 2 * inter, hidden, std=0.02),
                        normal(experts, hidden, inter, std=0.02), top_k, fmt, {"bf16": torch.bfloat16, "f32": torch.float32}[rows])
    x = normal(tokens, hidden, std=1.0)
    layer.calibrate(x[: min(tokens, 256)])
    want, got = layer.bf16(x).float(), layer(x).float()
    distance = ((got - want).norm() / want.norm()).item()
    chunk = milliseconds(lambda: layer(x))

    # a decode step: the input and output stay where the graph has them
    token = x[:1].clone()
    layer(token)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(token)
    graph.replay()
    step = milliseconds(graph.replay)
    # its rows are those of the chunk's first token
    assert torch.equal(out.float()[0], got[0]), "one token alone and in a chunk differ"
    moe.check_operators()
    return {"distance": distance, "chunk_ms": chunk, "token_ms": step}


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=8192)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inter", type=int, default=768)
    p.add_argument("--experts", type=int, default=128)
    p.add_argument("--top-k", type=int, default=8)
    p.add_argument("--format", choices=("nvfp4", "mxfp4"), default="nvfp4")
    p.add_argument("--rows", choices=("bf16", "f32"), default="bf16")
    a = p.parse_args()
    r = run(a.tokens, a.hidden, a.inter, a.experts, a.top_k, a.format, rows=a.rows)
    print(f"{a.format}: {r['distance']:.3f} from bf16, {r['chunk_ms'] * 1e3:.0f} us for {a.tokens} tokens, {r['token_ms'] * 1e3:.1f} us for one")
