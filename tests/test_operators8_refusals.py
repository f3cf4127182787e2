"""What the 8-bit operators and the end of a block refuse (no GPU needed: arguments are checked before any CUDA call)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from tests.test_operators_refusals import BF16, F32, NVFP4, ROOT, refused

P = ctypes.c_void_p
A, B, C, D, F, G, H = (P(0x10000 * i) for i in range(1, 8))     # aligned addresses that nothing reads


@pytest.fixture(scope="module", autouse=True)
def built():
    from serving_layer_moe_gb300 import build as b
    if not (os.path.exists(b.LIB) and os.path.exists(b.HOST)):
        b.build()


@pytest.fixture(scope="module")
def lib():
    from serving_layer_moe_gb300 import operators
    return operators._operators()


def quantize(lib, T=4, K=64, dt=BF16, x=A, k=1, place=None, codes=B, scales=C):
    return lib.moe_quantize_fp8(T, K, dt, x, k, place, codes, scales, None)


@pytest.mark.parametrize("kw,word", [
    (dict(K=24), b"multiple of 16"), (dict(K=0), b"multiple of 16"), (dict(K=(1 << 24) + 16), b"2^24"), (dict(T=-1), b"negative"), (dict(dt=NVFP4), b"dtype"),
    (dict(k=2), b"1 without place"), (dict(k=0, place=D), b"k >= 1"), (dict(T=1 << 30, k=4, place=D), b"rows are needed"), (dict(x=None), b"NULL"), (dict(codes=None), b"NULL"),
    (dict(x=P(0x10008)), b"16-byte"), (dict(codes=P(0x10008)), b"16-byte"), (dict(scales=P(0x10002)), b"4-byte"), (dict(k=2, place=P(0x10002)), b"4-byte")])
def test_quantize_refuses(lib, kw, word):
    refused(lib, quantize(lib, **kw), word)


@pytest.mark.parametrize("args,word", [
    ((1, 4, 40, BF16, A, B, C), b"multiple of 16"), ((-1, 4, 64, BF16, A, B, C), b"negative"), ((70000, 4, 64, BF16, A, B, C), b"65535"), ((1, -4, 64, BF16, A, B, C), b"negative"),
    ((1, 4, 64, 7, A, B, C), b"dtype"), ((1, 4, 64, F32, None, B, C), b"NULL"), ((1, 4, 64, F32, P(0x10004), B, C), b"16-byte"), ((1, 4, 64, F32, A, B, P(0x10002)), b"4-byte"),
    ((1, 0x7fffffff, 1 << 24, BF16, A, B, C), b"too many blocks")])
def test_quantize_weights_refuses(lib, args, word):
    refused(lib, lib.moe_quantize_fp8_weights(*args, None), word)


@pytest.mark.parametrize("args,word", [
    ((1, 4, 40, 0, A, B, BF16, C), b"multiple of 16"), ((2, 4, 64, 0, A, B, BF16, C), b"one matrix"), ((1, 4, 64, 1, A, B, NVFP4, C), b"dtype"), ((1, 4, 64, 1, A, None, BF16, C), b"NULL"),
    ((1, 4, 64, 1, A, B, BF16, P(0x10008)), b"16-byte")])
def test_dequantize_refuses(lib, args, word):
    refused(lib, lib.moe_dequantize_fp8(*args, None), word)


def matmul(lib, P_=8, E=2, N=128, K=64, xc=A, xs=B, wc=C, ws=D, off=F, act=0, od=BF16, out=G, oc=None, os_=None):
    return lib.moe_grouped_matmul_fp8(P_, E, N, K, xc, xs, wc, ws, off, act, od, out, oc, os_, None)


@pytest.mark.parametrize("kw,word", [
    (dict(P_=-1), b"P >= 0"), (dict(P_=0x7fffffff), b"at most"), (dict(E=0), b"E"), (dict(E=4097), b"4096"), (dict(N=0), b"N"), (dict(K=24), b"multiple of 16"), (dict(K=0), b"multiple of 16"), (dict(act=2), b"act"),
    (dict(act=1, N=192), b"multiple of 128"), (dict(od=3), b"out_dtype"), (dict(off=None), b"without offsets"), (dict(off=P(0x10002)), b"4-byte"), (dict(xc=None), b"NULL"), (dict(ws=None), b"NULL"),
    (dict(xc=P(0x10008)), b"16-byte"), (dict(wc=P(0x10004)), b"16-byte"), (dict(xs=P(0x10002)), b"4-byte"), (dict(out=P(0x10008)), b"16-byte"), (dict(out=None), b"act = 1"),
    (dict(out=None, act=1), b"out_codes"), (dict(out=None, act=1, oc=P(0x10008), os_=H), b"16-byte"), (dict(out=None, act=1, oc=A), b"out_scales")])
def test_matmul_refuses(lib, kw, word):
    refused(lib, matmul(lib, **kw), word)


def end(lib, T=4, k=2, N=64, yd=BF16, y=A, place=B, w=C, shared=None, pd=F32, post=None, rows=0, gate=None, alpha=1.0, rd=BF16, r=D, qd=F32, pre=F, eps=1e-6, h=G, zd=BF16, z=H):
    return lib.moe_combine_norm(T, k, N, yd, y, place, w, shared, pd, post, rows, gate, alpha, rd, r, qd, pre, eps, h, zd, z, None)


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), b"T >= 0"), (dict(k=0), b"k >= 1"), (dict(N=0), b"N"), (dict(N=32769), b"32768"), (dict(T=1 << 30, k=4), b"pairs"), (dict(yd=NVFP4), b"dtype"), (dict(rd=2), b"dtype"), (dict(zd=7), b"dtype"),
    (dict(eps=0.0), b"eps"), (dict(eps=-1.0), b"eps"), (dict(eps=float("nan")), b"eps"), (dict(eps=float("inf")), b"eps"), (dict(eps=1e-40), b"eps"), (dict(alpha=float("inf")), b"alpha"), (dict(alpha=float("nan")), b"alpha"),
    (dict(w=None), b"topk_w"), (dict(y=None), b"place needs"), (dict(place=None), b"k must be 1"), (dict(y=None, place=None, k=1, shared=A), b"need y"), (dict(y=None, place=None, k=1, gate=A), b"need y"),
    (dict(z=None), b"together"), (dict(pre=None), b"together"), (dict(pre=None, z=None, h=None), b"h or z"), (dict(r=None), b"residual"),
    (dict(y=P(0x10008)), b"aligned"), (dict(h=P(0x10004)), b"aligned"), (dict(post=P(0x10004)), b"aligned"), (dict(gate=P(0x10004)), b"aligned"), (dict(N=63, y=P(0x10001)), b"aligned"),
    (dict(N=63, rd=F32, r=P(0x10002)), b"aligned"), (dict(rows=1, gate=P(0x10002)), b"aligned"), (dict(place=P(0x10002)), b"4-byte")])
def test_combine_norm_refuses(lib, kw, word):
    refused(lib, end(lib, **kw), word)


def test_nothing_to_do_is_fine_without_memory(lib):
    assert quantize(lib, T=0, x=None, codes=None, scales=None) == 0
    assert lib.moe_quantize_fp8_weights(0, 4, 64, BF16, None, None, None, None) == 0 and lib.moe_quantize_fp8_weights(2, 0, 64, BF16, None, None, None, None) == 0
    assert lib.moe_dequantize_fp8(1, 0, 64, 0, None, None, BF16, None, None) == 0
    assert matmul(lib, P_=0, xc=None, xs=None, out=None) == 0
    assert end(lib, T=0, r=None) == 0


# The binding on tensors that say they are on a GPU and take no memory: what it refuses before any call, by name.
BINDING = """
import sys, torch
from torch._subclasses.fake_tensor import FakeTensorMode
import serving_layer_moe_gb300 as moe
moe.operators._host()
with FakeTensorMode(allow_non_fake_inputs=True):
    t = lambda *s, d=torch.bfloat16: torch.empty(*s, dtype=d, device="cuda")
    f32, f8, i32 = torch.float32, torch.float8_e4m3fn, torch.int32
    groups = lambda T=4, k=2, E=3: moe.ExpertGroups(t(E + 1, d=i32), t(E + 1, d=i32), t(T * k, d=i32), t(T, k, d=i32))
    rows = lambda R=8, K=64: moe.FP8Rows._of(t(R, K, d=f8), t(-(-K // 128), R, d=f32))
    weights = lambda *s: moe.FP8Weights._of(t(*s, d=f8), t(*s[:-2], -(-s[-2] // 128), -(-s[-1] // 128), d=f32))
    w, r = lambda: t(4, 2, d=f32), lambda: t(4, 64)
    calls = {
        "codes": lambda: moe.FP8Rows(t(8, 64), t(1, 8, d=f32)),
        "row_scales": lambda: moe.FP8Rows(t(8, 64, d=f8), t(8, 1, d=f32)),
        "row_K": lambda: moe.FP8Rows(t(8, 40, d=f8), t(1, 8, d=f32)),
        "weight_scales": lambda: moe.FP8Weights(t(2, 256, 64, d=f8), t(2, 1, 1, d=f32)),
        "weight_dims": lambda: moe.FP8Weights(t(64, d=f8), t(1, d=f32)),
        "quantize_K": lambda: moe.quantize_fp8(t(8, 40)),
        "quantize_type": lambda: moe.quantize_fp8(t(8, 64, d=torch.float16)),
        "quantize_groups": lambda: moe.quantize_fp8(t(8, 64), groups=groups()),
        "quantize_integers": lambda: moe.quantize_fp8(t(8, 64), groups=(0, 3, 8, 4, 2, 1, 2, 3, 4)),
        "weights_K": lambda: moe.quantize_fp8_weights(t(8, 40)),
        "weights_G": lambda: moe.quantize_fp8_weights(t(70000, 1, 16)),
        "dequantize": lambda: moe.dequantize_fp8(t(8, 64, d=f8)),
        "dequantize_type": lambda: moe.dequantize_fp8(rows(), out_dtype=torch.float16),
        "matmul_x": lambda: moe.matmul_fp8(t(8, 64), weights(128, 64)),
        "matmul_w": lambda: moe.matmul_fp8(rows(), rows()),
        "matmul_stack": lambda: moe.matmul_fp8(rows(), weights(3, 128, 64)),
        "matmul_K": lambda: moe.matmul_fp8(rows(), weights(128, 80)),
        "matmul_N": lambda: moe.matmul_fp8(rows(), weights(0, 64)),
        "matmul_act": lambda: moe.matmul_fp8(rows(), weights(128, 64), act="gelu"),
        "matmul_swiglu": lambda: moe.matmul_fp8(rows(), weights(192, 64), act="swiglu"),
        "matmul_quantize": lambda: moe.matmul_fp8(rows(), weights(128, 64), quantize=True),
        "matmul_type": lambda: moe.matmul_fp8(rows(), weights(128, 64), out_dtype=torch.float16),
        "grouped_groups": lambda: moe.grouped_matmul_fp8(rows(), weights(3, 128, 64), None),
        "grouped_experts": lambda: moe.grouped_matmul_fp8(rows(), weights(4, 128, 64), groups()),
        "grouped_rows": lambda: moe.grouped_matmul_fp8(rows(7), weights(3, 128, 64), groups()),
        "grouped_matrix": lambda: moe.grouped_matmul_fp8(rows(), weights(128, 64), groups()),
        "end_groups": lambda: moe.combine_norm(t(8, 64), None, w(), r()),
        "end_y": lambda: moe.combine_norm(None, groups(), w(), r()),
        "end_rows": lambda: moe.combine_norm(t(7, 64), groups(), w(), r()),
        "end_gates": lambda: moe.combine_norm(t(8, 64), groups(), t(4, 3, d=f32), r()),
        "end_tokens": lambda: moe.combine_norm(t(8, 64), groups(), w(), t(5, 64)),
        "end_width": lambda: moe.residual_norm(t(2, 32769), t(2, 32769)),
        "end_shared": lambda: moe.combine_norm(t(8, 64), groups(), w(), r(), shared=t(4, 64, d=f32)),
        "end_post": lambda: moe.combine_norm(t(8, 64), groups(), w(), r(), post=t(65)),
        "end_gate": lambda: moe.combine_norm(t(8, 64), groups(), w(), r(), gate=t(4, 64, d=f32)),
        "end_gate_type": lambda: moe.combine_norm(t(8, 64), groups(), w(), r(), gate=t(64)),
        "end_eps": lambda: moe.rms_norm(r(), t(64), eps=0.0),
        "end_scale": lambda: moe.residual_norm(r(), r(), residual_scale=float("inf")),
        "end_type": lambda: moe.rms_norm(r(), t(64), out_dtype=torch.float16),
        "end_weight": lambda: moe.rms_norm(r(), None),
        "end_residual": lambda: moe.residual_norm(None, r()),
    }
    for name, call in calls.items():
        try:
            call()
            print(name, "made")
        except ValueError as e:
            print(name, "refused", e)
"""
NAMES = [line.split('"')[1] for line in BINDING.splitlines() if line.startswith('        "')]


@pytest.fixture(scope="module")
def answers():
    r = subprocess.run([sys.executable, "-c", BINDING], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-500:], r.stderr[-2000:])
    return dict(line.split(" ", 1) for line in r.stdout.splitlines())


@pytest.mark.parametrize("call", NAMES)
def test_binding_refuses_as_values(answers, call):
    assert answers[call].startswith("refused"), answers[call]


def test_8bit_blocks_do_not_change():
    import serving_layer_moe_gb300 as moe
    q = moe.FP8Rows._of(torch.zeros(2, 16).to(torch.float8_e4m3fn), torch.zeros(1, 2))
    for name in ("codes", "scales", "shape", "K"):
        with pytest.raises(AttributeError):
            setattr(q, name, None)
