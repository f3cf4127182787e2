"""What the routed-expert operators refuse (no GPU needed: arguments are checked before any CUDA call)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
A, B, C, D, F, G, H = (P(0x10000 * i) for i in range(1, 8))     # aligned addresses that nothing reads
BF16, F32, NVFP4, MXFP4 = 1, 0, 3, 4


@pytest.fixture(scope="module")
def lib():
    from serving_layer_moe_gb300 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    from serving_layer_moe_gb300 import operators
    return operators._operators()


def refused(lib, status, word):
    assert status == 1
    assert word in lib.moe_last_error(), lib.moe_last_error()


def test_header_declares_and_library_exports_the_operators(lib):
    from serving_layer_moe_gb300 import OPERATOR_SYMBOLS
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_operators.h")).read(), flags=re.S)
    fns = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)))
    assert fns == sorted(OPERATOR_SYMBOLS)
    out = subprocess.run(["nm", "-D", "--defined-only", lib._name], capture_output=True, text=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(fns) <= exported


def test_sizes_without_a_device(lib):
    assert lib.moe_grouped_tiles(0, 5) == 0
    assert lib.moe_grouped_tiles(1, 5) == 1
    assert lib.moe_grouped_tiles(8, 128) == 8           # eight experts of one row each
    assert lib.moe_grouped_tiles(256, 2) == 3           # 1 + 255 rows
    assert lib.moe_grouped_tiles(1 << 40, 4096) == ((1 << 40) + 127 * 4096) // 128
    assert lib.moe_group_workspace(0, 8, 128) == 0 and lib.moe_group_workspace(32, 8, 128) == 0     # one block, no counts
    assert lib.moe_group_workspace(8192, 8, 256) >= 257 * 4


def route(lib, T=4, E=16, k=2, dt=F32, logits=A, scoring=0, bias=None, ng=1, tg=1, renorm=1, scale=1.0, ids=B, w=C,
          off=None, til=None, order=None, place=None, ws=None, n=0):
    return lib.moe_route(T, E, k, dt, logits, scoring, bias, ng, tg, renorm, scale, ids, w, off, til, order, place, ws, n, None)


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), b"T >= 0"), (dict(E=0), b"E"), (dict(E=5000), b"4096"), (dict(k=0), b"k"), (dict(k=17), b"more than E"),
    (dict(T=1 << 30, k=8), b"31 bits"), (dict(dt=2), b"logits_dtype"), (dict(scoring=2), b"scoring"), (dict(bias=D), b"softmax"),
    (dict(ng=2, tg=2), b"softmax"), (dict(scoring=1, ng=3, tg=3), b"n_group"), (dict(scoring=1, ng=8, tg=0), b"topk_group"),
    (dict(scoring=1, ng=8, tg=9), b"topk_group"), (dict(scoring=1, ng=16, tg=1), b"k = 2"), (dict(logits=None), b"NULL"),
    (dict(ids=None), b"NULL"), (dict(logits=P(0x10002)), b"aligned"), (dict(w=P(0x10001)), b"aligned"),
    (dict(off=D), b"all needed"), (dict(T=64, k=8, off=D, til=F, order=G, place=H), b"workspace"),
    (dict(T=64, k=8, off=D, til=F, order=G, place=H, ws=A, n=16), b"workspace"),
    (dict(off=D, til=F, order=P(0x10002), place=H, ws=A, n=1 << 20), b"aligned")])
def test_route_refuses(lib, kw, word):
    refused(lib, route(lib, **kw), word)


@pytest.mark.parametrize("args,word", [
    ((-1, 4, 2, A, B, C, D, F, G, 1 << 20), b"T >= 0"), ((4, 0, 2, A, B, C, D, F, G, 1 << 20), b"E"),
    ((4, 4, 2, None, B, C, D, F, G, 1 << 20), b"NULL"), ((4, 4, 2, A, None, C, D, F, G, 1 << 20), b"all needed"),
    ((400, 4, 2, A, B, C, D, F, None, 0), b"workspace"), ((4, 4, 2, P(0x10001), B, C, D, F, G, 1 << 20), b"aligned")])
def test_group_pairs_refuses(lib, args, word):
    refused(lib, lib.moe_group_pairs(*args, None), word)


@pytest.mark.parametrize("args,word", [
    ((1, 0, F32, A, B), b"at least one"), ((-1, 8, F32, A, B), b"G"), ((1, 8, 2, A, B), b"dtype"), ((1, 8, F32, None, B), b"NULL"),
    ((1, 8, F32, P(0x10002), B), b"aligned")])
def test_fp4_scale_refuses(lib, args, word):
    refused(lib, lib.moe_fp4_scale(*args, None), word)


def quantize(lib, G=1, N=4, K=64, dt=BF16, x=A, wd=NVFP4, g=None, gc=0, E=0, k=0, off=None, til=None, order=None, codes=B, scales=C):
    return lib.moe_quantize_fp4(G, N, K, dt, x, wd, g, gc, E, k, off, til, order, codes, scales, None)


@pytest.mark.parametrize("kw,word", [
    (dict(K=48), b"multiple of 32"), (dict(K=0), b"multiple of 32"), (dict(N=-1), b"negative"), (dict(dt=3), b"dtype"), (dict(wd=BF16), b"wdtype"),
    (dict(wd=MXFP4, g=D, gc=1), b"no matrix scale"), (dict(G=3, g=D, gc=2), b"g_count"), (dict(x=None), b"NULL"),
    (dict(x=P(0x10008)), b"16-byte"), (dict(codes=P(0x10004)), b"16-byte"), (dict(off=D), b"grouped"),
    (dict(off=D, til=F, order=G, E=0, k=2), b"grouped"), (dict(G=2, off=D, til=F, order=G, E=4, k=2), b"grouped"),
    (dict(off=P(0x10002), til=F, order=G, E=4, k=2), b"4-byte")])
def test_quantize_refuses(lib, kw, word):
    refused(lib, quantize(lib, **kw), word)


@pytest.mark.parametrize("args,word", [
    ((1, 4, 40, NVFP4, A, B, None, 0, 0, None, None, BF16, C), b"multiple of 32"),
    ((1, 4, 64, NVFP4, A, B, None, 0, 0, None, None, NVFP4, C), b"dtype"),
    ((1, 4, 64, NVFP4, A, B, None, 0, 0, None, None, BF16, None), b"NULL"),
    ((1, 4, 64, NVFP4, A, B, None, 0, 4, D, None, BF16, C), b"grouped"),
    ((3, 4, 64, MXFP4, A, B, D, 2, 0, None, None, BF16, C), b"g_count")])
def test_dequantize_refuses(lib, args, word):
    refused(lib, lib.moe_dequantize_fp4(*args, None), word)


def matmul(lib, P_=8, E=2, N=64, K=64, x=A, rows=8, order=None, place=None, k=2, w=B, off=C, til=D, act=0, od=BF16, out=F, ws=None, n=0):
    return lib.moe_grouped_matmul(P_, E, N, K, x, rows, order, place, k, w, off, til, act, od, out, ws, n, None)


@pytest.mark.parametrize("kw,word", [
    (dict(P_=-1), b"P >= 0"), (dict(E=0), b"E"), (dict(E=4097), b"4096"), (dict(N=0), b"N"), (dict(K=12), b"multiple of 8"), (dict(act=2), b"act"),
    (dict(act=1, N=48), b"multiple of 32"), (dict(od=3), b"out_dtype"), (dict(off=None), b"offsets"), (dict(x=None), b"NULL"),
    (dict(x=P(0x10008)), b"16-byte"), (dict(w=P(0x10002)), b"16-byte"), (dict(order=G, place=H, k=0), b"order"), (dict(order=G), b"place"), (dict(order=G, place=H, k=3), b"divides"), (dict(rows=0), b"rows"), (dict(rows=7), b"rows"),
    (dict(P_=128, rows=64, order=G, place=H), b"workspace"), (dict(P_=128, rows=64, order=G, place=H, ws=P(0x10008), n=1 << 20), b"workspace")])
def test_grouped_matmul_refuses(lib, kw, word):
    refused(lib, matmul(lib, **kw), word)


def matmul_fp4(lib, P_=8, E=2, N=64, K=64, wd=NVFP4, xc=A, xs=B, gx=None, wc=C, ws=D, gw=None, gwc=0, off=F, til=G, act=0, od=BF16,
               out=H, oc=None, os_=None, go=None):
    return lib.moe_grouped_matmul_fp4(P_, E, N, K, wd, xc, xs, gx, wc, ws, gw, gwc, off, til, act, od, out, oc, os_, go, None)


@pytest.mark.parametrize("kw,word", [
    (dict(K=72), b"multiple of 32"), (dict(wd=BF16), b"wdtype"), (dict(wd=MXFP4, act=1, N=128, out=None, oc=A, os_=B, go=C), b"no matrix scale"), (dict(gw=A, gwc=3), b"gw_count"),
    (dict(xc=None), b"NULL"), (dict(ws=P(0x10008)), b"16-byte"), (dict(out=None), b"act = 1"), (dict(out=None, act=1, N=96), b"multiple of 32"),
    (dict(out=None, act=1, N=128), b"out_codes"), (dict(out=P(0x10002)), b"16-byte"), (dict(gx=P(0x10002)), b"4-byte")])
def test_grouped_matmul_fp4_refuses(lib, kw, word):
    refused(lib, matmul_fp4(lib, **kw), word)


@pytest.mark.parametrize("args,word", [
    ((-1, 2, 8, F32, A, B, C, F32, D), b"T >= 0"), ((1, 0, 8, F32, A, B, C, F32, D), b"k >= 1"), ((1, 2, 8, 3, A, B, C, F32, D), b"y_dtype"),
    ((1, 2, 8, F32, None, B, C, F32, D), b"NULL"), ((1, 2, 8, F32, P(0x10004), B, C, F32, D), b"aligned"),
    ((1, 2, 9, BF16, P(0x10001), B, C, F32, D), b"aligned")])
def test_combine_refuses(lib, args, word):
    refused(lib, lib.moe_combine(*args, None), word)


def test_binding_refuses_host_tensors_and_wrong_types():
    import serving_layer_moe_gb300 as moe
    with pytest.raises(ValueError, match="CUDA device"):
        moe.route(torch.zeros(2, 8), 2)
    with pytest.raises(ValueError, match="logits must be"):
        moe.route(torch.zeros(2, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="topk_ids must be"):
        moe.group_pairs(torch.zeros(2, 2, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="not contiguous"):
        moe.fp4_scale(torch.zeros(4, 8).T)
    with pytest.raises(ValueError, match="wdtype"):
        moe.quantize_fp4(torch.zeros(4, 32), "fp8")
    with pytest.raises(ValueError, match="FP4Rows"):
        moe.grouped_matmul_fp4(torch.zeros(4, 32), None, None)
    with pytest.raises(ValueError, match="FP4Rows"):
        moe.dequantize_fp4(torch.zeros(4, 32))
