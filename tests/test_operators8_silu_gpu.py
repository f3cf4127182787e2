"""silu of fp32 results at gates far below zero, as the header has it: within 11 half units, or 0 below -87.3, where it is under 1.1e-36."""
import numpy as np
import pytest
import torch

from tests.test_operators_gpu import EPS, dev, host

pytestmark = pytest.mark.gpu


def test_gates_far_below_zero():
    """Gate and up of token i: its scale times the codes -1 and 1, both exact."""
    import serving_layer_moe_gb300 as moe
    v = np.concatenate([np.linspace(0.125, 87, 300), np.linspace(87, 110, 200)]).astype(np.float32)
    codes = torch.zeros(len(v), 16, device="cuda")
    codes[:, 0] = 1
    w = torch.zeros(128, 16, device="cuda")
    w[:64, 0], w[64:, 0] = -1, 1
    f8 = torch.float8_e4m3fn
    got = host(moe.matmul_fp8(moe.FP8Rows(codes.to(f8), dev(v[None])), moe.FP8Weights(w.to(f8), torch.ones(1, 1, device="cuda")), act="swiglu", out_dtype=torch.float32))
    x = v.astype(np.float64)
    silu = -x / (1 + np.exp(x))
    want = silu * x
    near = np.abs(got - want[:, None]) <= 13 * EPS * np.abs(want)[:, None]        # silu, and the product with up
    assert near[x < 87.3].all()
    assert (near | (got == 0))[x >= 87.3].all() and (np.abs(silu[x >= 87.3]) < 1.1e-36).all()
