"""moe_operators_check: one flag for every operator's kernels, read by one copy."""
import glob
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_check_waits_for_one_copy():
    """A copy to the host's own memory is waited for, so each costs the check a wait of its own."""
    text = "".join(open(f).read() for f in glob.glob(os.path.join(ROOT, "serving_layer_moe_gb300", "csrc", "*.cu*")))
    assert len(re.findall("cudaMemcpyFromSymbolAsync", text)) == 1


# The flag's address, and how many pairs of CTAs a device holds, are looked up by a process's first 8-bit product: here that one is captured,
# on a stream that is not torch's own.
FIRST_CALL = """
import sys, torch
import serving_layer_moe_gb300 as moe
gen = torch.Generator(device="cuda").manual_seed(1)
x, w = moe.quantize_fp8(torch.randn(int(sys.argv[1]), 272, device="cuda", generator=gen)), moe.quantize_fp8_weights(torch.randn(384, 272, device="cuda", generator=gen))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = moe.matmul_fp8(x, w, out_dtype=torch.float32)
g.replay()
moe.check_operators()
assert torch.equal(y, moe.matmul_fp8(x, w, out_dtype=torch.float32)) and y.abs().sum() > 0
print("right")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [40, 1000])
def test_the_first_product_may_be_captured(rows):
    """Single CTAs, and pairs."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL, str(rows)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "right", (r.stdout[-300:], r.stderr[-2000:])


@pytest.mark.gpu
def test_the_check_is_quiet_after_calls_that_went_well():
    import torch

    import serving_layer_moe_gb300 as moe
    x, w = moe.quantize_fp8(torch.ones(5, 128, device="cuda")), moe.quantize_fp8_weights(torch.ones(256, 128, device="cuda"))
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        moe.matmul_fp8(x, w)
        moe.check_operators(stream)
