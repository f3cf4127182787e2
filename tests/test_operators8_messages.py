"""What the 8-bit operators' refusals say (no GPU needed)."""
import os
import subprocess
import sys

import pytest

from tests.test_operators_refusals import ROOT


@pytest.fixture(scope="module", autouse=True)
def built():
    from serving_layer_moe_gb300 import build as b
    if not (os.path.exists(b.LIB) and os.path.exists(b.HOST)):
        b.build()


# Groups of four tokens with no experts each, on tensors that say they are on a GPU and take no memory.
NO_EXPERTS = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import serving_layer_moe_gb300 as moe
moe.operators._host()
with FakeTensorMode(allow_non_fake_inputs=True):
    i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
    gr = moe.ExpertGroups(i(4), i(4), i(0), i(4, 0))
    try:
        moe.quantize_fp8(torch.empty(4, 64, dtype=torch.bfloat16, device="cuda"), groups=gr)
    except ValueError as e:
        print("refused", e)
"""


def test_groups_without_experts_are_refused_by_what_they_lack():
    r = subprocess.run([sys.executable, "-c", NO_EXPERTS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused groups hold no experts a token", (r.stdout, r.stderr[-1000:])


def test_a_call_that_was_not_made_blames_no_one_format(monkeypatch):
    import torch

    from serving_layer_moe_gb300 import operators
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="tensors that its arguments hold") as e:
        operators._again(lambda: None, 0, None)
    assert "bit" not in str(e.value)
