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
