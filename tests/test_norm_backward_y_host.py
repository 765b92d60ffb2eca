"""The norm backward looks at y also where the kept x stands in for it (no GPU needed: the
refusal comes first)."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from mixture_experts_routed_gb300 import build as B


@pytest.mark.parametrize("y", [torch.zeros((3, 64)), torch.zeros((4, 128)),
                               torch.zeros((4, 64), dtype=torch.bfloat16)])
def test_y_of_another_forward(y):
    B.build()
    c = moe.norm_config(4, 64, "f32")
    t, w, r = torch.zeros((4, 64)), torch.ones(64), torch.ones(4)
    with pytest.raises(moe.MoEError, match="y is .* not "):
        moe.block_norm_backward(c, t, t, y, t, w, None, w, r, moe.KeptNorm(r, t), ws=torch.zeros(8))
