"""The layer for a few tokens where no token has an expert."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from test_gpu_i_few_tokens import compare, layer
from workloads import make_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 8, 32])
@pytest.mark.parametrize("E,k,router,kw", [(8, 2, 0, {}), (72, 8, 1, {}),
                                           (32, 3, 2, dict(n_group=8, topk_group=3))])
def test_no_token_with_an_expert(cuda_ok, T, E, k, router, kw):
    # NaN logits choose nothing: zero rows, the router's flag, and a workspace that serves the next
    c = layer(T, 320, E, k, 192, router, seed=T, **kw)
    i = make_inputs(c, device="cuda")
    ws = moe.alloc_workspace(c, "few")
    none = torch.full_like(i["x"], float("nan"))
    for _ in range(2):
        out = torch.full_like(i["x"], 7.0)
        moe.forward_few(c, none, i["Wg"], i["bias"], i["W1"], i["W2"], ws=ws, out=out)
        torch.cuda.synchronize()
        assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX
        assert bool((out == 0).all())
        out = moe.forward_few(c, i["x"], i["Wg"], i["bias"], i["W1"], i["W2"], ws=ws)
        torch.cuda.synchronize()
        assert moe.get_device_error(ws) == moe.MOE_OK
        compare(c, i, out)
