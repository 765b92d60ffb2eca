"""8-bit products on one CTA and on pairs, often enough for a race that shows once in thousands of
calls: scales that change from stage to stage (one read before it is there changes the sum), calls
back to back behind one another, compared on the device, with one synchronisation at the end."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from test_gpu_u_fp8 import problem, run_grad, run_product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,K,N", [([700, 300, 900], 2048, 1536), ([460, 1, 930], 4160, 704),
                                        ([130, 60, 200], 2048, 1536), ([20, 0, 3], 4160, 704)])
def test_products_repeat(cuda_ok, counts, K, N):
    p = problem(counts, K, N, seed=sum(counts))
    c, off, ws = p["c"], p["off"], p["ws"]
    want = run_product(p, False), run_product(p, True), run_grad(p)
    y, dx, dW = (torch.empty_like(t) for t in want)
    moved = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(3000):
        moe.fp8_product(c, p["x"], p["wq"], p["wsc"], off, ws=ws, out=y)
        moe.fp8_product(c, p["dy"], p["wq"], p["wsc"], off, ws=ws, transposed=True, out=dx)
        moe.fp8_weight_grad(c, p["x"], p["dy"], off, ws=ws, out=dW)
        moved += (y != want[0]).any() | (dx != want[1]).any() | (dW != want[2]).any()
    assert int(moved) == 0
    assert moe.get_device_error(ws) == moe.MOE_OK
