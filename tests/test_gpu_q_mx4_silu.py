"""The 4-bit product's SiLU with fp32 output, against SiLU in 64 bits of the same product without
it (the same sums in the same order): z / (1 + e) with e = exp(-z) to 2 units in the last place
(4 half steps), one addition and one division: 6 half steps of fp32, 8 allowed. Where e passes
the fp32 range the result is 0 for at most 88.7 e^-88.7 = 2.7e-37."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import F64, U32
from test_gpu_j_mx4 import gen, offsets_of

pytestmark = pytest.mark.gpu


# few rows (split sums), one block a tile, pairs of blocks
@pytest.mark.parametrize("counts", [[2, 1], [32], [200, 100], [400, 130]])
@pytest.mark.parametrize("K,N", [(64, 192), (512, 384)])
def test_silu_in_fp32(cuda_ok, counts, K, N):
    R, E = sum(counts), len(counts)
    g = gen(K + N + R)
    x = 64 * K ** -0.5 * torch.randn((R, K), generator=g, device="cuda")
    W = torch.randn((E, K, N), generator=g, device="cuda")
    off = offsets_of(counts)
    c = moe.mx4_config(R, K, N, E, dtype="f32", out_dtype="f32")
    ws = moe.alloc_mx4_workspace(c)
    q, sc = moe.mx4_quantize_rows(c, x, off, ws=ws)
    wq, wsc = moe.mx4_quantize_weights(c, W)
    z = moe.mx4_product(c, q, sc, wq, wsc, off, ws=ws).to(F64)
    assert float(z.min()) < -88 and float(z.max()) > 88  # the whole range of exp
    cs = moe.mx4_config(R, K, N, E, dtype="f32", out_dtype="f32", silu=1)
    got = moe.mx4_product(cs, q, sc, wq, wsc, off, ws=ws).to(F64)
    assert moe.get_device_error(ws) == moe.MOE_OK
    want = z * torch.sigmoid(z)
    over = (got - want).abs() - (8 * U32 * want.abs() + 2.7e-37)
    assert bool((over <= 0).all()), float(((got - want).abs() / want.abs().clamp(min=1e-30)).max())
