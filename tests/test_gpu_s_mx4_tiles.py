"""4-bit products with several tiles to a block (or pair of blocks) and contractions of several
stages: while a tile's second accumulator still drains, the first half's products of some stages
go ahead, and the issuer then goes back to them for the second half, across the ends of the rings
of data (4 or 6 stages) and of scales (4 or 5). And the border between single blocks and pairs.
Tolerances as in test_gpu_j_mx4."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from test_gpu_j_mx4 import product

pytestmark = pytest.mark.gpu

SINGLE = [60 + 37 * i % 69 for i in range(64)]        # 60..128 rows: 384 tiles of 1472 columns
PAIRS = [250 + 97 * i % 260 for i in range(24)]       # 250..509: 288 tiles over 76 pairs


@pytest.mark.parametrize("K", [1536, 2048, 2112])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [SINGLE, PAIRS], ids=["single", "pairs"])
def test_several_tiles_of_several_stages(cuda_ok, counts, K, out_dtype):
    c, q, sc, wq, wsc, off, ws, out = product(counts, K, 1472, out_dtype, seed=K)
    again = torch.zeros_like(out)
    for _ in range(5):
        moe.mx4_product(c, q, sc, wq, wsc, off, ws=ws, out=again)
        assert torch.equal(again, out)
    assert moe.get_device_error(ws) == moe.MOE_OK


# stage counts around the rings' lengths, with column tiles of both halves and of one
@pytest.mark.parametrize("K", [768, 1024, 1280, 1344])
@pytest.mark.parametrize("N", [320, 384, 512])
@pytest.mark.parametrize("pairs", [False, True])
def test_other_contractions(cuda_ok, K, N, pairs):
    product([300] * 60 if pairs else [100 + i % 28 for i in range(120)], K, N, seed=K + N)


@pytest.mark.parametrize("rows", [191, 192, 193])
@pytest.mark.parametrize("K,N", [(64, 64), (1408, 192), (2048, 1472)])
def test_the_border_of_pairs(cuda_ok, rows, K, N):
    product([rows], K, N, seed=rows)
    product([2 * rows - 3, 3], K, N, seed=rows)
