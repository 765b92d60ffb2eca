"""The norms around a block where a row group walks more rows than its ring holds: slots filled
again, the next row's sum and statistics taken a row ahead, column sums over rows, in every form
(gate, halves, type). On 152 SMs a warp's rows make at most 4864 groups backward and 3040 forward,
a block's of 4096 columns 152 both ways: seven rows or more in some groups and one more or less in
others. Tolerances as in test_gpu_h_block_norm."""
import pytest
import torch

from test_gpu_h_block_norm import both

pytestmark = pytest.mark.gpu
FORMS = [(kind, halves) for halves in ((True, True), (True, False))
         for kind in ("none", "token", "channel", "element")] + [("none", (False, True))]


@pytest.mark.parametrize("kind,halves", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(35001, 64), (1081, 4096)])
def test_many_rows_a_group(cuda_ok, T, d, dtype, kind, halves):
    both(T, d, dtype, kind, *halves, seed=T)


# rows for which a ring holds two (an element gate, the widest rows of the ring), groups of
# several warps with an odd last row, rows of 160 and 288 threads
@pytest.mark.parametrize("T,d,dtype,kind", [
    (777, 8192, "bf16", "element"), (777, 8192, "bf16", "token"), (10007, 192, "bf16", "token"),
    (10007, 256, "bf16", "element"), (9001, 128, "f32", "token"), (2003, 1088, "bf16", "element"),
    (1403, 2112, "f32", "token")])
def test_other_rings(cuda_ok, T, d, dtype, kind):
    both(T, d, dtype, kind, True, True, seed=d)


# rows too wide for the ring
@pytest.mark.parametrize("kind,halves", FORMS)
@pytest.mark.parametrize("T,d,dtype", [(157, 4160, "f32"), (5, 16448, "bf16")])
def test_wide_rows(cuda_ok, T, d, dtype, kind, halves):
    both(T, d, dtype, kind, *halves, seed=d)
