"""The router's losses where very many tokens or sequences are summed."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import U32
from train_plain import F64

pytestmark = pytest.mark.gpu


# Equal tokens, so that every addition to a running sum rounds the same way. A sum may pass 128
# roundings, however many its terms: one run of terms after the other adds up in fp32 (32 of
# them), the runs' sums are added without loss, and blocks, warps and lanes are joined in trees.
# exp, log and the quotients add 16 half steps, twice for z's squares.
@pytest.mark.parametrize("T", [1 << 18, 1 << 23, 1 << 26])
def test_sums_over_very_many_tokens(cuda_ok, T):
    row = torch.tensor([0.3, -0.2, 1.1, 0.45], device="cuda")
    L = row.expand(T, 4).contiguous()
    idx = torch.full((T, 1), 2, dtype=torch.int32, device="cuda")
    c = moe.router_loss_config(T, 4, 1, balance=1.0, z=1.0)
    ws = moe.alloc_router_loss_workspace(c)
    r = moe.router_loss(c, L, idx, ws=ws)
    assert moe.get_device_error(ws) == moe.MOE_OK
    r64 = row.to(F64)
    bal, z = float(4 * torch.softmax(r64, 0)[2]), float(torch.logsumexp(r64, 0) ** 2)
    assert r.counts.tolist() == [[0, 0, T, 0]] and r.tokens.tolist() == [T, 1, T]
    assert abs(float(r.loss[1]) - bal) <= 144 * U32 * bal
    assert abs(float(r.loss[2]) - z) <= 160 * U32 * z
    assert abs(float(r.loss[0]) - bal - z) <= 160 * U32 * (bal + z)


def test_very_many_sequences(cuda_ok):
    # of one token each, every one with the same terms: a thousand to a thread that adds them up
    T = 1 << 20
    row = torch.tensor([0.3, -0.2], device="cuda")
    L = row.expand(T, 2).contiguous()
    idx = torch.ones((T, 1), dtype=torch.int32, device="cuda")
    off = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    c = moe.router_loss_config(T, 2, 1, S=T, balance=1.0, z=1.0)
    ws = moe.alloc_router_loss_workspace(c)
    r = moe.router_loss(c, L, idx, ws=ws, offsets=off)
    assert moe.get_device_error(ws) == moe.MOE_OK
    r64 = row.to(F64)
    bal, z = float(2 * torch.softmax(r64, 0)[1]), float(torch.logsumexp(r64, 0) ** 2)
    assert r.tokens[-2:].tolist() == [T, T]
    assert abs(float(r.loss[1]) - bal) <= 144 * U32 * bal
    assert abs(float(r.loss[2]) - z) <= 160 * U32 * z
