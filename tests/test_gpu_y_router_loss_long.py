"""The router's losses where very many tokens or sequences are summed."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import U32
from train_plain import F64
from test_gpu_v_router_loss import check, gen, problem

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


@pytest.mark.parametrize("E,k", [(8, 2), (40, 3), (128, 4), (256, 8)])
def test_chunks_of_several_runs(cuda_ok, E, k):
    # a long batch whole, in sequences that end inside chunks, masked, the same bits again
    T = 130001
    L, idx = problem(T, E, k, seed=E)
    r, g = check(L, idx, balance=0.7, z=0.01)
    again, h = check(L, idx, balance=0.7, z=0.01)
    assert torch.equal(r.loss, again.loss) and torch.equal(g, h)
    mask = torch.rand((T,), generator=gen(E), device="cuda") > 0.3
    mask[5000:9000] = False
    check(L, idx, [3, 300, 300, 70001, 129000], mask, balance=0.7, z=0.01, dloss=2.0)


def test_an_infinity_among_very_many(cuda_ok):
    """A z loss past the range of fp32 is an infinity, not a NaN, and the balance loss is not
    touched: squares of 3e19 in one token."""
    T = 130001
    L = torch.zeros((T, 4), device="cuda")
    L[70000] = 3e19
    idx = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    c = moe.router_loss_config(T, 4, 1, balance=1.0, z=0.0)
    r = moe.router_loss(c, L, idx, ws=moe.alloc_router_loss_workspace(c))
    assert float(r.loss[2]) == float("inf") and abs(float(r.loss[1]) - 1) <= 160 * U32
