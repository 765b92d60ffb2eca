"""The router's losses and their gradient where logits share an offset."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import U32
from train_plain import F64
from test_gpu_v_router_loss import check, gen, problem

pytestmark = pytest.mark.gpu


# A common offset changes no p: its relative error stays that of exp(L - max) and its sum,
# whatever the logits' size (the half steps of rel in `check`, where the span is the logits' own).
@pytest.mark.parametrize("offset", [100.0, -1000.0, 1000.0, 30000.0])
@pytest.mark.parametrize("T,E,k", [(64, 8, 2), (300, 40, 3), (257, 64, 4), (200, 256, 8)])
def test_logits_with_a_common_offset(cuda_ok, offset, T, E, k):
    L, idx = problem(T, E, k, seed=T + E)
    L = L + offset
    check(L, idx, balance=0.7, z=0.0)
    check(L, idx, offs=[3, 40, 40, T - 5], balance=0.7, z=0.0, dloss=-2.5)
    check(L, idx, balance=0.02, z=0.003)


def test_the_gradient_of_an_even_load_with_an_offset(cuda_ok):
    """f is 1 for every expert, so p (f - sum p f) is 0, the difference of two equal terms: what is
    left of it is 128 half steps of them, and those of the span of L - max. (p off by half a step of
    10000 would leave a thousand times that.)"""
    T, E, k = 4096, 8, 2
    L = 0.5 * torch.randn((T, E), generator=gen(8), device="cuda") + 10000.0
    idx = torch.stack([torch.arange(T, device="cuda") % E,
                       (torch.arange(T, device="cuda") * 5 + 3) % E], 1).to(torch.int32)
    idx[:16, 1] = (idx[:16, 0] + 1) % E
    c = moe.router_loss_config(T, E, k, balance=1.0)
    r = moe.router_loss(c, L, idx, ws=moe.alloc_router_loss_workspace(c))
    g = moe.router_loss_backward(c, L, r).to(F64)
    p = torch.softmax(L.to(F64), 1)
    f = E * torch.bincount(idx.flatten().long(), minlength=E).to(F64) / (k * T)
    want = p * (f - (p * f).sum(1, keepdim=True)) / T
    terms = float((p * 2 * f / T).norm())
    assert float((g - want).norm()) <= (128 + 4 * 8) * U32 * terms


@pytest.mark.parametrize("offset", [1e8, -3e9, 1e12])
@pytest.mark.parametrize("E", [8, 40, 100, 256])
def test_logits_of_any_size(cuda_ok, offset, E):
    # steps of 8, 256 and 65536 apart: each token has one expert or some equal ones
    L, idx = problem(200, E, 3, seed=9)
    check(L * abs(offset) * 2.0 ** -22 + offset, idx, balance=0.7, z=0.0)
