"""The router's losses where a token may take no expert at all."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from test_gpu_v_router_loss import check, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(8, 2), (64, 4), (256, 8)])
@pytest.mark.parametrize("value", [-float("inf"), float("inf")])
def test_a_token_without_a_softmax(cuda_ok, E, k, value):
    T = 40
    L, idx = problem(T, E, k, seed=E)
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[17] = False
    want, g = check(L, idx, None, mask)
    bad = L.clone()
    if value < 0:
        bad[17] = value  # nothing that it may take
    else:
        bad[17, 3] = value
    c = moe.router_loss_config(T, E, k, balance=0.02, z=0.003)
    ws = moe.alloc_router_loss_workspace(c)
    # masked, it does not matter
    r = moe.router_loss(c, bad, idx, ws=ws, mask=mask)
    assert torch.equal(r.loss, want.loss)
    assert torch.equal(moe.router_loss_backward(c, bad, r, mask=mask), g)
    # else the losses say so, and of the gradients its own alone
    r = moe.router_loss(c, bad, idx, ws=ws)
    assert bool(r.loss[:2].isnan().all()) and not bool(torch.isfinite(r.loss[2]))
    d = moe.router_loss_backward(c, bad, r)
    others = torch.arange(T, device="cuda") != 17
    assert bool(d[17].isnan().any()) and bool(torch.isfinite(d[others]).all())


def test_the_lowest_finite_value_is_a_mask_too(cuda_ok):
    """Logits of the type's lowest value: experts that are not taken; a token of nothing else takes
    all of them alike."""
    T, E, k = 64, 16, 2
    L, idx = problem(T, E, k, seed=2)
    low = torch.finfo(torch.float32).min
    L[:, 5:9] = low
    L[11] = low
    idx = torch.topk(L, k, dim=1).indices.to(torch.int32)
    c = moe.router_loss_config(T, E, k, balance=1.0, z=0.0)
    r = moe.router_loss(c, L, idx, ws=moe.alloc_router_loss_workspace(c))
    g = moe.router_loss_backward(c, L, r)
    p = torch.softmax(L.double(), 1)
    f = E * torch.bincount(idx.flatten().long(), minlength=E).double() / (k * T)
    assert abs(float(r.loss[1]) - float((f * p.mean(0)).sum())) <= 160 * 2.0 ** -24 * float(
        (f * p.mean(0)).sum())
    want = p * (f - (p * f).sum(1, keepdim=True)) / T
    terms = p * (f + (p * f).sum(1, keepdim=True)) / T
    # (160 half steps: 128 of the sums, 32 of exp's argument)
    assert bool(((g.double() - want).abs() <= 160 * 2.0 ** -24 * terms + 2.0 ** -140).all())
