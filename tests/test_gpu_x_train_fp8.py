"""The example block's training step with 8-bit experts, router losses and dropout on the GPU,
against a plain 64-bit composition that quantises and rounds at the same places."""
import os
import sys

import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import F64, half_step
from train_plain import dropout_keep, fp8_values, router_loss

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
from expert_block import ExpertBlock  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rows(T, d, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((T, d), generator=g, device="cuda").to(BF)


def bf(v):
    return v.to(BF).to(F64)


def near(got, want, limit, name=""):
    err = float((got.to(F64) - want).norm() / want.norm())
    assert err <= limit, (name, err)


class Straight(torch.autograd.Function):
    """The value given, the gradient unchanged."""

    @staticmethod
    def forward(ctx, v, value):
        return value

    @staticmethod
    def backward(ctx, g):
        return g, None


def rounded(v):
    return Straight.apply(v, bf(v.detach()))


class Expert(torch.autograd.Function):
    """One expert's rows in 8 bits, forward and backward as the products take them."""

    @staticmethod
    def forward(ctx, x, W1, W2, w):
        def q(v, along):
            return fp8_values(v, *along)[0]

        row, col, block = (1, 128), (128, 1), (128, 128)
        w1, w2 = q(W1, block), q(W2, block)
        z = bf(q(x, row) @ w1)
        h = z * torch.sigmoid(z)
        ctx.save_for_backward(x, z, h, w1, w2, w)
        return q(h, row) @ w2

    @staticmethod
    def backward(ctx, g):
        # g: of y = one row's output; it comes as db times the row's routing weight
        x, z, h, w1, w2, w = ctx.saved_tensors
        row, col = (1, 128), (128, 1)
        dy = g
        dh = bf(fp8_values(dy, *row)[0] @ w2.t())
        s = torch.sigmoid(z)
        dz = dh * s * (1 + z * (1 - s))
        dx = fp8_values(dz, *row)[0] @ w1.t()
        dW1 = fp8_values(x, *col)[0].t() @ fp8_values(dz, *col)[0]
        dW2 = fp8_values(h, *col)[0].t() @ fp8_values(dy, *col)[0]
        return dx, dW1, dW2, None


@pytest.mark.parametrize("T,k", [(64, 4), (300, 2)])
def test_step(cuda_ok, T, k):
    d, f, E, p = 256, 192, 4, 0.25
    block = ExpertBlock(d, f, E, k, alpha=0.5, beta=1.5, seed=T)
    x = rows(T, d, 2)
    dout, dnext = rows(T, d, 3), rows(T, d, 4).float()
    state = torch.tensor([99, 7], dtype=torch.int64, device="cuda")
    out, n, loss, grads, wss = block.train_step_fp8(x, dout, dnext, state, p=p, balance=0.3,
                                                    z_loss=0.2)
    for ws in wss:
        assert moe.get_device_error(ws) == moe.MOE_OK

    keep, scale = dropout_keep(0, T * d, 0, 99, 7, p)
    keep = keep.view(T, d).cuda().to(F64) * scale
    v = {q: getattr(block, q).to(F64).requires_grad_(True) for q in
         ("Wg", "bias", "W1", "W2", "w_pre", "w_post", "w_next", "gate")}
    v["x"] = x.to(F64).requires_grad_(True)

    def normed(u, w):
        return u / torch.sqrt(u.square().mean(1, keepdim=True) + 1e-6) * w

    a = rounded(normed(v["x"], v["w_pre"]))
    L = a @ v["Wg"] + v["bias"]
    idx = torch.topk(L.detach(), k).indices
    # (tokens whose choice could fall either way at the kernel's precision)
    top = torch.sort(L.detach(), 1, descending=True).values
    gap = (top[:, k - 1] - top[:, k]) if k < E else torch.ones(T)
    assert float(gap.min()) > 1e-5
    w = torch.softmax(torch.gather(L, 1, idx), 1)
    b = torch.zeros_like(a)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            order = torch.argsort(t)
            t, j = t[order], j[order]
            we = w[t, j][:, None]
            b = b.index_add(0, t, we * Expert.apply(a[t], v["W1"][e], v["W2"][e], we.detach()))
    b = rounded(rounded(b) * keep)
    y = 0.5 * v["x"] + 1.5 * v["gate"] * normed(b, v["w_post"])
    nn = normed(y, v["w_next"])
    want_loss, counts = router_loss(L, idx, k, [0, T], None, 0.3, 0.2)
    total = (y * dout.to(F64)).sum() + (nn * dnext.to(F64)).sum() + want_loss[0]
    want = dict(zip(v, torch.autograd.grad(total, list(v.values()))))
    assert torch.equal(loss.counts.long(), counts)
    near(loss.loss, want_loss.detach(), 1e-5)
    # out and n: rounded twice, and codes that fall the other way where the sides' values before
    # them straddle a border: a step of an eighth of itself in at most one value of a hundred
    # adds 0.125 / sqrt(100) of a sum's norm at the most
    near(out, y.detach(), 4 * half_step(BF) + 0.0125)
    near(n, nn.detach(), 4 * half_step(BF) + 0.0125)
    # the gradients: four quantisations on the way, and n, z, b, db, dh and dx rounded to bf16
    for name, g in want.items():
        near(grads[name], g, 8 * half_step(BF) + 4 * 0.0125, name)
