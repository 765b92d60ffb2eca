"""The example block (norms, the experts in each of their forms, gate and residual) on the GPU,
against plain 64-bit compositions. What is rounded between the calls is rounded here too, so the
tolerances are those of the calls."""
import os
import sys

import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import F64, choose, half_step, mx4_quantize, mx4_values, norm_forward

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
from expert_block import ExpertBlock  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rows(T, d, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((T, d), generator=g, device="cuda").to(BF)


def plain(block, x, quantized):
    """(out, n, sure): the block's outputs in 64 bits, and the tokens whose choice is."""
    w = {k: getattr(block, k).to(F64) for k in
         ("Wg", "bias", "w_pre", "w_post", "w_next", "gate")}
    n = norm_forward(x.to(F64), None, None, None, w["w_pre"], "none", 1e-6, 1, 1)["n"][0]
    n = n.to(BF).to(F64)
    idx, wt, gap = choose(n @ w["Wg"] + w["bias"], 0, block.k, 8, 1, 1)

    def four(v):
        return mx4_values(*mx4_quantize(v)) if quantized else v

    b = torch.zeros_like(n)
    for e in range(block.E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        W1, W2 = block.W1[e].to(F64), block.W2[e].to(F64)
        z = four(n[t]) @ (four(W1.t()).t() if quantized else W1)
        h = z * torch.sigmoid(z)
        if quantized:
            h = four(h.to(BF).to(F64))
        b[t] += wt[t, j][:, None] * (h @ (four(W2.t()).t() if quantized else W2))
    f = norm_forward(x.to(F64), b.to(BF).to(F64), w["w_post"], w["gate"], w["w_next"], "channel",
                     1e-6, block.alpha, block.beta)
    return f["out"][0], f["n"][0], gap.cuda() > 1e-3


def near(got, want, limit):
    err = float((got.to(F64) - want).norm() / want.norm())
    assert err <= limit, err


# n and b are rounded to bf16 before their next use on both sides; where the two sides' values
# straddle a border those roundings differ by a step, and out and n are rounded once: four half
# steps of bf16 bound the norm of the difference
LIMIT = 4 * half_step(BF)


@pytest.mark.parametrize("T", [1, 5, 32])
def test_decode(cuda_ok, T):
    block = ExpertBlock(512, 384, 16, 2, alpha=0.5, beta=1.5, seed=T)
    x = rows(T, 512, T)
    ws = moe.alloc_workspace(block.config(T), "few")
    out, n = block.decode(x, ws)
    assert moe.get_device_error(ws) == moe.MOE_OK
    want_out, want_n, sure = plain(block, x, False)
    assert int((~sure).sum()) <= 1
    near(out[sure], want_out[sure], LIMIT)
    near(n[sure], want_n[sure], LIMIT)


@pytest.mark.parametrize("T", [3, 700])
def test_prefill_in_4_bits(cuda_ok, T):
    block = ExpertBlock(512, 384, 16, 2, seed=T).quantize()
    x = rows(T, 512, T)
    ws = moe.alloc_workspace(block.config(T), "scratch")
    mws = moe.alloc_mx4_workspace(moe.mx4_config(1, 512, 384, 16))
    out, n = block.prefill(x, ws, mws)
    assert moe.get_device_error(ws) == moe.MOE_OK and moe.get_device_error(mws) == moe.MOE_OK
    want_out, want_n, sure = plain(block, x, True)
    # a value at a 4-bit border may fall either way: a step of a quarter of itself in at most
    # one value of a hundred of a row adds 0.25 / sqrt(100) / 6 of that row at the most
    assert int(sure.sum()) >= T - 1 - T // 50
    near(out[sure], want_out[sure], LIMIT + 0.005)
    near(n[sure], want_n[sure], LIMIT + 0.005)


def test_train_step_gradients(cuda_ok):
    # against the formula's gradients by differentiation in 64 bits
    T, d = 64, 256
    block = ExpertBlock(d, 128, 4, 4, alpha=0.5, beta=1.5, seed=1)  # every expert: no choice
    x = rows(T, d, 2)
    dout, dnext = rows(T, d, 3), rows(T, d, 4).float()
    out, n, grads, (ws, bws) = block.train_step(x, dout, dnext)
    assert moe.get_device_error(ws) == moe.MOE_OK and moe.get_device_error(bws) == moe.MOE_OK

    p = {k: getattr(block, k).to(F64).requires_grad_(True) for k in
         ("Wg", "bias", "W1", "W2", "w_pre", "w_post", "w_next", "gate")}
    p["x"] = x.to(F64).requires_grad_(True)

    def normed(v, w):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6) * w

    a = normed(p["x"], p["w_pre"])
    wt = torch.softmax(a @ p["Wg"] + p["bias"], 1)
    b = torch.zeros_like(a)
    for e in range(4):
        z = a @ p["W1"][e]
        b = b + wt[:, e:e + 1] * ((z * torch.sigmoid(z)) @ p["W2"][e])
    y = 0.5 * p["x"] + 1.5 * p["gate"] * normed(b, p["w_post"])
    nn = normed(y, p["w_next"])
    loss = (y * dout.to(F64)).sum() + (nn * dnext.to(F64)).sum()
    want = dict(zip(p, torch.autograd.grad(loss, list(p.values()))))
    # n, h, b, db and dx are rounded to bf16 on the way: at most eight half steps in each
    # gradient's norm
    for k, v in want.items():
        near(grads[k], v, 8 * half_step(BF))
    near(out, y.detach(), LIMIT)
    near(n, nn.detach(), LIMIT)


def test_decode_step_in_a_graph(cuda_ok):
    block = ExpertBlock(512, 384, 16, 2, seed=3)
    x = rows(4, 512, 5)
    ws = moe.alloc_workspace(block.config(4), "few")
    out, n = block.decode(x, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            o2, n2 = block.decode(x, ws)
        for _ in range(3):
            o2.zero_()
            graph.replay()
        s.synchronize()
    assert torch.equal(out, o2) and torch.equal(n, n2)
