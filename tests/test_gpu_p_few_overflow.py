"""The layer for a few tokens where an expert's hidden values pass bf16's range: h is carried as
two bf16 parts, and the second part of an infinite value is not infinity minus infinity. A value
between bf16's largest and fp32's keeps its value."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import F64, half_step

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def run(x, W1, W2, T, E):
    d, f = W1.shape[1:]
    c = moe.make_config(T, d, E, 1, f, "bf16", pre_k=1)
    Wg = torch.zeros((d, E), dtype=BF, device="cuda")
    ws = moe.alloc_workspace(c, "few")
    out = moe.forward_few(c, x, Wg, None, W1, W2, ws=ws)
    torch.cuda.synchronize()
    assert moe.get_device_error(ws) == moe.MOE_OK
    return out, c, Wg


@pytest.mark.parametrize("T", [1, 5, 16, 32])
def test_infinite_hidden_values(cuda_ok, T):
    # token 0's first hidden value overflows to infinity; its outputs are infinities of W2's
    # signs, as the full forward has them, and the other tokens' are finite
    E, d, f = 2, 128, 192
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn((T, d), generator=g, device="cuda").to(BF)
    x[0] = 2.0 ** 120
    W1 = torch.randn((E, d, f), generator=g, device="cuda").to(BF)
    W1[:, :, 0] = 2.0 ** 10
    W1[:, :, 1:] = W1[:, :, 1:].abs() * -(2.0 ** -124)  # (SiLU of moderate values)
    x[1:, :] *= 2.0 ** -4
    W2 = torch.randn((E, f, d), generator=g, device="cuda").to(BF)
    W2[W2 == 0] = 1
    out, c, Wg = run(x, W1, W2, T, E)
    full = moe.forward(c, x, Wg, None, W1, W2, ws=moe.alloc_workspace(c))
    want = torch.sign(W2[0, 0].float()) * float("inf")
    assert torch.equal(full[0].float(), want)
    assert torch.equal(out[0].float(), want)
    assert bool(out[1:].isfinite().all())


@pytest.mark.parametrize("T", [1, 7])
def test_values_above_bf16s_largest(cuda_ok, T):
    # z = (1.9921875 + 0.005859375) 2^127 is finite in fp32 and past the middle between bf16's
    # largest value and 2^128, so it rounds to infinity in bf16
    E, d, f = 1, 64, 64
    x = torch.zeros((T, d), dtype=BF, device="cuda")
    x[:, :2] = torch.tensor([1.0, 1.5 * 2.0 ** -8], device="cuda").to(BF)
    W1 = torch.zeros((E, d, f), dtype=BF, device="cuda")
    W1[0, 0, 0] = torch.finfo(BF).max
    W1[0, 1, 0] = 2.0 ** 127
    W2 = torch.zeros((E, f, d), dtype=BF, device="cuda")
    W2[0, 0] = 2.0 ** -100
    out, _, _ = run(x, W1, W2, T, E)
    z = W1[0, :2, 0].to(F64) @ x[0, :2].to(F64)
    assert float(z) < torch.finfo(torch.float32).max
    want = z * 2.0 ** -100
    # h to 2^-17, sums of two terms, the rounding of out
    tol = (half_step(BF) + 2.0 ** -17 + 8 * half_step(torch.float32)) * want
    assert bool(((out.to(F64) - want).abs() <= tol).all()), (out[0, 0], want)
