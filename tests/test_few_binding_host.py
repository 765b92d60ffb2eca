"""The binding of the layer for a few tokens refuses tensors that are not the call's: another
length or type would be read, or written, past its end. Host tensors: each refusal comes before
the library is called (no GPU needed)."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from mixture_experts_routed_gb300 import build as B

BF = torch.bfloat16


def tensors(T=4, d=64, E=8, f=128):
    return dict(x=torch.zeros((T, d), dtype=BF), Wg=torch.zeros((d, E), dtype=BF),
                bias=torch.zeros(E), W1=torch.zeros((E, d, f), dtype=BF),
                W2=torch.zeros((E, f, d), dtype=BF), out=torch.zeros((T, d), dtype=BF))


def call(t, noise=None, **kw):
    c = moe.make_config(4, 64, 8, kw.pop("k", 2), 128, "bf16", **kw)
    return moe.forward_few(c, t["x"], t["Wg"], t["bias"], t["W1"], t["W2"], out=t["out"],
                           noise=noise, ws=torch.zeros(1 << 16, dtype=torch.uint8))


@pytest.mark.parametrize("name,shape", [
    ("x", (3, 64)), ("x", (4, 128)), ("Wg", (64, 4)), ("Wg", (8, 64)), ("bias", (4,)),
    ("W1", (8, 64, 64)), ("W1", (4, 64, 128)), ("W1", (8, 128, 64)), ("W2", (8, 64, 128)),
    ("W2", (2, 128, 64)), ("out", (3, 64)), ("out", (4, 32))])
def test_other_shapes(name, shape):
    B.build()
    t = tensors()
    t[name] = torch.zeros(shape, dtype=t[name].dtype)
    with pytest.raises(moe.MoEError, match=f"{name} is .* not "):
        call(t)


@pytest.mark.parametrize("name", ["x", "Wg", "bias", "W1", "W2", "out"])
def test_other_types(name):
    B.build()
    t = tensors()
    t[name] = t[name].to(torch.float16)
    with pytest.raises(moe.MoEError, match=f"{name} is .*float16, not "):
        call(t)


def test_samples_of_the_soft_router():
    B.build()
    soft = dict(k=8, router=moe.MOE_ROUTER_SOFT_GUMBEL, tau=1.0)
    for noise in (torch.zeros((4, 4)), torch.zeros((3, 8)), torch.zeros((4, 8), dtype=BF)):
        with pytest.raises(moe.MoEError, match="noise is .* not "):
            call(tensors(), noise=noise, **soft)
