"""The plain norm gradients the GPU tests compare with, against autograd and against central
differences of the plain forward (CPU, 64 bits)."""
import itertools

import pytest
import torch

from block_plain import F64, norm_backward, norm_forward, norm_problem

EPS = 1e-5


def _wide(i):
    return {k: None if v is None else v.to(F64) for k, v in i.items()}


@pytest.mark.parametrize("kind,halves", list(itertools.product(
    ["none", "token", "channel", "element"], [(True, True), (True, False), (False, True)])))
def test_gradients_match_autograd_and_differences(kind, halves):
    post, pre = halves
    i = _wide(norm_problem(5, 64, torch.float32, kind, post, pre, 3))
    alpha, beta = 0.75, 1.5
    names = [k for k in ("x", "b", "w_post", "gate", "w_pre") if i[k] is not None]

    def loss(t):
        r = norm_forward(t["x"], t["b"], t["w_post"], t["gate"], t["w_pre"],
                         kind if post else "none", EPS, alpha, beta)
        y = r["out"][0] if post else t["x"]
        s = (y * i["dout"]).sum()
        return s + (r["n"][0] * i["dn"]).sum() if pre else s

    t = {k: None if v is None else v.clone().requires_grad_(True) for k, v in i.items()}
    auto = dict(zip(names, torch.autograd.grad(loss(t), [t[k] for k in names])))
    f = norm_forward(i["x"], i["b"], i["w_post"], i["gate"], i["w_pre"], kind if post else "none",
                     EPS, alpha, beta)
    y = f["out"][0] if post else i["x"]
    got = norm_backward(i["dout"], i["dn"], y, i["b"], i["w_post"], i["gate"], i["w_pre"],
                        f["rstd_post"][0] if post else None, f["rstd_pre"][0] if pre else None,
                        kind, alpha, beta)
    grad_of = {"x": "dx", "b": "db", "w_post": "dw_post", "gate": "dgate", "w_pre": "dw_pre"}
    for k in names:
        torch.testing.assert_close(got[grad_of[k]][0], auto[k], rtol=1e-10, atol=1e-10)
        # central differences along a random direction: error O(h^2), h = 1e-5
        v = torch.randn(i[k].shape, generator=torch.Generator().manual_seed(1), dtype=F64)
        h = 1e-5
        num = (loss({**i, k: i[k] + h * v}) - loss({**i, k: i[k] - h * v})) / (2 * h)
        assert abs(num - (got[grad_of[k]][0] * v).sum()) <= 1e-6 * (1 + abs(num))
