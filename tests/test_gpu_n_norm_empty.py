"""The norms around a block with no rows: a token or element gate's gradient is then empty, and
an empty tensor has no address."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["none", "token", "channel", "element"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pre", [True, False])
def test_no_rows_with_each_gate(cuda_ok, kind, dtype, pre):
    d, td = 128, torch.bfloat16 if dtype == "bf16" else torch.float32
    c = moe.norm_config(0, d, dtype, gate=kind)
    e = torch.empty((0, d), dtype=td, device="cuda")
    w = torch.ones(d, device="cuda")
    gate = {"none": None, "token": torch.empty(0, device="cuda"), "channel": w, "element": e}[kind]
    w_pre, dn = (w, torch.empty((0, d), device="cuda")) if pre else (None, None)
    r = moe.block_norm(c, e, e, w, gate, w_pre, want_rstd=True)
    g = moe.block_norm_backward(c, e, dn, r["out"], e, w, gate, w_pre, r["rstd_post"],
                                r["rstd_pre"], ws=moe.alloc_norm_workspace(c))
    assert g["dx"].shape == g["db"].shape == (0, d)
    assert bool((g["dw_post"] == 0).all()) and (not pre or bool((g["dw_pre"] == 0).all()))
    if kind != "none":
        assert g["dgate"].shape == gate.shape and bool((g["dgate"] == 0).all())
