"""The norms around a block at the ends of the fp32 range: rows of zeros with a very small eps
(rstd up to 1 / sqrt(eps)), rows whose root mean square is far above 1, rows whose sum of squares
passes the range (rstd 0, as the header says). Neither a square nor a cube of rstd has to fit
fp32, only the results do. Both forms: rows of the ring, and rows too wide for it.

Tolerances as in test_gpu_h_block_norm (derived there: 256 half steps of fp32 of the absolute
terms, T more for a column sum, half a step of the output's type)."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import norm_backward, norm_problem
from test_gpu_h_block_norm import both, check, wide

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# a warp's rows, a block's, rows too wide for the ring
LENGTHS = [192, 1088, 16448]
KINDS = ["none", "token", "channel", "element"]


def on_gpu(i):
    return {k: None if v is None else v.cuda() for k, v in i.items()}


@pytest.mark.parametrize("d", LENGTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,halves", [("none", (True, True)), ("token", (True, True)),
                                         ("channel", (True, True)), ("element", (True, True)),
                                         ("token", (True, False)), ("none", (False, True))])
@pytest.mark.parametrize("eps", [1e-30, 1e-37])
def test_zero_rows_with_a_small_eps(cuda_ok, d, dtype, kind, halves, eps):
    i = norm_problem(7, d, DT[dtype], kind, *halves, d)
    if halves[0]:
        i["b"][0] = 0       # the branch alone
        i["b"][1] = 0       # and the whole row
    i["x"][1] = 0
    both(7, d, dtype, kind, *halves, eps=eps, i=on_gpu(i))


@pytest.mark.parametrize("d", LENGTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [1e13, 2e15, 1e16])
def test_large_rows(cuda_ok, d, dtype, kind, scale):
    # dout of those rows is 0, so that their dx is what comes through the norm
    i = norm_problem(7, d, DT[dtype], kind, True, True, d)
    for name, rows in (("x", [1, 3]), ("b", [2, 3])):
        i[name][rows] = (i[name][rows].double() * scale).to(DT[dtype])
    i["dout"][1:4] = 0
    both(7, d, dtype, kind, True, True, i=on_gpu(i))


@pytest.mark.parametrize("d", LENGTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
def test_rows_past_the_range_have_rstd_0(cuda_ok, d, dtype, kind):
    alpha, beta = 0.75, 1.5
    i = norm_problem(7, d, DT[dtype], kind, True, True, d)
    i["b"][2] = torch.sign(i["b"][2]) * 3e38
    i["x"][4] = torch.sign(i["x"][4]) * 2.5e38
    i = on_gpu(i)
    c = moe.norm_config(7, d, dtype, gate=kind, alpha=alpha, beta=beta)
    r = moe.block_norm(c, i["x"], i["b"], i["w_post"], i["gate"], i["w_pre"], want_rstd=True)
    g = moe.block_norm_backward(c, i["dout"], i["dn"], None, i["b"], i["w_post"], i["gate"],
                                i["w_pre"], r["rstd_post"], r["rstd_pre"],
                                ws=moe.alloc_norm_workspace(c))
    rb, ro = wide(r["rstd_post"]), wide(r["rstd_pre"].rstd)
    assert rb[2] == 0 and ro[4] == 0
    w = {k: wide(v) for k, v in i.items()}
    gate = {"none": lambda v: 1.0, "token": lambda v: v[:, None]}.get(kind, lambda v: v)(w["gate"])
    branch = beta * gate * (w["b"] * rb[:, None] * w["w_post"])
    y, ay = alpha * w["x"] + branch, (alpha * w["x"]).abs() + branch.abs()
    check("out", r["out"], (y, ay), DT[dtype])
    n = y * ro[:, None] * w["w_pre"]
    # (the kept rstd is used: only the terms' own roundings)
    check("n", r["n"], (n, (ay * ro[:, None] * w["w_pre"]).abs() + n.abs()), DT[dtype])
    want = norm_backward(w["dout"], w["dn"], y, w["b"], w["w_post"], w["gate"], w["w_pre"], rb, ro,
                         kind, alpha, beta, ay)
    for name, val in want.items():
        full = name in ("dx", "db") or (name == "dgate" and kind == "element")
        cols = name.startswith("dw") or (name == "dgate" and kind == "channel")
        check(name, g[name], val, DT[dtype] if full else torch.float32, 7 if cols else 0)
