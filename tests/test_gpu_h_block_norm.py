"""The norms around a block on the GPU against the plain 64-bit forms.

Tolerances: an output may be off by half a step of its type (its one rounding), and by the fp32
roundings of the terms it is made of. A row's sums add d values, at most 128 in a thread for the
lengths here and then a tree (relative error of a sum of positive terms below 140 half steps of
fp32); the terms around them add fewer than 20 roundings: 256 half steps of fp32 of the absolute
terms cover both. A column sum adds T rows in some order: T more half steps."""
import itertools

import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import F64, U32, half_step, norm_backward, norm_forward, norm_problem

pytestmark = pytest.mark.gpu
TERMS = 256


def check(name, got, want, dtype, rows=0):
    value, terms = want
    got = got.cpu().to(F64)
    assert got.shape == value.shape, name
    tol = half_step(dtype) * value.abs() + (TERMS + rows) * U32 * terms
    # what is stored below the type's smallest normal number is off by its smallest step
    tol = tol + torch.finfo(dtype).smallest_normal
    over = (got - value).abs() - tol
    assert bool((over <= 0).all()), (name, float(over.max()), float((got - value).abs().max()))


def wide(t):
    return None if t is None else t.cpu().to(F64)


def both(T, d, dtype, kind, post, pre, seed=0, alpha=0.75, beta=1.5, eps=1e-5, i=None):
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    i = i or norm_problem(T, d, dt, kind, post, pre, seed, "cuda")
    c = moe.norm_config(T, d, dtype, gate=kind, eps=eps, alpha=alpha, beta=beta)
    r = moe.block_norm(c, i["x"], i["b"], i["w_post"], i["gate"], i["w_pre"], want_rstd=True)
    w = {k: wide(v) for k, v in i.items()}
    k = kind if post else "none"
    f = norm_forward(w["x"], w["b"], w["w_post"], w["gate"], w["w_pre"], k, eps, alpha, beta)
    kept = r["rstd_pre"]
    if post and pre:
        assert isinstance(kept, moe.KeptNorm) and kept.x is i["x"]
        r = {**r, "rstd_pre": kept.rstd}
    for name, want in f.items():
        check(name, r[name], want, torch.float32 if name.startswith("rstd") else dt)
    ws = moe.alloc_norm_workspace(c)
    ws.fill_(0xff)  # the workspace needs no zeroing: NaN bytes must not show
    g = moe.block_norm_backward(c, i["dout"], i["dn"], r["out"] if post else i["x"], i["b"], i["w_post"], i["gate"],
                                i["w_pre"], r["rstd_post"], kept, ws=ws)
    y64, ay = f["out"] if post else (w["x"], w["x"].abs())
    want = norm_backward(w["dout"], w["dn"], y64, w["b"], w["w_post"], w["gate"], w["w_pre"],
                         wide(r["rstd_post"]), wide(r["rstd_pre"]), k, alpha, beta, ay)
    assert {n for n, v in g.items() if v is not None} == set(want)
    for name, val in want.items():
        full = name in ("dx", "db") or (name == "dgate" and kind == "element")
        cols = name.startswith("dw") or (name == "dgate" and kind == "channel")
        check(name, g[name], val, dt if full else torch.float32, T if cols else 0)
    return r, g


@pytest.mark.parametrize("dtype,kind,halves", list(itertools.product(
    ["bf16", "f32"], ["none", "token", "channel", "element"],
    [(True, True), (True, False), (False, True)])))
def test_each_form(cuda_ok, dtype, kind, halves):
    both(37, 320, dtype, kind, *halves)


# each way a row is shared: a warp, 128, 256, 512 threads, rows too wide for registers; few
# rows and many; the last vectors of a row held by some threads only
@pytest.mark.parametrize("T,d", [(1, 64), (1, 7168), (2, 4160), (3, 8192), (5, 16384), (2, 65536),
                                 (153, 64), (160, 576), (300, 1088), (155, 2112), (700, 4096),
                                 (161, 5184), (333, 7168), (154, 16448), (2440, 192)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths(cuda_ok, T, d, dtype):
    both(T, d, dtype, "channel", True, True, seed=T + d)


@pytest.mark.parametrize("T,d,kind", [(1, 64, "token"), (300, 2048, "channel"),
                                      (77, 7168, "element"), (9, 20480, "none")])
def test_weights_gradients_follow_the_unrounded_forward(cuda_ok, T, d, kind):
    # against the formula's gradients of the unrounded chain: out is formed in fp32 for them, not
    # read as bf16, so no sum is off by 2^-16 of its terms, nor of its value
    i = norm_problem(T, d, torch.bfloat16, kind, True, True, 4, "cuda")
    c = moe.norm_config(T, d, gate=kind, alpha=0.75, beta=1.5)
    r = moe.block_norm(c, i["x"], i["b"], i["w_post"], i["gate"], i["w_pre"], want_rstd=True)
    g = moe.block_norm_backward(c, i["dout"], i["dn"], r["out"], i["b"], i["w_post"], i["gate"],
                                i["w_pre"], r["rstd_post"], r["rstd_pre"],
                                ws=moe.alloc_norm_workspace(c))
    w = {k: wide(v) for k, v in i.items()}
    f = norm_forward(w["x"], w["b"], w["w_post"], w["gate"], w["w_pre"], kind, 1e-6, 0.75, 1.5)
    want = norm_backward(w["dout"], w["dn"], f["out"][0], w["b"], w["w_post"], w["gate"],
                         w["w_pre"], f["rstd_post"][0], f["rstd_pre"][0], kind, 0.75, 1.5)
    for name in ("dw_pre", "dw_post") + (("dgate",) if kind in ("token", "channel") else ()):
        value, terms = want[name]
        tol = (2.0 ** -16 + (TERMS + T) * U32) * terms
        assert bool(((g[name].cpu().to(F64) - value).abs() <= tol).all()), name
        err = float((g[name].cpu().to(F64) - value).norm() / value.norm())
        assert err <= 2.0 ** -16, (name, err)


def test_empty_batch(cuda_ok):
    c = moe.norm_config(0, 128, "bf16", gate="channel")
    e = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, device="cuda")
    r = moe.block_norm(c, e, e, w, w, w, want_rstd=True)
    assert r["n"].shape == (0, 128)
    g = moe.block_norm_backward(c, e, torch.empty((0, 128), device="cuda"), e, e, w, w, w,
                                r["rstd_post"], r["rstd_pre"], ws=moe.alloc_norm_workspace(c))
    for name in ("dw_post", "dw_pre", "dgate"):
        assert bool((g[name] == 0).all()), name


def test_zero_rows_and_values_at_the_ends(cuda_ok):
    # a zero row: rstd = 1 / sqrt(eps); infinities and NaN stay in their own row
    i = norm_problem(6, 256, torch.float32, "none", True, True, 1)
    i["b"][0] = 0
    i["x"][1] = 0
    i["b"][1] = 0
    i = {k: None if v is None else v.cuda() for k, v in i.items()}
    r, _ = both(6, 256, "f32", "none", True, True, i=i)
    clean = {k: v.clone() for k, v in r.items() if k in ("out", "n")}
    i["b"][3, 7] = float("nan")
    i["x"][4, 9] = float("inf")
    c = moe.norm_config(6, 256, "f32", alpha=0.75, beta=1.5, eps=1e-5)
    r = moe.block_norm(c, i["x"], i["b"], i["w_post"], None, i["w_pre"])
    for t in (0, 1, 2, 5):
        assert torch.equal(r["n"][t], clean["n"][t]) and torch.equal(r["out"][t], clean["out"][t])
    assert bool(r["n"][3].isnan().all()) and bool(r["n"][4, 9].isnan())


def test_same_bits_again_and_in_a_graph_on_another_stream(cuda_ok):
    T, d = 777, 2048
    i = norm_problem(T, d, torch.bfloat16, "channel", True, True, 5, "cuda")
    c = moe.norm_config(T, d, "bf16", gate="channel")
    ws = moe.alloc_norm_workspace(c)

    def step():
        r = moe.block_norm(c, i["x"], i["b"], i["w_post"], i["gate"], i["w_pre"], want_rstd=True)
        g = moe.block_norm_backward(c, i["dout"], i["dn"], r["out"], i["b"], i["w_post"],
                                    i["gate"], i["w_pre"], r["rstd_post"], r["rstd_pre"], ws=ws)
        return [r["out"], r["n"]] + [g[k] for k in sorted(g)]

    first = [t.clone() for t in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = step()
        for t in outs:
            t.zero_()
        graph.replay()
    s.synchronize()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)
