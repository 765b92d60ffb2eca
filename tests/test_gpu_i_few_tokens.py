"""The whole layer for a few tokens, on the GPU, against the plain 64-bit layer (its tolerance
is derived there, plus half a step of bf16 for the one rounding of out). Tokens whose choice
hangs on less than the logits' errors are left out; the inputs leave at most one a case."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import F64, few_layer, half_step
from workloads import MoEConfig, make_inputs

pytestmark = pytest.mark.gpu


def layer(T, d, E, k, f, router=0, seed=0, **kw):
    kw.setdefault("pre_k", min(8, E))
    return MoEConfig("few", T=T, d=d, E=E, k=k, f=f, dtype="bf16", router=router, seed=seed,
                     bias="normal", bias_var=0.5, **kw)


def compare(c, i, out, skip=1):
    want, tol, gap = few_layer(c, i)
    sure = gap > 1e-4
    assert int((~sure).sum()) <= skip
    got, want, tol = out.to(F64)[sure], want[sure], tol[sure]
    over = (got - want).abs() - (half_step(torch.bfloat16) * (want.abs() + tol) + tol)
    assert bool((over <= 0).all()), (float(over.max()), float((got - want).abs().max()))


def run(c, skip=1):
    i = make_inputs(c, device="cuda")
    ws = moe.alloc_workspace(c, "few")
    for _ in range(2):  # the second finds the counters as the first left them
        out = moe.forward_few(c, i["x"], i["Wg"], i["bias"], i["W1"], i["W2"], ws=ws,
                              noise=i.get("gumbel"))
        torch.cuda.synchronize()
        assert moe.get_device_error(ws) == moe.MOE_OK
        compare(c, i, out, skip)
    return i, ws, out


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 32])
def test_token_counts(cuda_ok, T):
    run(layer(T, 512, 16, 3, 320, seed=T))


# steps fewer than the grid's blocks; odd numbers of 64-wide blocks; one expert; experts not a
# multiple of 8 and more than one gate group; widths of the workload's layers
@pytest.mark.parametrize("T,d,E,k,f", [
    (1, 64, 1, 1, 64), (3, 64, 5, 2, 128), (32, 128, 8, 2, 256), (4, 192, 3, 3, 64),
    (5, 1088, 67, 8, 448), (32, 320, 256, 8, 64), (1, 2048, 64, 2, 1408), (2, 4096, 8, 2, 1088),
    (13, 7168, 9, 8, 192), (32, 64, 200, 1, 1984)])
def test_shapes(cuda_ok, T, d, E, k, f):
    run(layer(T, d, E, k, f, seed=d + f))


@pytest.mark.parametrize("router,kw", [
    (1, dict(pre_k=8)), (1, dict(pre_k=3)), (2, dict(n_group=8, topk_group=3)),
    (2, dict(n_group=4, topk_group=1))])
@pytest.mark.parametrize("T", [1, 6, 32])
def test_routers(cuda_ok, T, router, kw):
    run(layer(T, 256, 32, 3, 192, router=router, seed=T, **kw))


@pytest.mark.parametrize("T,E,tau", [(1, 16, 1.0), (32, 16, 0.5), (9, 3, 2.0)])
def test_soft_gating(cuda_ok, T, E, tau):
    run(layer(T, 320, E, E, 128, router=3, seed=T, tau=tau))


def test_every_token_to_the_same_experts(cuda_ok):
    # a bias that outweighs the logits: two experts take all 32 tokens, the others none
    c = layer(32, 256, 24, 2, 384, seed=3)
    i = make_inputs(c, device="cuda")
    i["bias"] = torch.zeros(24, device="cuda")
    i["bias"][[5, 17]] = torch.tensor([100.0, 90.0], device="cuda")
    ws = moe.alloc_workspace(c, "few")
    out = moe.forward_few(c, i["x"], i["Wg"], i["bias"], i["W1"], i["W2"], ws=ws)
    compare(c, i, out, 0)


def test_equal_logits_take_the_lower_ids(cuda_ok):
    # a zero gate and no bias: every logit is equal, so experts 0..k-1
    c = layer(5, 128, 12, 4, 128, seed=4)
    i = make_inputs(c, device="cuda")
    i["Wg"].zero_()
    ws = moe.alloc_workspace(c, "few")
    out = moe.forward_few(c, i["x"], i["Wg"], None, i["W1"], i["W2"], ws=ws)
    x = i["x"].to(F64)
    want = torch.zeros_like(x)
    for e in range(4):
        z = x @ i["W1"][e].to(F64)
        want += 0.25 * ((z * torch.sigmoid(z)) @ i["W2"][e].to(F64))
    torch.testing.assert_close(out.to(F64), want, rtol=2.0 ** -8, atol=1e-3)


def test_agrees_with_the_full_forward(cuda_ok):
    # the same choices and, up to h's rounding in the full forward, the same values
    c = layer(24, 512, 32, 4, 512, seed=6)
    i = make_inputs(c, device="cuda")
    few = moe.forward_few(c, i["x"], i["Wg"], i["bias"], i["W1"], i["W2"],
                          ws=moe.alloc_workspace(c, "few")).float()
    full = moe.forward(c, i["x"], i["Wg"], i["bias"], i["W1"], i["W2"],
                       ws=moe.alloc_workspace(c)).float()
    # h: half a step of bf16 on each term, random signs; out: half a step on each side
    assert float((few - full).norm() / full.norm()) <= 2 * 2.0 ** -8


def test_nan_rows_stay_alone_and_are_flagged_as_the_router_does(cuda_ok):
    # infinite activations make NaN logits; their token chooses nothing and the others keep
    # their values
    c = layer(8, 256, 8, 2, 128, seed=8)
    i, ws, out = run(c)
    x = i["x"].clone()
    x[3] = float("nan")
    bad = moe.forward_few(c, x, i["Wg"], i["bias"], i["W1"], i["W2"], ws=ws)
    torch.cuda.synchronize()
    assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX
    keep = [t for t in range(8) if t != 3]
    # without token 3 fewer experts may be read, so sums may be split elsewhere
    torch.testing.assert_close(bad[keep].float(), out[keep].float(), rtol=2.0 ** -7, atol=1e-4)


def test_same_bits_in_a_graph_on_another_stream(cuda_ok):
    c = layer(11, 1024, 64, 8, 704, seed=9)
    i, ws, out = run(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            again = moe.forward_few(c, i["x"], i["Wg"], i["bias"], i["W1"], i["W2"], ws=ws)
        for _ in range(20):
            again.zero_()
            graph.replay()
            s.synchronize()
            assert torch.equal(again, out)
    assert moe.get_device_error(ws) == moe.MOE_OK


def test_a_workspace_serves_layers_of_other_shapes(cuda_ok):
    big, small = layer(32, 512, 64, 8, 512, seed=1), layer(3, 128, 4, 2, 64, seed=2)
    ws = moe.alloc_workspace(big, "few")
    for c in (big, small, big, small):
        i = make_inputs(c, device="cuda")
        compare(c, i, moe.forward_few(c, i["x"], i["Wg"], i["bias"], i["W1"], i["W2"], ws=ws))
        assert moe.get_device_error(ws) == moe.MOE_OK


def test_no_tokens(cuda_ok):
    c = layer(0, 128, 8, 2, 128)
    i = make_inputs(c, device="cuda")
    out = moe.forward_few(c, i["x"], i["Wg"], i["bias"], i["W1"], i["W2"],
                          ws=moe.alloc_workspace(c, "few"))
    assert out.shape == (0, 128)
