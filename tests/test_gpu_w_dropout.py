"""Dropout on the GPU against the generator in Python integers: which elements are kept is
compared exactly; a kept one is off by one rounding of fp32 and half a step of its type."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import U32, half_step
from train_plain import F64, dropout_keep

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def state_of(seed, step):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


def near(got, want, terms, dtype):
    tol = 2 * U32 * terms + half_step(dtype) * (want.abs() + 2 * U32 * terms)
    # (half a step of the least numbers)
    tol = tol + torch.finfo(dtype).smallest_normal * half_step(dtype)
    assert bool(((got.to(F64) - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 64), (7, 192), (33, 128)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999999])
def test_forward_and_backward(cuda_ok, dtype, T, d, p):
    dt, g = DT[dtype], gen(T + d)
    x = torch.randn((T, d), generator=g, device="cuda").to(dt)
    res = torch.randn((T, d), generator=g, device="cuda").to(dt)
    # both halves of the seed, its sign, a step past 32 bits (its low half counts)
    seed, step, site = -0x0123456789abcdef, (1 << 35) + 77, 3
    c = moe.dropout_config(T, d, dtype, p=p, site=site)
    keep, scale = dropout_keep(0, T * d, site, seed, step, p)
    keep = keep.view(T, d).cuda()
    kept = torch.where(keep, x.to(F64) * scale, torch.zeros((), dtype=F64, device="cuda"))
    st = state_of(seed, step)
    out = moe.dropout(c, x, st)
    near(out, kept, kept.abs(), dt)
    assert bool((out[~keep] == 0).all())
    assert torch.equal(moe.dropout_backward(c, x, st), out)
    both = moe.dropout(c, x, st, residual=res)
    near(both, kept + res.to(F64), kept.abs() + res.to(F64).abs(), dt)
    assert torch.equal(both[~keep], res[~keep])


def test_sites_steps_and_seeds_draw_their_own(cuda_ok):
    x = torch.ones((64, 1024), device="cuda")
    outs = []
    for site, seed, step in ((0, 5, 0), (1, 5, 0), (0, 6, 0), (0, 5, 1), (0, 5 + (1 << 32), 0)):
        c = moe.dropout_config(64, 1024, "f32", p=0.5, site=site)
        outs.append(moe.dropout(c, x, state_of(seed, step)) != 0)
    for i in range(5):
        # 65536 draws of one half: five standard deviations are 640
        assert abs(int(outs[i].sum()) - 32768) < 640
        for j in range(i):
            assert abs(int((outs[i] == outs[j]).sum()) - 32768) < 640


def test_a_launch_of_many_blocks(cuda_ok):
    # the last elements of a tensor of 84 million
    T, d = 16385, 5120
    x = torch.ones((T, d), dtype=torch.bfloat16, device="cuda")
    c = moe.dropout_config(T, d, p=0.25, site=9)
    out = moe.dropout(c, x, state_of(1 << 40, 3))
    for first in (0, T * d // 2 - 64, T * d - 8192):
        n = min(8192, T * d - first)
        keep, scale = dropout_keep(first, n, 9, 1 << 40, 3, 0.25)
        assert torch.equal((out.view(-1)[first:first + n] != 0).cpu(), keep)
    # 0.75 of 83.9 million: five standard deviations are 20000
    assert abs(int((out != 0).sum()) - 0.75 * T * d) < 20000


def test_elements_past_32_bits(cuda_ok):
    # groups of 8 past 2^29, elements past 2^32
    T, d = (1 << 16) + 5, 65536
    x = torch.ones((T, d), dtype=torch.bfloat16, device="cuda")
    c = moe.dropout_config(T, d, p=0.5, site=2)
    moe.dropout(c, x, state_of(11, 12), out=x)
    first = T * d - 4096
    keep, _ = dropout_keep(first, 4096, 2, 11, 12, 0.5)
    assert torch.equal((x.view(-1)[first:] != 0).cpu(), keep)
    keep, _ = dropout_keep((1 << 32) - 2048, 4096, 2, 11, 12, 0.5)
    assert torch.equal((x.view(-1)[(1 << 32) - 2048:][:4096] != 0).cpu(), keep)


def test_what_is_dropped_may_be_anything(cuda_ok):
    x = torch.full((16, 256), float("nan"), device="cuda")
    x[::2] = float("inf")
    res = torch.randn((16, 256), generator=gen(1), device="cuda")
    c = moe.dropout_config(16, 256, "f32", p=0.5)
    keep = dropout_keep(0, 16 * 256, 0, 3, 4, 0.5)[0].view(16, 256).cuda()
    out = moe.dropout(c, x, state_of(3, 4), residual=res)
    assert torch.equal(out[~keep], res[~keep]) and not bool(torch.isfinite(out[keep]).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(cuda_ok, dtype):
    x = torch.randn((33, 320), generator=gen(2), device="cuda").to(DT[dtype])
    res = torch.randn((33, 320), generator=gen(3), device="cuda").to(DT[dtype])
    c, st = moe.dropout_config(33, 320, dtype, p=0.3), state_of(7, 8)
    want = moe.dropout(c, x, st, residual=res)
    a, b = x.clone(), res.clone()
    moe.dropout(c, a, st, residual=res, out=a)
    moe.dropout(c, x, st, residual=b, out=b)
    assert torch.equal(a, want) and torch.equal(b, want)


def test_no_rows(cuda_ok):
    c = moe.dropout_config(0, 64)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert moe.dropout(c, x, state_of(1, 2)).shape == (0, 64)


def test_a_replayed_graph_draws_anew(cuda_ok):
    x = torch.ones((64, 512), device="cuda")
    c, st = moe.dropout_config(64, 512, "f32", p=0.5), state_of(9, 100)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = moe.dropout(c, x, st)
            back = moe.dropout_backward(c, x, st)
            st[1] += 1
    seen = []
    for i in range(3):
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        keep, _ = dropout_keep(0, 4096, 0, 9, 100 + i, 0.5)
        assert torch.equal((out.view(-1)[:4096] != 0).cpu(), keep)
        assert torch.equal(out, back)
        seen.append(out.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
