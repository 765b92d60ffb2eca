"""The router's losses on the GPU against their plain form in 64 bits. Sums over E experts, then
over tokens in chunks, in fp32: a term passes fewer than 64 + T / 300 roundings, and exp, log and
the quotients add about 16 half steps: 128 + T / 256 half steps of the (positive) terms for the
losses and their parts. lse and p are off by half steps of |L - max| too, in exp's argument."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import U32
from train_plain import F64, router_loss, router_loss_gradient

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def problem(T, E, k, seed=0, std=1.0):
    g = gen(seed)
    L = std * (torch.randn((T, E), generator=g, device="cuda")
               + 0.5 * torch.randn((1, E), generator=g, device="cuda"))
    return L, torch.topk(L, k, dim=1).indices.to(torch.int32)


def check(L, idx, offs=None, mask=None, balance=0.02, z=0.003, dloss=None, ws=None):
    T, E = L.shape
    k = idx.shape[1]
    c = moe.router_loss_config(T, E, k, S=1 if offs is None else len(offs) - 1, balance=balance,
                               z=z)
    ws = moe.alloc_router_loss_workspace(c) if ws is None else ws
    off = None if offs is None else torch.tensor(offs, dtype=torch.int32, device="cuda")
    r = moe.router_loss(c, L, idx, ws=ws, offsets=off, mask=mask)
    dl = None if dloss is None else torch.tensor([dloss], device="cuda")
    g = moe.router_loss_backward(c, L, r, dloss=dl, offsets=off, mask=mask)
    assert moe.get_device_error(ws) == moe.MOE_OK
    offs = [0, T] if offs is None else offs
    L64 = L.to(F64)
    want, counts = router_loss(L64, idx, k, offs, mask, balance, z)
    assert torch.equal(r.counts.long(), counts)
    n = [int(mask[a:b].bool().sum()) if mask is not None else b - a
         for a, b in zip(offs, offs[1:])]
    assert r.tokens.tolist() == n + [sum(v > 0 for v in n), sum(n)]
    span = float((L64.max() - L64.min()).clamp(min=1)) if T else 1.0
    rel = (128 + T / 256 + 4 * span) * U32
    # z's terms are squares: twice the relative error of lse, whose absolute one is half steps of
    # the largest logit
    top = float(L64.abs().max()) if T else 0.0
    assert abs(float(r.loss[1]) - float(want[1])) <= rel * float(want[1])
    assert abs(float(r.loss[2]) - float(want[2])) <= rel * (float(want[2]) + (top + 8) ** 2)
    both = abs(balance) * float(want[1]) + abs(z) * (float(want[2]) + (top + 8) ** 2)
    assert abs(float(r.loss[0]) - float(want[0])) <= rel * both
    # the gradient: a p times a difference, each known to rel of its terms
    v = 1.0 if dloss is None else dloss
    gw = v * router_loss_gradient(L64, idx, k, offs, mask, balance, z)
    p = torch.softmax(L64, 1)
    tol = torch.zeros_like(gw)
    used = max(1, sum(m > 0 for m in n))
    for s, (a, b) in enumerate(zip(offs, offs[1:])):
        if n[s]:
            f = E * counts[s].to(F64) / (k * n[s])
            tol[a:b] = abs(v) * p[a:b] * (
                abs(balance) / (used * n[s]) * (f + (p[a:b] * f).sum(1, keepdim=True))
                + 2 * abs(z) / sum(n) * (torch.logsumexp(L64[a:b], 1, keepdim=True).abs() + top))
    # (below 2^-126 p is known to two steps of 2^-149, and its factor is below 2^8)
    assert bool(((g.to(F64) - gw).abs() <= rel * tol + 2.0 ** -140).all())
    return r, g


@pytest.mark.parametrize("T", [1, 7, 8, 9, 255, 2433])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (33, 3), (64, 2), (256, 8), (16, 16)])
def test_batch(cuda_ok, T, E, k):
    check(*problem(T, E, k, seed=T + E))


@pytest.mark.parametrize("E,k", [(8, 2), (65, 4), (256, 8)])
def test_sequences(cuda_ok, E, k):
    # of one token, of none, tokens before the first and behind the last, masked tokens, a
    # sequence that is masked whole
    L, idx = problem(700, E, k, seed=E)
    mask = torch.rand((700,), generator=gen(1), device="cuda") > 0.2
    mask[300:420] = False
    for offs in ([0, 700], [3, 3, 4, 300, 420, 650], [0, 1, 2, 3, 699], [0] * 9 + [700],
                 [0, 350, 700]):
        check(L, idx, offs)
        check(L, idx, offs, mask, dloss=-1.75)
    check(L, idx, None, mask.to(torch.uint8))


def test_many_sequences(cuda_ok):
    L, idx = problem(5000, 40, 2, seed=3)
    cut = torch.sort(torch.randint(0, 5001, (998,), generator=gen(4), device="cuda")).values
    check(L, idx, [0] + cut.tolist() + [5000])


def test_more_sequences_than_tokens(cuda_ok):
    L, idx = problem(50, 16, 2, seed=12)
    cut = torch.sort(torch.randint(0, 51, (69998,), generator=gen(5), device="cuda")).values
    c = moe.router_loss_config(50, 16, 2, S=69999, balance=0.5, z=0.1)
    off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), 50)]).to(torch.int32)
    r = moe.router_loss(c, L, idx, ws=moe.alloc_router_loss_workspace(c), offsets=off)
    # the sequences of none do not matter
    some = torch.unique(off)
    c2 = moe.router_loss_config(50, 16, 2, S=len(some) - 1, balance=0.5, z=0.1)
    r2 = moe.router_loss(c2, L, idx, ws=moe.alloc_router_loss_workspace(c2), offsets=some)
    assert torch.allclose(r.loss, r2.loss, rtol=1e-5)
    assert r.tokens[-2:].tolist() == r2.tokens[-2:].tolist()
    g = moe.router_loss_backward(c, L, r, offsets=off)
    assert torch.allclose(g, moe.router_loss_backward(c2, L, r2, offsets=some), rtol=1e-5, atol=1e-9)


def test_long_batch(cuda_ok):
    check(*problem(70000, 64, 6, seed=5))


def test_wide_logits_and_masked_experts(cuda_ok):
    L, idx = problem(300, 64, 2, seed=6, std=30.0)
    check(L, idx)
    # experts that a token may not take: their p is 0, and so is their gradient
    L = torch.where(torch.rand_like(L) < 0.3, -float("inf"), L)
    idx = torch.topk(L, 2, dim=1).indices.to(torch.int32)
    c = moe.router_loss_config(300, 64, 2, balance=1.0, z=0.1)
    r = moe.router_loss(c, L, idx, ws=moe.alloc_router_loss_workspace(c))
    g = moe.router_loss_backward(c, L, r)
    want, _ = router_loss(L.to(F64), idx, 2, [0, 300], None, 1.0, 0.1)
    assert torch.allclose(r.loss.to(F64), want, rtol=1e-4)
    assert not bool(g[L == -float("inf")].any()) and bool(torch.isfinite(g).all())


def test_what_masked_tokens_hold_does_not_matter(cuda_ok):
    L, idx = problem(64, 16, 2, seed=7)
    mask = torch.ones(64, dtype=torch.bool, device="cuda")
    mask[10:20] = False
    a = check(L, idx, [0, 30, 60], mask)
    bad, worse = L.clone(), idx.clone()
    bad[10:20] = float("nan")
    bad[60:] = float("inf")
    worse[10:20] = -5
    worse[60:] = 1 << 30
    c = moe.router_loss_config(64, 16, 2, S=2, balance=0.02, z=0.003)
    ws = moe.alloc_router_loss_workspace(c)
    off = torch.tensor([0, 30, 60], dtype=torch.int32, device="cuda")
    r = moe.router_loss(c, bad, worse, ws=ws, offsets=off, mask=mask)
    g = moe.router_loss_backward(c, bad, r, offsets=off, mask=mask)
    assert moe.get_device_error(ws) == moe.MOE_OK
    assert torch.equal(r.loss, a[0].loss) and torch.equal(g, a[1])


def test_nan_is_passed_on(cuda_ok):
    L, idx = problem(64, 16, 2, seed=8)
    L[5, 3] = float("nan")
    c = moe.router_loss_config(64, 16, 2)
    r = moe.router_loss(c, L, idx, ws=moe.alloc_router_loss_workspace(c))
    assert bool(r.loss[1:].isnan().all())


def test_no_tokens(cuda_ok):
    for offs, T in ((None, 0), ([0, 0, 0], 0), ([4, 4, 4], 9)):
        L, idx = torch.zeros((T, 8), device="cuda"), torch.zeros((T, 2), dtype=torch.int32,
                                                                 device="cuda")
        r, g = check(L, idx, offs)
        assert r.loss.tolist() == [0, 0, 0] and not bool(g.any())
    L, idx = problem(9, 8, 2)
    r, g = check(L, idx, None, torch.zeros(9, dtype=torch.bool, device="cuda"))
    assert r.loss.tolist() == [0, 0, 0] and not bool(g.any())


@pytest.mark.parametrize("offs", [[0, 5, 4, 64], [0, 2, 3, 65], [-1, 2, 3, 64]])
def test_bad_offsets(cuda_ok, offs):
    L, idx = problem(64, 8, 2)
    c = moe.router_loss_config(64, 8, 2, S=3)
    ws = moe.alloc_router_loss_workspace(c)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 5, 5, 64], dtype=torch.int32, device="cuda")
    r = moe.router_loss(c, L, idx, ws=ws, offsets=good)
    kept = [t.clone() for t in r[:3]]
    ptrs = [t.data_ptr() for t in r]
    st = moe._lib.load().moe_router_loss(
        moe.api.ctypes.byref(c), L.data_ptr(), idx.data_ptr(), off.data_ptr(), None, *ptrs,
        ws.data_ptr(), ws.nbytes, torch.cuda.current_stream().cuda_stream)
    assert st == moe.MOE_OK
    assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(r[:3], kept))
    # the workspace is as good as before
    check(L, idx, [0, 5, 5, 64], ws=ws)


def test_bad_choices_are_flagged_and_not_counted(cuda_ok):
    L, idx = problem(64, 8, 2)
    idx[3, 1], idx[9, 0] = 8, -1
    c = moe.router_loss_config(64, 8, 2)
    ws = moe.alloc_router_loss_workspace(c)
    r = moe.router_loss(c, L, idx, ws=ws)
    assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX
    assert int(r.counts.sum()) == 126


def test_same_bits_again_and_in_a_graph(cuda_ok):
    L, idx = problem(6000, 256, 8, seed=9)
    off = torch.tensor([0, 100, 100, 4000, 6000], dtype=torch.int32, device="cuda")
    c = moe.router_loss_config(6000, 256, 8, S=4, z=0.1)
    ws = moe.alloc_router_loss_workspace(c)
    want = moe.router_loss(c, L, idx, ws=ws, offsets=off)
    g0 = moe.router_loss_backward(c, L, want, offsets=off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            r = moe.router_loss(c, L, idx, ws=ws, offsets=off)
            g = moe.router_loss_backward(c, L, r, offsets=off)
        for _ in range(10):
            r.loss.zero_()
            g.zero_()
            graph.replay()
            s.synchronize()
            assert torch.equal(r.loss, want.loss) and torch.equal(g, g0)
            assert torch.equal(r.counts, want.counts)


def test_in_the_layers_backward(cuda_ok):
    """dlogits joins the router's gradient: x, W_g and the bias get its share, the experts none."""
    for dtype, E, T, d in (("bf16", 64, 192, 256), ("f32", 8, 70, 128), ("bf16", 12, 40, 128)):
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        g = gen(11)

        def draw(*shape, std=1.0, to=dt):
            return (std * torch.randn(shape, generator=g, device="cuda")).to(to)

        f, k = 128, 2
        x, Wg, bias = draw(T, d), draw(d, E, std=d ** -0.5), draw(E, to=torch.float32)
        W1, W2 = draw(E, d, f, std=d ** -0.5), draw(E, f, d, std=f ** -0.5)
        dout = draw(T, d)
        c = moe.make_config(T, d, E, k, f, dtype)
        ws, bws = moe.alloc_workspace(c), moe.alloc_workspace(c, "backward")
        moe.forward(c, x, Wg, bias, W1, W2, ws=ws)
        idx, _, L = moe.route(c, x, Wg, bias, want_logits=True)
        lc = moe.router_loss_config(T, E, k, balance=0.5, z=0.1)
        r = moe.router_loss(lc, L, idx, ws=moe.alloc_router_loss_workspace(lc))
        dL = moe.router_loss_backward(lc, L, r)
        a = moe.backward(c, x, Wg, bias, W1, W2, dout, fwd_ws=ws, ws=bws)
        b = moe.backward(c, x, Wg, bias, W1, W2, dout, fwd_ws=ws, ws=bws, dlogits=dL)
        assert moe.get_device_error(bws) == moe.MOE_OK
        assert torch.equal(a["dW1"], b["dW1"]) and torch.equal(a["dW2"], b["dW2"])
        assert not torch.equal(a["dWg"], b["dWg"])
        # alone, where nothing comes from the output: dL through the gate, in bf16 layers in two
        # bf16 parts (2^-17 of it is lost), sums of n terms in n / 8 + 64 half steps
        b = moe.backward(c, x, Wg, bias, W1, W2, torch.zeros_like(dout), fwd_ws=ws, ws=bws,
                         dlogits=dL)
        assert not bool(b["dW1"].any()) and not bool(b["dW2"].any())
        lost = 2.0 ** -17 if dtype == "bf16" else 0.0
        D, X, G = dL.to(F64), x.to(F64), Wg.to(F64)
        for got, want, terms, n in ((b["dx"], D @ G.t(), D.abs() @ G.abs().t(), E),
                                    (b["dWg"], X.t() @ D, X.abs().t() @ D.abs(), T),
                                    (b["dbias"], D.sum(0), D.abs().sum(0), T)):
            assert bool(((got.to(F64) - want).abs() <= (lost + (n / 8 + 64) * U32) * terms).all())
