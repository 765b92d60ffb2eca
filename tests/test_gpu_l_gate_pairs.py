"""The tensor-core gate with the contraction split over pairs of CTAs: a CTA writes its partial
sums into its peer's shared memory, where the peer's operands were, so it must not be early.
Fresh kernels before each call shift the two against each other; the result may not move."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,E,k", [(8192, 7168, 16, 2), (8192, 2048, 64, 2), (4097, 4096, 8, 2)])
def test_split_gate_repeats(T, d, E, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(T + d + E)
    c = moe.make_config(T, d, E, k, 1024, "bf16", pre_k=min(8, E))
    x = torch.randn((T, d), generator=g, device="cuda").to(torch.bfloat16)
    Wg = (d ** -0.5 * torch.randn((d, E), generator=g, device="cuda")).to(torch.bfloat16)
    nc = moe.norm_config(T, d)
    w = torch.ones(d, device="cuda")
    n = moe.block_norm(nc, x, w_pre=w)["n"]
    idx, wt, logits = (v.clone() for v in moe.route(c, n, Wg, want_logits=True))
    assert int(idx.min()) >= 0 and int(idx.max()) < E
    for _ in range(100):
        n2 = moe.block_norm(nc, x, w_pre=w)["n"]
        i2, w2, l2 = moe.route(c, n2, Wg, want_logits=True)
        assert torch.equal(l2, logits) and torch.equal(i2, idx) and torch.equal(w2, wt)
