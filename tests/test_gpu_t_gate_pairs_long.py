"""The tensor-core gate on pairs of blocks, often enough for a race that shows once in 1500 calls:
thousands of calls back to back behind another kernel, compared on the device, with one
synchronisation at the end."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,E,k", [(8192, 7168, 16, 2), (4097, 7168, 16, 2), (8192, 2048, 64, 2),
                                     (9600, 4096, 8, 2)])
def test_split_gate_repeats(cuda_ok, T, d, E, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(T + d + E)
    c = moe.make_config(T, d, E, k, 1024, "bf16", pre_k=min(8, E))
    x = torch.randn((T, d), generator=g, device="cuda").to(torch.bfloat16)
    Wg = (d ** -0.5 * torch.randn((d, E), generator=g, device="cuda")).to(torch.bfloat16)
    nc, w = moe.norm_config(T, d), torch.ones(d, device="cuda")
    n = moe.block_norm(nc, x, w_pre=w)["n"]
    first = [v.clone() for v in moe.route(c, n, Wg, want_logits=True)]
    assert int(first[0].min()) >= 0 and int(first[0].max()) < E
    idx, wt, logits = (torch.empty_like(v) for v in first)
    n2, moved = torch.empty_like(n), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(4000):
        moe.block_norm(nc, x, w_pre=w, n=n2)
        moe.route(c, n2, Wg, topk_idx=idx, topk_w=wt, logits=logits)
        moved += (logits != first[2]).any() | (idx != first[0]).any() | (wt != first[1]).any()
    assert int(moved) == 0
