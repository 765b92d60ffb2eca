"""Rows whose src is out of range are rows of zeros, whatever their routing weight is."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from train_plain import decode
from test_gpu_u_fp8 import DT, columns_of, gen, offsets_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", [None, "silu", "silu_grad"])
@pytest.mark.parametrize("weight", [float("inf"), -float("inf"), float("nan"), -3.0])
def test_a_bad_source_and_its_weight(cuda_ok, dtype, act, weight):
    C, counts, T = 320, [40, 0, 131], 30
    R = sum(counts)
    g = gen(6)
    x = torch.randn((T + 1, C), generator=g, device="cuda").to(DT[dtype])
    x[T] = 0  # what a bad source stands for
    src = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((R,), generator=g, device="cuda") + 0.5
    z = torch.randn((R, C), generator=g, device="cuda").to(DT[dtype]) if act == "silu_grad" else None
    off, bad = offsets_of(counts), [0, 39, 40, 127, 170]
    good = src.clone()
    good[bad] = T
    c = moe.fp8_config(R, C, 64, 3, dtype, x_rows=T + 1)
    ws = moe.alloc_fp8_workspace(c)
    want = moe.fp8_quantize_rows(c, x, off, ws=ws, src=good, row_weight=w, act=act, z=z,
                                 columns=True)
    assert moe.get_device_error(ws) == moe.MOE_OK
    c = moe.fp8_config(R, C, 64, 3, dtype, x_rows=T)
    src[bad] = torch.tensor([T, -1, 1 << 30, -(1 << 31), T], dtype=torch.int32, device="cuda")
    w[bad] = weight
    tiles = 3
    for rows, columns in ((True, False), (False, True), (True, True)):
        r = moe.fp8_quantize_rows(c, x[:T], off, ws=ws, src=src, row_weight=w, act=act, z=z,
                                  rows=rows, columns=columns)
        assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX
        if rows:
            assert not bool((r.q[bad] & 0x7f).any())
            assert torch.equal(r.scale[:, :3], want.scale[:, :3])
            assert torch.equal(decode(r.q, r.scale[:, :3].contiguous(), 1, 128),
                               decode(want.q, want.scale[:, :3].contiguous(), 1, 128))
        if columns:
            s, t = columns_of(r.cscale, C)[:tiles], columns_of(want.cscale, C)[:tiles]
            assert torch.equal(s, t)
            n = tiles * 128
            assert torch.equal(decode(r.cq[:n], s, 128, 1), decode(want.cq[:n], t, 128, 1))
