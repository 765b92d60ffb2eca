"""The plain forms the GPU tests of 8-bit products, router losses and dropout compare with."""
import math

import pytest
import torch

from train_plain import (F64, decode, dropout_keep, e4m3, fp8_scales, fp8_values, philox,
                         router_loss, router_loss_gradient)


def test_e4m3_is_torchs_on_a_grid():
    v = torch.cat([torch.linspace(-448, 448, 20001, dtype=F64),
                   torch.linspace(-0.05, 0.05, 20001, dtype=F64)])
    v = v.float().to(F64)  # (torch's cast starts from fp32)
    assert torch.equal(e4m3(v), v.float().to(torch.float8_e4m3fn).to(F64))


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (449.0, 1), (224.0, -1), (1.75, -8),
                                    (1.7500001, -7), (1.0, -8), (2.0 ** -126, -127),
                                    (3.4e38, 120), (2.0 ** -149, -127)])
def test_scales_by_hand(amax, e):
    v = torch.zeros((1, 128), dtype=F64)
    v[0, 77] = -amax
    assert int(fp8_scales(v, 1, 128)) == e + 127


def test_scales_of_zeros_and_of_what_is_not_finite():
    v = torch.zeros((3, 256), dtype=F64)
    v[1, 130] = math.inf
    v[2, 5] = math.nan
    s = fp8_scales(v, 1, 128)
    assert s.tolist() == [[127, 127], [127, 255], [255, 127]]


def test_values_are_near_and_the_codes_fill_the_range():
    g = torch.Generator().manual_seed(1)
    v = torch.randn((256, 320), generator=g, dtype=F64)
    for rows, cols in ((1, 128), (128, 1), (128, 128)):
        got, s = fp8_values(v, rows, cols)
        scale = torch.exp2(s.to(F64) - 127).repeat_interleave(rows, 0).repeat_interleave(cols, 1)
        scale = scale[:256, :320]
        # half a step: 2^-4 of the value, or of the least normal value
        assert bool(((got - v).abs() <= torch.maximum(v.abs(), scale * 2.0 ** -6) * 2.0 ** -4).all())
        assert bool(((got / scale).abs() <= 448).all())
        q = (got / scale).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(decode(q, s, rows, cols), got)


def test_router_loss_by_hand():
    # two experts, two tokens that choose expert 0, p = (3/4, 1/4) and (1/2, 1/2)
    L = torch.tensor([[math.log(3), 0.0], [0.0, 0.0]], dtype=F64)
    idx = torch.zeros((2, 1), dtype=torch.int64)
    loss, counts = router_loss(L, idx, 1, [0, 2], None, 0.5, 0.25)
    assert counts.tolist() == [[2, 0]]
    bal, z = 2 * (0.75 + 0.5) / 2, (math.log(4) ** 2 + math.log(2) ** 2) / 2
    assert torch.allclose(loss, torch.tensor([0.5 * bal + 0.25 * z, bal, z], dtype=F64))


def test_even_load_gives_one():
    g = torch.Generator().manual_seed(2)
    L = torch.randn((64, 8), generator=g, dtype=F64)
    idx = (torch.arange(128) % 8).view(64, 2)
    assert abs(float(router_loss(L, idx, 2, [0, 64], None, 1, 0)[0][1]) - 1) < 1e-12


@pytest.mark.parametrize("offs,masked", [([0, 9], False), ([0, 3, 3, 8], True), ([1, 2, 9], False)])
def test_router_gradient_against_differences_and_differentiation(offs, masked):
    g = torch.Generator().manual_seed(3)
    L = torch.randn((9, 5), generator=g, dtype=F64)
    idx = torch.topk(L, 2).indices
    mask = torch.tensor([1, 0, 1, 1, 1, 0, 1, 1, 1]) if masked else None
    want = router_loss_gradient(L, idx, 2, offs, mask, 0.7, 0.3)
    leaf = L.clone().requires_grad_(True)
    auto, = torch.autograd.grad(router_loss(leaf, idx, 2, offs, mask, 0.7, 0.3)[0][0], [leaf])
    assert torch.allclose(want, auto, atol=1e-14)
    h = 1e-5
    for t in range(9):
        for e in range(5):
            d = torch.zeros_like(L)
            d[t, e] = h
            up, dn = (router_loss(L + s * d, idx, 2, offs, mask, 0.7, 0.3)[0][0] for s in (1, -1))
            assert abs(float((up - dn) / (2 * h) - want[t, e])) < 1e-9


def test_philox_known_answers():
    # the generator's published vectors
    assert philox([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    f = 0xffffffff
    assert philox([f] * 4, [f] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert philox([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0]) == \
        [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def test_share_kept():
    keep, scale = dropout_keep(0, 40000, 0, 123, 4, 0.25)
    # 40000 draws of 3/4: five standard deviations are 433
    assert abs(int(keep.sum()) - 30000) < 433 and scale == 4 / 3
    assert bool(dropout_keep(0, 64, 0, 1, 1, 0.0)[0].all())
    other = dropout_keep(0, 40000, 1, 123, 4, 0.25)[0]
    assert abs(int((other & keep).sum()) - 22500) < 5 * 100
