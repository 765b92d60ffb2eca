"""The plain 4-bit rounding the GPU tests compare with, against the format's own statements."""
import torch

from block_plain import F64, GRID, mx4_quantize, mx4_values, scales_of_tiles, unpack_codes


def test_values_on_the_grid_are_kept_and_ties_go_to_the_even_code():
    v = torch.zeros((1, 32), dtype=F64)
    v[0, :8], v[0, 8:16] = GRID, -GRID
    code, s = mx4_quantize(v)
    assert s.item() == 127 and torch.equal(mx4_values(code, s), v)
    v = torch.zeros((1, 32), dtype=F64)
    v[0, :8] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5], dtype=F64)
    v[0, 8] = 7.99
    code, s = mx4_quantize(v)
    assert code[0, :9].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 7] and s.item() == 127


def test_scales():
    v = torch.zeros((7, 32), dtype=F64)
    for r, a in enumerate([0.0, 1.0, 3.99, 4.0, 2.0 ** -133, float("inf"), float("nan")]):
        v[r, 3] = a
    assert mx4_quantize(v)[1][:, 0].tolist() == [127, 125, 126, 127, 0, 255, 255]


def test_each_value_is_a_nearest_one():
    v = torch.randn((50, 64), dtype=F64, generator=torch.Generator().manual_seed(0)) * 3
    code, s = mx4_quantize(v)
    step = torch.exp2(s.to(F64) - 127).repeat_interleave(32, 1)
    inside = v.abs() <= 6 * step
    err = (mx4_values(code, s) - v).abs() / step
    grid = torch.cat([GRID, -GRID])
    best = ((v / step)[..., None] - grid).abs().amin(-1)
    assert torch.allclose(err[inside], best[inside], rtol=0, atol=1e-12)
    assert bool((mx4_values(code, s)[~inside].abs() == 6 * step[~inside]).all())


def test_layout_helpers():
    q = torch.tensor([[0x21, 0x43]], dtype=torch.uint8)
    assert unpack_codes(q).tolist() == [[1, 2, 3, 4]]
    K, tiles = 192, 2
    scale = torch.zeros(tiles * 2 * 512, dtype=torch.uint8)
    t, i, b = 1, 77, 5
    scale[(t * 2 + b // 4) * 512 + (i % 32) * 16 + (i // 32) * 4 + b % 4] = 9
    got = scales_of_tiles(scale, tiles, K)
    assert got.shape == (256, 6) and got[128 + 77, 5] == 9 and int((got != 0).sum()) == 1
