"""Microscaled 4-bit rows, weights and products on the GPU. Quantisation is a function of the
input bits and is compared exactly with nearest-grid-value rounding in 64 bits. A product's
terms are exact in fp32 and it adds K of them, at worst one rounding each; the tensor cores add
64 at a time and split sums are joined, so K / 8 + 64 half steps of the absolute terms cover
it, plus half a step of the output's type."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import (F64, U32, half_step, mx4_quantize, mx4_values, scales_of_tiles,
                         unpack_codes)

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def spread(shape, dtype, seed):
    """Normal values times powers of two from 2^-20 to 2^20 per 64 columns, with zeros, exact
    ties and a block of zeros."""
    g = gen(seed)
    v = torch.randn(shape, generator=g, device="cuda")
    p = torch.randint(-20, 21, (*shape[:-1], shape[-1] // 64), generator=g, device="cuda")
    v = torch.ldexp(v, p.repeat_interleave(64, -1))
    v[..., ::7] = 0
    ties = torch.tensor([4, 0.25, -0.75, 1.25, -1.75, 2.5, 3.5, -5, 7.9], device="cuda")
    v[..., 0, :9] = ties
    v[..., 0, 9:32] = 0
    v[..., -1, -32:] = 0
    return v.to(dtype)


def offsets_of(counts):
    return torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


def row_tiles(counts):
    """(tile row of each routed row, number of tiles)"""
    at, tiles = [], 0
    for n in counts:
        at += [tiles * 128 + i for i in range(n)]
        tiles += -(-n // 128)
    return torch.tensor(at, dtype=torch.long, device="cuda"), tiles


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [64, 128, 192, 256, 320, 1408])
@pytest.mark.parametrize("counts", [[1], [5, 0, 130], [0, 0, 128, 129, 1, 0]])
def test_rows(cuda_ok, dtype, K, counts):
    R, E = sum(counts), len(counts)
    x = spread((R, K), DT[dtype], K + R)
    c = moe.mx4_config(R, K, 64, E, dtype)
    off = offsets_of(counts)
    q, s = moe.mx4_quantize_rows(c, x, off, ws=moe.alloc_mx4_workspace(c))
    code, sc = mx4_quantize(x.to(F64))
    at, tiles = row_tiles(counts)
    assert torch.equal(unpack_codes(q).long(), code)
    assert torch.equal(scales_of_tiles(s, tiles, K)[at], sc)
    back = moe.mx4_dequantize_rows(c, q, s, off)
    assert torch.equal(back.to(F64), mx4_values(code, sc))


def test_gathered_rows_and_a_bad_source(cuda_ok):
    K, counts = 320, [40, 3, 0, 100]
    R, T = sum(counts), 30
    x = spread((T, K), torch.bfloat16, 1)
    src = torch.randint(0, T, (R,), generator=gen(2), device="cuda", dtype=torch.int32)
    c = moe.mx4_config(R, K, 64, 4, x_rows=T)
    ws, off = moe.alloc_mx4_workspace(c), offsets_of(counts)
    q, s = moe.mx4_quantize_rows(c, x, off, src=src, ws=ws)
    want = mx4_values(*mx4_quantize(x[src.long()].to(F64)))
    assert torch.equal(moe.mx4_dequantize_rows(c, q, s, off).to(F64), want)
    assert moe.get_device_error(ws) == moe.MOE_OK
    src[7], src[41] = T, -1
    q, s = moe.mx4_quantize_rows(c, x, off, src=src, ws=ws)
    want[[7, 41]] = 0
    assert torch.equal(moe.mx4_dequantize_rows(c, q, s, off).to(F64), want)
    assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_ends_of_the_range(cuda_ok, dtype):
    # subnormals, the largest numbers, infinities and NaN: a block with one of the last two is
    # NaN, its neighbours are not touched
    dt = DT[dtype]
    x = torch.zeros((8, 128), dtype=dt, device="cuda")
    big, tiny = torch.finfo(dt).max, torch.finfo(dt).smallest_normal
    x[0, :4] = torch.tensor([big, -big, big / 3, 1.0], device="cuda").to(dt)
    x[1, :4] = torch.tensor([tiny, -tiny / 2, tiny / 8, tiny / 64], device="cuda").to(dt)
    x[2, 40] = float("inf")
    x[3, 40] = -float("inf")
    x[4, 40] = float("nan")
    x[5] = -0.0
    x[6, :2] = torch.tensor([4 * tiny, 3.9 * tiny], device="cuda").to(dt)
    x[:, 96:] = torch.randn((8, 32), generator=gen(3), device="cuda").to(dt)
    c = moe.mx4_config(8, 128, 64, 1, dtype)
    off = offsets_of([8])
    q, s = moe.mx4_quantize_rows(c, x, off, ws=moe.alloc_mx4_workspace(c))
    code, sc = mx4_quantize(x.to(F64))
    assert torch.equal(scales_of_tiles(s, 1, 128)[:8], sc)
    fine = (sc != 255).repeat_interleave(32, 1)
    assert torch.equal(unpack_codes(q).long()[fine], code[fine])
    back = moe.mx4_dequantize_rows(c, q, s, off)
    assert bool(back[~fine].isnan().all())
    assert torch.equal(back[fine].to(F64), mx4_values(code, sc)[fine])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,K,N", [(1, 64, 64), (3, 320, 192), (2, 1408, 128), (5, 256, 448)])
def test_weights(cuda_ok, dtype, E, K, N):
    W = spread((E, N, K), DT[dtype], E + K).transpose(1, 2).contiguous()
    c = moe.mx4_config(1, K, N, E, dtype)
    q, s = moe.mx4_quantize_weights(c, W)
    want = torch.empty((E, K, N), dtype=F64, device="cuda")
    nt = -(-N // 128)
    per = nt * -(-K // 128) * 512
    for e in range(E):
        code, sc = mx4_quantize(W[e].t().to(F64))
        assert torch.equal(unpack_codes(q[e]).long(), code)
        assert torch.equal(scales_of_tiles(s[e * per:(e + 1) * per], nt, K)[:N], sc)
        want[e] = mx4_values(code, sc).t()
    assert torch.equal(moe.mx4_dequantize_weights(c, q, s).to(F64), want)


def product(counts, K, N, out_dtype="f32", silu=0, seed=0, wipe=True):
    R, E = sum(counts), len(counts)
    g = gen(seed)
    x = torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn((E, K, N), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
    # rows, columns and blocks of other sizes, so that a scale in the wrong place shows
    x *= torch.exp2(torch.randint(-6, 7, (R, 1), generator=g, device="cuda").float())
    x.view(R, -1, 32).mul_(torch.exp2(
        torch.randint(-3, 4, (R, K // 32, 1), generator=g, device="cuda").float()))
    W *= torch.exp2(torch.randint(-4, 5, (E, 1, N), generator=g, device="cuda").float())
    W.view(E, -1, 32, N).mul_(torch.exp2(
        torch.randint(-3, 4, (E, K // 32, 1, N), generator=g, device="cuda").float()))
    c = moe.mx4_config(R, K, N, E, out_dtype=out_dtype, silu=silu)
    ws, off = moe.alloc_mx4_workspace(c), offsets_of(counts)
    wq, wsc = moe.mx4_quantize_weights(c, W)
    # scale bytes that no row owns are never seen: NaN there
    n = moe._lib.load().moe_mx4_row_scale_size(moe.api.ctypes.byref(c))
    sc = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    q, sc = moe.mx4_quantize_rows(c, x, off, ws=ws, scale=sc)
    out = torch.full((R, N), float("nan"), dtype=DT[out_dtype], device="cuda")
    moe.mx4_product(c, q, sc, wq, wsc, off, ws=ws, out=out)
    torch.cuda.synchronize()
    assert moe.get_device_error(ws) == moe.MOE_OK
    a = moe.mx4_dequantize_rows(c, q, sc, off).to(F64)
    lo = 0
    for e, n in enumerate(counts):
        if n:
            w = moe.mx4_dequantize_weights(c, wq, wsc)[e].to(F64)
            y, ya = a[lo:lo + n] @ w, a[lo:lo + n].abs() @ w.abs()
            tol = (K / 8 + 64) * U32 * ya
            if silu:  # |SiLU'| < 1.1; __expf and the division: 8 half steps of fp32
                y, tol = y * torch.sigmoid(y), 1.1 * tol + 8 * U32 * (y.abs() + y * y)
            got = out[lo:lo + n].to(F64)
            over = (got - y).abs() - (half_step(DT[out_dtype]) * (y.abs() + tol) + tol)
            assert bool((over <= 0).all()), (e, float(over.max()))
            lo += n
    return c, q, sc, wq, wsc, off, ws, out


# one row; segments of one row, a tile, a tile and one row, none; short and odd contractions
# and widths; few rows everywhere (split over the contraction) and many
@pytest.mark.parametrize("counts", [[1], [1, 0, 1], [32, 3], [33, 3], [0, 128, 129, 1, 0],
                                    [300, 0, 20]])
@pytest.mark.parametrize("K,N", [(64, 64), (128, 128), (192, 320), (256, 256), (1408, 448),
                                 (2048, 1472)])
def test_products(cuda_ok, counts, K, N):
    product(counts, K, N, seed=K + N + len(counts))


# many rows per expert: pairs of blocks, 256 rows a tile; the second block's rows none, one,
# some or all
@pytest.mark.parametrize("counts", [[128], [257], [513, 0], [300, 129, 1, 600], [1500, 0, 2, 40]])
@pytest.mark.parametrize("K,N", [(64, 64), (192, 128), (256, 320), (1408, 192), (2048, 1472)])
def test_pairs(cuda_ok, counts, K, N):
    product(counts, K, N, seed=K + N + len(counts))


@pytest.mark.parametrize("counts", [[2, 1], [200, 100], [400, 130]])
@pytest.mark.parametrize("silu", [0, 1])
def test_bf16_and_silu(cuda_ok, counts, silu):
    product(counts, 512, 384, "bf16", silu, seed=silu)


def test_many_experts_and_more_tiles_than_blocks(cuda_ok):
    product([i % 5 for i in range(256)], 256, 320, seed=1)
    product([i * 9 % 140 for i in range(64)], 320, 1408, "bf16", seed=2)
    product([i * 97 % 700 for i in range(32)], 320, 1408, "bf16", seed=3)


def test_long_contraction(cuda_ok):
    product([1, 1], 4096, 1408, seed=5)
    product([140], 7168, 576, seed=6)
    product([300], 7168, 320, seed=7)


def test_nan_blocks_reach_their_rows_and_columns_only(cuda_ok):
    for counts in ([3, 2], [100, 60], [300, 290]):
        c, q, sc, wq, wsc, off, ws, out = product(counts, 256, 192, seed=7)
        x = moe.mx4_dequantize_rows(c, q, sc, off)
        x[1, 70] = float("nan")
        W = moe.mx4_dequantize_weights(c, wq, wsc)
        W[1, 5, 9] = float("inf")
        q, sc = moe.mx4_quantize_rows(c, x, off, ws=ws)
        wq, wsc = moe.mx4_quantize_weights(c, W)
        got = moe.mx4_product(c, q, sc, wq, wsc, off, ws=ws)
        bad = torch.zeros_like(got, dtype=torch.bool)
        bad[1] = True
        bad[counts[0]:, 9] = True
        assert torch.equal(got.isnan(), bad)
        assert torch.equal(got[~bad], out[~bad])


def test_same_bits_again_and_in_a_graph(cuda_ok):
    for counts in ([2, 0, 1], [150, 3, 99], [700, 300, 90]):
        c, q, sc, wq, wsc, off, ws, out = product(counts, 2048, 320, seed=8)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                again = moe.mx4_product(c, q, sc, wq, wsc, off, ws=ws)
            for _ in range(10):
                again.zero_()
                graph.replay()
                s.synchronize()
                assert torch.equal(again, out)


@pytest.mark.parametrize("off", [[0, 5, 4, 8], [0, 2, 3, 9], [-1, 2, 3, 8]])
def test_bad_offsets_are_flagged_and_nothing_is_written(cuda_ok, off):
    c = moe.mx4_config(8, 128, 64, 3)
    ws = moe.alloc_mx4_workspace(c)
    off = torch.tensor(off, dtype=torch.int32, device="cuda")
    x = torch.ones((8, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.full((8, 64), 7, dtype=torch.uint8, device="cuda")
    _, sc = moe.mx4_quantize_rows(c, x, off, ws=ws, q=q)
    assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX
    assert bool((q == 7).all())
    wq, wsc = moe.mx4_quantize_weights(c, torch.ones((3, 128, 64), dtype=torch.bfloat16,
                                                     device="cuda"))
    out = torch.full((8, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.mx4_product(c, q, sc, wq, wsc, off, ws=ws, out=out)
    assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX
    assert bool((out == 3).all())


def test_rows_outside_the_segments_are_not_written(cuda_ok):
    c = moe.mx4_config(8, 128, 64, 2, out_dtype="f32")
    ws = moe.alloc_mx4_workspace(c)
    off = torch.tensor([2, 4, 7], dtype=torch.int32, device="cuda")
    x = torch.ones((8, 128), dtype=torch.bfloat16, device="cuda")
    q, sc = moe.mx4_quantize_rows(c, x, off, ws=ws)
    wq, wsc = moe.mx4_quantize_weights(c, torch.ones((2, 128, 64), dtype=torch.bfloat16,
                                                     device="cuda"))
    out = torch.full((8, 64), 3.0, device="cuda")
    moe.mx4_product(c, q, sc, wq, wsc, off, ws=ws, out=out)
    assert bool((out[2:7] == 128).all()) and bool((out[:2] == 3).all()) and bool((out[7] == 3).all())
    assert moe.get_device_error(ws) == moe.MOE_OK


def test_no_rows(cuda_ok):
    c = moe.mx4_config(0, 128, 64, 2)
    ws = moe.alloc_mx4_workspace(c)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    q, sc = moe.mx4_quantize_rows(c, torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"),
                                  off, ws=ws)
    wq, wsc = moe.mx4_quantize_weights(c, torch.ones((2, 128, 64), dtype=torch.bfloat16,
                                                     device="cuda"))
    assert moe.mx4_product(c, q, sc, wq, wsc, off, ws=ws).shape == (0, 64)


def test_an_output_aligned_to_16_bytes_only(cuda_ok):
    for counts in ([3], [200], [300, 300]):
        for dt in ("f32", "bf16"):
            c, q, sc, wq, wsc, off, ws, out = product(counts, 256, 192, dt, seed=9)
            buf = torch.zeros(out.numel() + 64, dtype=out.dtype, device="cuda")
            view = buf[16 // out.element_size():][:out.numel()].view(out.shape)
            assert view.data_ptr() % 32 == 16
            moe.mx4_product(c, q, sc, wq, wsc, off, ws=ws, out=view)
            assert torch.equal(view, out)
            assert not bool(buf[:16 // out.element_size()].any())
