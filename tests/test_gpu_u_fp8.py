"""8-bit rows, columns, weights and their products on the GPU. Quantisation without an
activation is a function of the input bits and is compared exactly. A product's terms are exact
in fp32 and it adds C of them; the tensor cores add 32 at a time and split sums are joined, so C /
8 + 64 half steps of the absolute terms cover it, plus half a step of the output's type."""
import pytest
import torch

import mixture_experts_routed_gb300 as moe
from block_plain import U32, half_step
from train_plain import F64, decode, fp8_scales, fp8_values, spread

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U8 = torch.uint8


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def mixed(shape, dtype, seed):
    """Normal values times powers of two from 2^-20 to 2^20 per 64 columns and per row, with
    zeros, ties and blocks of zeros."""
    g = gen(seed)
    v = torch.randn(shape, generator=g, device="cuda")
    p = torch.randint(-20, 21, (*shape[:-1], shape[-1] // 64), generator=g, device="cuda")
    v = torch.ldexp(v, p.repeat_interleave(64, -1))
    v[..., ::7] = 0
    ties = torch.tensor([448, 17, -19, 21, 0.0009765625, -0.0029296875, 464 / 2, -1.0625, 1.1875],
                        device="cuda")
    v[..., 0, :9] = ties
    v[..., 0, 9:64] = 0
    v[..., -1, :] = 0
    return v.to(dtype)


def offsets_of(counts, first=0):
    return torch.tensor([first] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


def column_form(v, counts):
    """(values [tiles * 128, C], scales [tiles, C]) of the columns' form."""
    values, scales, lo = [], [], 0
    for n in counts:
        if n:
            a, s = fp8_values(v[lo:lo + n], 128, 1)
            pad = torch.zeros((-n % 128, v.shape[1]), dtype=F64, device=v.device)
            nan = s[-1:].expand(len(pad), -1) == 255
            values.append(torch.cat([a, torch.where(nan, float("nan"), pad)]))
            scales.append(s)
        lo += n
    return torch.cat(values), torch.cat(scales)


def columns_of(cscale, C):
    """The scales [tile, C] of a columns' form, in the columns' order."""
    n = len(cscale)
    return cscale.view(n, -1, 32, 4).transpose(2, 3).reshape(n, -1)[:, :C].contiguous()


def same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


def check_rows(r, v, counts):
    C = v.shape[1]
    if r.q is not None:
        want, s = fp8_values(v, 1, 128)
        sc = r.scale[:, :s.shape[1]]
        assert torch.equal(sc, s)
        assert same(decode(r.q, sc, 1, 128), want)
    if r.cq is not None:
        want, s = column_form(v, counts)
        n = len(s)
        got = columns_of(r.cscale, C)[:n]
        assert torch.equal(got, s)
        assert same(decode(r.cq[:n * 128], got, 128, 1), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 128, 192, 1408])
@pytest.mark.parametrize("counts", [[1], [5, 0, 130], [0, 0, 128, 129, 1, 0]])
def test_rows_and_columns(cuda_ok, dtype, C, counts):
    R, E = sum(counts), len(counts)
    x = mixed((R, C), DT[dtype], C + R)
    c = moe.fp8_config(R, C, 64, E, dtype)
    off, ws = offsets_of(counts), moe.alloc_fp8_workspace(c)
    both = moe.fp8_quantize_rows(c, x, off, ws=ws, columns=True)
    check_rows(both, x.to(F64), counts)
    rows = moe.fp8_quantize_rows(c, x, off, ws=ws)
    cols = moe.fp8_quantize_rows(c, x, off, ws=ws, rows=False, columns=True)
    assert rows.cq is None and cols.q is None
    check_rows(rows, x.to(F64), counts)
    check_rows(cols, x.to(F64), counts)
    back = moe.fp8_dequantize_rows(c, rows)
    assert torch.equal(back.to(F64), fp8_values(x.to(F64), 1, 128)[0])
    assert moe.get_device_error(ws) == moe.MOE_OK


def test_rows_of_the_outputs_side(cuda_ok):
    # N columns, the product's K another
    c = moe.fp8_config(40, 64, 320, 1)
    x = mixed((40, 320), torch.bfloat16, 3)
    r = moe.fp8_quantize_rows(c, x, offsets_of([40]), ws=moe.alloc_fp8_workspace(c), columns=True)
    check_rows(r, x.to(F64), [40])
    assert torch.equal(moe.fp8_dequantize_rows(c, r).to(F64), fp8_values(x.to(F64), 1, 128)[0])


def test_gathered_and_weighted_rows_and_a_bad_source(cuda_ok):
    C, counts = 320, [40, 3, 0, 100]
    R, T = sum(counts), 30
    x = mixed((T, C), torch.bfloat16, 1)
    src = torch.randint(0, T, (R,), generator=gen(2), device="cuda", dtype=torch.int32)
    w = torch.rand((R,), generator=gen(3), device="cuda")
    c = moe.fp8_config(R, C, 64, 4, x_rows=T)
    ws, off = moe.alloc_fp8_workspace(c), offsets_of(counts)
    v = (x[src.long()].float() * w[:, None]).to(F64)
    check_rows(moe.fp8_quantize_rows(c, x, off, ws=ws, src=src, row_weight=w, columns=True), v,
               counts)
    assert moe.get_device_error(ws) == moe.MOE_OK
    src[7], src[41] = T, -1
    v[[7, 41]] = 0
    check_rows(moe.fp8_quantize_rows(c, x, off, ws=ws, src=src, row_weight=w, columns=True), v,
               counts)
    assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX


def near_codes(q, s, v, rows, cols):
    """v known to 2^-20: each code is one of the nearest, each scale the least that holds it."""
    b = spread(s, rows, cols, v.shape).to(F64) - 127
    got = decode(q, s, rows, cols)
    half = torch.maximum(v.abs(), torch.exp2(b - 6)) * 2.0 ** -4
    assert bool(((got - v).abs() <= half * (1 + 2.0 ** -15) + v.abs() * 2.0 ** -20).all())
    lo = fp8_scales(v * (1 - 2.0 ** -20), rows, cols)
    hi = fp8_scales(v * (1 + 2.0 ** -20), rows, cols)
    assert bool(((s >= lo) & (s <= hi)).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "silu_grad"])
def test_activations(cuda_ok, dtype, act):
    # exp and the quotients: some ten roundings of fp32, below 2^-20
    counts, C = [50, 0, 140], 320
    R = sum(counts)
    g = gen(5)
    z = (torch.randn((R, C), generator=g, device="cuda") * 3).to(DT[dtype])
    z[0, :8] = torch.tensor([0.0, -0.0, 80, -80, 200, -200, 1e-30, -1e-30], device="cuda")
    w = torch.rand((R,), generator=g, device="cuda") + 0.5
    z64 = z.to(F64)
    sg = torch.sigmoid(z64)
    c = moe.fp8_config(R, C, 64, 3, dtype)
    off, ws = offsets_of(counts), moe.alloc_fp8_workspace(c)
    if act == "silu":
        x, zz, v = z, None, z64 * sg
    else:
        x = torch.randn((R, C), generator=g, device="cuda").to(DT[dtype])
        zz, v = z, x.to(F64) * sg * (1 + z64 * (1 - sg))
    # (near SiLU' = 0, at z = -1.28, the difference of two terms of 1/5 is left: its absolute error)
    v = v * w.to(F64)[:, None]
    if act == "silu_grad":
        far = (z64 + 1.2784645).abs() > 0.25
        x = torch.where(far, x, torch.zeros_like(x))
        v = torch.where(far, v, torch.zeros_like(v))
    r = moe.fp8_quantize_rows(c, x, off, ws=ws, row_weight=w, columns=True, act=act, z=zz)
    near_codes(r.q, r.scale[:, :3].contiguous(), v, 1, 128)
    lo, tile, cs = 0, 0, columns_of(r.cscale, C)
    for n in counts:
        tiles = -(-n // 128)
        if n:
            near_codes(r.cq[tile * 128:tile * 128 + n], cs[tile:tile + tiles], v[lo:lo + n],
                       128, 1)
        lo, tile = lo + n, tile + tiles
    assert moe.get_device_error(ws) == moe.MOE_OK


def test_limits_of_the_activations(cuda_ok):
    inf, nan = float("inf"), float("nan")
    z = torch.zeros((4, 128), device="cuda")
    z[0, 0], z[1, 0], z[2, 0], z[3, 0] = inf, -inf, 300.0, nan
    c = moe.fp8_config(4, 128, 64, 1, "f32")
    off, ws = offsets_of([4]), moe.alloc_fp8_workspace(c)
    r = moe.fp8_quantize_rows(c, torch.ones_like(z), off, ws=ws, act="silu_grad", z=z)
    v = decode(r.q, r.scale[:, :1].contiguous(), 1, 128)
    assert v[0, 0] == 1 and v[1, 0] == 0 and v[2, 0] == 1 and bool(v[3].isnan().all())
    assert bool((v[:3, 1:] == 0.5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_ends_of_the_range(cuda_ok, dtype):
    # subnormals, the largest numbers, infinities and NaN: a block with one of the last two is
    # NaN, its neighbours are not touched
    dt = DT[dtype]
    x = torch.zeros((9, 256), dtype=dt, device="cuda")
    big, tiny = torch.finfo(dt).max, torch.finfo(dt).smallest_normal
    x[0, :4] = torch.tensor([big, -big, big / 3, 1.0], device="cuda").to(dt)
    x[1, :4] = torch.tensor([tiny, -tiny / 2, tiny / 8, tiny / 64], device="cuda").to(dt)
    x[2, 40] = float("inf")
    x[3, 41] = -float("inf")
    x[4, 42] = float("nan")
    x[5] = -0.0
    x[6, :2] = torch.tensor([448 * tiny, 450 * tiny], device="cuda").to(dt)
    x[:, 128:] = torch.randn((9, 128), generator=gen(3), device="cuda").to(dt)
    c = moe.fp8_config(9, 256, 64, 1, dtype)
    r = moe.fp8_quantize_rows(c, x, offsets_of([9]), ws=moe.alloc_fp8_workspace(c), columns=True)
    check_rows(r, x.to(F64), [9])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,K,N", [(1, 64, 64), (3, 320, 192), (2, 1408, 128), (5, 256, 448)])
def test_weights(cuda_ok, dtype, E, K, N):
    W = mixed((E, K, N), DT[dtype], E + K)
    W[0, 0, 0] = 3e38  # a block of its own size
    c = moe.fp8_config(1, K, N, E, dtype)
    q, s = moe.fp8_quantize_weights(c, W)
    back = moe.fp8_dequantize_weights(c, q, s)
    for e in range(E):
        want, sc = fp8_values(W[e].to(F64), 128, 128)
        assert torch.equal(s[e], sc)
        assert torch.equal(decode(q[e], s[e], 128, 128), want)
        assert torch.equal(back[e].to(F64), want.to(DT[dtype]).to(F64))


def test_weights_with_an_infinity(cuda_ok):
    W = torch.ones((2, 256, 192), device="cuda")
    W[1, 130, 5] = float("inf")
    c = moe.fp8_config(1, 256, 192, 2, "f32")
    q, s = moe.fp8_quantize_weights(c, W)
    bad = torch.zeros_like(W, dtype=torch.bool)
    bad[1, 128:, :128] = True
    back = moe.fp8_dequantize_weights(c, q, s)
    assert torch.equal(back.isnan(), bad) and bool((back[~bad] == 1).all())


# ---------------------------------------------------------------- products
def problem(counts, K, N, out_dtype="f32", silu=0, seed=0, first=0, behind=0):
    R, E = first + sum(counts) + behind, len(counts)
    g = gen(seed)

    def draw(*shape):
        """Rows and 128-blocks of other sizes, so that a scale in the wrong place shows."""
        v = torch.randn(shape, generator=g, device="cuda")
        v *= torch.exp2(torch.randint(-6, 7, (*shape[:-1], 1), generator=g, device="cuda").float())
        p = torch.randint(-3, 4, (*shape[:-2], -(-shape[-2] // 128), -(-shape[-1] // 128)),
                          generator=g, device="cuda").float()
        p = p.repeat_interleave(128, -2).repeat_interleave(128, -1)
        return (v * torch.exp2(p)[..., :shape[-2], :shape[-1]]).to(torch.bfloat16)

    x, dy = draw(R, K), draw(R, N)
    W = draw(E, K, N) * K ** -0.5
    c = moe.fp8_config(R, K, N, E, out_dtype=out_dtype, silu=silu)
    ws, off = moe.alloc_fp8_workspace(c), offsets_of(counts, first)
    wq, wsc = moe.fp8_quantize_weights(c, W)
    xr = moe.fp8_quantize_rows(c, x, off, ws=ws, columns=True)
    dr = moe.fp8_quantize_rows(c, dy, off, ws=ws, columns=True)
    return dict(c=c, ws=ws, off=off, wq=wq, wsc=wsc, x=xr, dy=dr, counts=counts, first=first)


def within(got, y, terms, length, dtype, silu=False):
    tol = (length / 8 + 64) * U32 * terms
    if silu:  # |SiLU'| < 1.1; exp and the quotient: 8 half steps of fp32
        y, tol = y * torch.sigmoid(y), 1.1 * tol + 8 * U32 * (y.abs() + y * y)
    over = (got.to(F64) - y).abs() - (half_step(dtype) * (y.abs() + tol) + tol)
    assert bool((over <= 0).all()), float(over.max())


def check_products(p, transposed, out):
    c, lo = p["c"], p["first"]
    r = p["dy"] if transposed else p["x"]
    dt = out.dtype
    a = decode(r.q, r.scale[:, :-(-r.q.shape[1] // 128)].contiguous(), 1, 128)
    assert bool(out[:lo].isnan().all())
    for e, n in enumerate(p["counts"]):
        if n:
            w = decode(p["wq"][e], p["wsc"][e], 128, 128)
            w = w.t() if transposed else w
            within(out[lo:lo + n], a[lo:lo + n] @ w, a[lo:lo + n].abs() @ w.abs(), w.shape[0], dt,
                   c.silu and not transposed)
            lo += n
    assert bool(out[lo:].isnan().all())


def run_product(p, transposed):
    c = p["c"]
    dt = torch.float32 if c.out_dtype == moe._lib.MOE_DTYPE_F32 else torch.bfloat16
    out = torch.full((c.R, c.K if transposed else c.N), float("nan"), dtype=dt, device="cuda")
    moe.fp8_product(c, p["dy"] if transposed else p["x"], p["wq"], p["wsc"], p["off"], ws=p["ws"],
                    transposed=transposed, out=out)
    torch.cuda.synchronize()
    assert moe.get_device_error(p["ws"]) == moe.MOE_OK
    return out


def check_grad(p, dW):
    c, tile = p["c"], 0
    xs, ds = columns_of(p["x"].cscale, c.K), columns_of(p["dy"].cscale, c.N)
    for e, n in enumerate(p["counts"]):
        tiles = -(-n // 128)
        if not n:
            assert not bool(dW[e].any())
            continue
        t = slice(tile * 128, (tile + tiles) * 128)
        a = decode(p["x"].cq[t], xs[tile:tile + tiles], 128, 1)
        b = decode(p["dy"].cq[t], ds[tile:tile + tiles], 128, 1)
        within(dW[e], a.t() @ b, a.abs().t() @ b.abs(), n, torch.float32)
        tile += tiles


def run_grad(p):
    c = p["c"]
    dW = torch.full((c.E, c.K, c.N), float("nan"), device="cuda")
    moe.fp8_weight_grad(c, p["x"], p["dy"], p["off"], ws=p["ws"], out=dW)
    torch.cuda.synchronize()
    assert moe.get_device_error(p["ws"]) == moe.MOE_OK
    return dW


SIZES = [(64, 64), (128, 128), (192, 320), (256, 256), (1408, 448), (2048, 1472)]


# one row; segments of one row, a tile, a tile and one row, none; few rows everywhere and many
@pytest.mark.parametrize("counts", [[1], [1, 0, 1], [32, 3], [33, 3], [0, 128, 129, 1, 0],
                                    [300, 0, 20], [513, 0], [300, 129, 1, 600], [1500, 0, 2, 40]])
@pytest.mark.parametrize("K,N", SIZES)
def test_products(cuda_ok, counts, K, N):
    p = problem(counts, K, N, seed=K + N + len(counts))
    check_products(p, False, run_product(p, False))
    check_products(p, True, run_product(p, True))
    check_grad(p, run_grad(p))


@pytest.mark.parametrize("counts", [[2, 1], [200, 100], [400, 130]])
@pytest.mark.parametrize("silu", [0, 1])
def test_bf16_and_silu(cuda_ok, counts, silu):
    p = problem(counts, 512, 384, "bf16", silu, seed=silu)
    check_products(p, False, run_product(p, False))
    if not silu:
        check_products(p, True, run_product(p, True))
    p = problem(counts, 512, 384, "f32", silu, seed=silu)
    check_products(p, False, run_product(p, False))


def test_many_experts_and_more_tiles_than_blocks(cuda_ok):
    for counts, K, N, dt in (([i % 5 for i in range(256)], 256, 320, "f32"),
                             ([i * 9 % 140 for i in range(64)], 320, 1408, "bf16"),
                             ([i * 97 % 700 for i in range(32)], 1408, 320, "bf16")):
        p = problem(counts, K, N, dt, seed=len(counts))
        check_products(p, False, run_product(p, False))
        check_products(p, True, run_product(p, True))
        check_grad(p, run_grad(p))


def test_long_contractions(cuda_ok):
    for counts, K, N in (([1, 1], 4096, 1408), ([140], 7168, 576), ([300], 576, 7168),
                         ([9000], 192, 320), ([3, 5000, 0, 700], 320, 576)):
        p = problem(counts, K, N, seed=K)
        check_products(p, False, run_product(p, False))
        check_products(p, True, run_product(p, True))
        check_grad(p, run_grad(p))


def test_the_largest_contractions_and_widths(cuda_ok):
    for counts, K, N in (([3], 65536, 64), ([130, 2], 65536, 64), ([500], 64, 65536),
                         ([1, 2], 64, 65536)):
        p = problem(counts, K, N, "bf16", seed=K)
        check_products(p, False, run_product(p, False))
        check_products(p, True, run_product(p, True))
        check_grad(p, run_grad(p))


# Long sums keep fp32's precision: an accumulator that drops what is below its
# last place loses half a step on average with each of its additions, four to 128
# steps of the contraction, so the norm of the error has to stay below that of a
# chain of 2048 steps, 64 additions (Y and dX: 4096, 128).
@pytest.mark.parametrize("counts,K,N", [([16384], 256, 320), ([20000, 0, 5, 2049], 192, 256)])
def test_precision_of_long_weight_gradients(cuda_ok, counts, K, N):
    p = problem(counts, K, N, seed=K)
    dW, tile = run_grad(p), 0
    check_grad(p, dW)
    xs, ds = columns_of(p["x"].cscale, K), columns_of(p["dy"].cscale, N)
    for e, n in enumerate(counts):
        t = slice(tile, tile + -(-n // 128))
        a, b = (decode(r.cq[t.start * 128:t.stop * 128], s[t], 128, 1)
                for r, s in ((p["x"], xs), (p["dy"], ds)))
        y = a.t() @ b
        assert float((dW[e].to(F64) - y).norm()) <= 64 * U32 * float(y.norm())
        tile = t.stop


# One tile cut among all blocks; as many tiles as blocks almost, so that a block's part
# is long; few and many rows
@pytest.mark.parametrize("counts,K,N", [([3], 65536, 64), ([2], 16384, 25600), ([300, 1], 16640, 320),
                                        ([1000], 16384, 256)])
@pytest.mark.parametrize("silu", [0, 1])
def test_precision_of_long_products(cuda_ok, counts, K, N, silu):
    p = problem(counts, K, N, silu=silu, seed=K)
    out = run_product(p, False)
    check_products(p, False, out)
    if not silu:
        a, lo = decode(p["x"].q, p["x"].scale[:, :K // 128].contiguous(), 1, 128), 0
        for e, n in enumerate(counts):
            y = a[lo:lo + n] @ decode(p["wq"][e], p["wsc"][e], 128, 128)
            assert float((out[lo:lo + n].to(F64) - y).norm()) <= 128 * U32 * float(y.norm())
            lo += n


@pytest.mark.parametrize("counts", [[2, 0, 3], [150, 40, 300]])
def test_rows_of_no_segment(cuda_ok, counts):
    # before the first and behind the last: not quantised, not written, no part of any sum
    p = problem(counts, 256, 192, first=5, behind=9)
    check_products(p, False, run_product(p, False))
    check_products(p, True, run_product(p, True))
    check_grad(p, run_grad(p))


def test_quantising_leaves_rows_of_no_segment(cuda_ok):
    c = moe.fp8_config(8, 128, 64, 2)
    ws = moe.alloc_fp8_workspace(c)
    q = torch.full((8, 128), 7, dtype=U8, device="cuda")
    s = torch.full((8, 4), 9, dtype=U8, device="cuda")
    x = torch.ones((8, 128), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([2, 4, 7], dtype=torch.int32, device="cuda")
    st = moe._lib.load().moe_fp8_quantize_rows(
        moe.api.ctypes.byref(c), 128, x.data_ptr(), None, None, 0, None, off.data_ptr(),
        q.data_ptr(), s.data_ptr(), None, None, ws.data_ptr(), ws.nbytes,
        torch.cuda.current_stream().cuda_stream)
    assert st == moe.MOE_OK
    assert bool((q[:2] == 7).all()) and bool((q[7:] == 7).all()) and not bool((q[2:7] == 7).any())
    assert s[:, 0].tolist() == [9, 9, 119, 119, 119, 119, 119, 9]


def test_what_lies_behind_the_tiles_is_not_read(cuda_ok):
    # code tensors are sized for the worst case; NaN codes and scales in the rest
    p = problem([100, 0, 30], 256, 192)
    clean = run_grad(p)
    for r in (p["x"], p["dy"]):
        r.cq[256:] = 0x7f
        r.cscale[2:] = 255
        r.scale[:, 2:] = 255
    assert torch.equal(run_grad(p), clean)
    check_products(p, False, run_product(p, False))
    check_products(p, True, run_product(p, True))


def test_nan_blocks_reach_their_rows_and_columns_only(cuda_ok):
    for counts in ([3, 2], [100, 60], [300, 290]):
        p = problem(counts, 256, 320, seed=7)
        c, R = p["c"], sum(counts)
        y, dx, dW = run_product(p, False), run_product(p, True), run_grad(p)
        p["x"].scale[1, 0] = 255          # row 1, k below 128
        p["dy"].scale[0, 2] = 255         # row 0, n of 256 and more
        p["wsc"][1, 1, 0] = 255           # expert 1, k of 128 and more, n below 128
        p["x"].cscale[0, 1, 4 * 9] = 255  # expert 0, k = 128 + 9
        y2, dx2, dW2 = run_product(p, False), run_product(p, True), run_grad(p)
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[1] = True
        bad[counts[0]:, :128] = True
        assert torch.equal(y2.isnan(), bad) and torch.equal(y2[~bad], y[~bad])
        bad = torch.zeros_like(dx, dtype=torch.bool)
        bad[0] = True
        bad[counts[0]:, 128:] = True
        assert torch.equal(dx2.isnan(), bad) and torch.equal(dx2[~bad], dx[~bad])
        bad = torch.zeros_like(dW, dtype=torch.bool)
        bad[0, 137] = True
        assert torch.equal(dW2.isnan(), bad) and torch.equal(dW2[~bad], dW[~bad])


def test_same_bits_again_and_in_a_graph(cuda_ok):
    for counts in ([2, 0, 1], [150, 3, 99], [700, 300, 90]):
        p = problem(counts, 2048, 320, seed=8)
        want = run_product(p, False), run_product(p, True), run_grad(p)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            a = (p["c"], p["off"])
            with torch.cuda.graph(graph, stream=s):
                got = (moe.fp8_product(a[0], p["x"], p["wq"], p["wsc"], a[1], ws=p["ws"]),
                       moe.fp8_product(a[0], p["dy"], p["wq"], p["wsc"], a[1], ws=p["ws"],
                                       transposed=True),
                       moe.fp8_weight_grad(a[0], p["x"], p["dy"], a[1], ws=p["ws"]))
            for _ in range(10):
                for t in got:
                    t.zero_()
                graph.replay()
                s.synchronize()
                for t, w in zip(got, want):
                    assert torch.equal(t, w)


def test_two_streams_at_once(cuda_ok):
    ps = [problem(counts, 1408, 320, seed=9) for counts in ([3, 0, 20], [500, 0, 300])]
    want = [(run_product(p, False), run_grad(p)) for p in ps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, p in enumerate(ps):
            with torch.cuda.stream(streams[i]):
                got[i].append((moe.fp8_product(p["c"], p["x"], p["wq"], p["wsc"], p["off"],
                                               ws=p["ws"]),
                               moe.fp8_weight_grad(p["c"], p["x"], p["dy"], p["off"], ws=p["ws"])))
    torch.cuda.synchronize()
    for i in range(2):
        for y, dW in got[i]:
            assert torch.equal(y, want[i][0].nan_to_num()) and torch.equal(dW, want[i][1])


@pytest.mark.parametrize("off", [[0, 5, 4, 8], [0, 2, 3, 9], [-1, 2, 3, 8]])
def test_bad_offsets_are_flagged_and_nothing_is_written(cuda_ok, off):
    p = problem([3, 2, 3], 128, 64)
    c, ws = p["c"], p["ws"]
    off = torch.tensor(off, dtype=torch.int32, device="cuda")
    x = torch.ones((8, 128), dtype=torch.bfloat16, device="cuda")
    moe.fp8_quantize_rows(c, x, off, ws=ws)
    assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX
    out = torch.full((8, 64), 3.0, dtype=torch.float32, device="cuda")
    moe.fp8_product(c, p["x"], p["wq"], p["wsc"], off, ws=ws, out=out)
    assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX and bool((out == 3).all())
    dW = torch.full((3, 128, 64), 3.0, device="cuda")
    moe.fp8_weight_grad(c, p["x"], p["dy"], off, ws=ws, out=dW)
    assert moe.get_device_error(ws) == moe.MOE_ERR_BAD_INDEX and bool((dW == 3).all())
    # the workspace is as good as before
    check_products(p, False, run_product(p, False))


def test_no_rows(cuda_ok):
    c = moe.fp8_config(0, 128, 64, 2)
    ws = moe.alloc_fp8_workspace(c)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    r = moe.fp8_quantize_rows(c, x, off, ws=ws, columns=True)
    d = moe.fp8_quantize_rows(c, x[:, :64].contiguous(), off, ws=ws, columns=True)
    wq, wsc = moe.fp8_quantize_weights(c, torch.ones((2, 128, 64), dtype=torch.bfloat16,
                                                     device="cuda"))
    assert moe.fp8_product(c, r, wq, wsc, off, ws=ws).shape == (0, 64)
    assert moe.fp8_dequantize_rows(c, r).shape == (0, 128)
    assert not bool(moe.fp8_weight_grad(c, r, d, off, ws=ws).any())
    # rows that no expert has
    c = moe.fp8_config(5, 128, 64, 2)
    r = moe.fp8_quantize_rows(c, torch.ones((5, 128), dtype=torch.bfloat16, device="cuda"), off,
                              ws=ws, columns=True)
    d = moe.fp8_quantize_rows(c, torch.ones((5, 64), dtype=torch.bfloat16, device="cuda"), off,
                              ws=ws, columns=True)
    dW = torch.full((2, 128, 64), 3.0, device="cuda")
    assert not bool(moe.fp8_weight_grad(c, r, d, off, ws=ws, out=dW).any())


def test_an_output_aligned_to_16_bytes_only(cuda_ok):
    for counts in ([3], [200], [300, 300]):
        for dt in ("f32", "bf16"):
            p = problem(counts, 256, 192, dt, seed=9)
            out = run_product(p, False)
            buf = torch.zeros(out.numel() + 64, dtype=out.dtype, device="cuda")
            view = buf[16 // out.element_size():][:out.numel()].view(out.shape)
            assert view.data_ptr() % 32 == 16
            moe.fp8_product(p["c"], p["x"], p["wq"], p["wsc"], p["off"], ws=p["ws"], out=view)
            assert torch.equal(view, out)
            assert not bool(buf[:16 // out.element_size()].any())
        dW = run_grad(p)
        buf = torch.zeros(dW.numel() + 64, device="cuda")
        view = buf[4:][:dW.numel()].view(dW.shape)
        moe.fp8_weight_grad(p["c"], p["x"], p["dy"], p["off"], ws=p["ws"], out=view)
        assert torch.equal(view, dW) and not bool(buf[:4].any())
