"""Refusals of the 8-bit products, the router's losses and dropout: status codes found on the
host, before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from mixture_experts_routed_gb300 import _lib as L
from mixture_experts_routed_gb300 import build as B

V = ctypes.c_void_p
ODD = V((1 << 20) + 2)  # 2-byte aligned only
BIG = 1 << 40
INVALID, UNSUPPORTED, SMALL = (L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED,
                               L.MOE_ERR_WORKSPACE_TOO_SMALL)
NAN, INF = float("nan"), float("inf")


def at(i):
    """Address i, 2^34 bytes from the others, never read: every call here is refused first."""
    return V((i + 1) << 34)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def make(cls, base, kw):
    base = dict(base, **kw)
    return cls(*[base[n] for n, _ in cls._fields_])


def fp8(**kw):
    return make(L.MoeFp8Config, dict(R=8, K=128, N=192, E=2, dtype=1, out_dtype=1, silu=0,
                                     x_rows=0), kw)


def order(names, base, kw):
    base.update(kw)
    return [base[n] for n in names]


def rows(lib, c, **kw):
    names = "cols x src weight act z offsets q scale cq cscale ws n".split()
    a = dict(zip(names, [128, at(0), None, None, 0, None, at(1), at(2), at(3), at(4), at(5), at(6),
                         BIG]))
    return lib.moe_fp8_quantize_rows(ctypes.byref(c), *order(names, a, kw), None)


def weights(lib, c, **kw):
    names = "W q scale".split()
    a = dict(zip(names, [at(0), at(1), at(2)]))
    return lib.moe_fp8_quantize_weights(ctypes.byref(c), *order(names, a, kw), None)


def product(lib, c, **kw):
    names = "transposed q scale wq wsc offsets out ws n".split()
    a = dict(zip(names, [0, *[at(i) for i in range(7)], BIG]))
    return lib.moe_fp8_product(ctypes.byref(c), *order(names, a, kw), None)


def grad(lib, c, **kw):
    names = "x xs dy dys offsets dW ws n".split()
    a = dict(zip(names, [*[at(i) for i in range(7)], BIG]))
    return lib.moe_fp8_weight_grad(ctypes.byref(c), *order(names, a, kw), None)


def back_weights(lib, c, **kw):
    names = "wq wsc W".split()
    return lib.moe_fp8_dequantize_weights(
        ctypes.byref(c), *order(names, dict(zip(names, [at(0), at(1), at(2)])), kw), None)


def back_rows(lib, c, **kw):
    names = "cols q scale x".split()
    return lib.moe_fp8_dequantize_rows(
        ctypes.byref(c), *order(names, dict(zip(names, [128, at(0), at(1), at(2)])), kw), None)


FP8_CALLS = (rows, weights, product, grad, back_weights, back_rows)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), INVALID), (dict(K=0), INVALID), (dict(K=96), INVALID), (dict(N=0), INVALID),
    (dict(N=100), INVALID), (dict(E=0), INVALID), (dict(E=257), INVALID), (dict(dtype=2), INVALID),
    (dict(out_dtype=-1), INVALID), (dict(silu=2), INVALID), (dict(x_rows=-1), INVALID),
    (dict(K=65600), UNSUPPORTED), (dict(N=65600), UNSUPPORTED), (dict(R=(1 << 24) + 1), UNSUPPORTED)])
def test_fp8_configs(lib, kw, status):
    c = fp8(**kw)
    for call in FP8_CALLS:
        assert call(lib, c) == status
    r = ctypes.byref(c)
    assert lib.moe_fp8_workspace_size(r) == lib.moe_fp8_weight_scale_size(r) == 0
    assert lib.moe_fp8_column_rows(r) == lib.moe_fp8_row_scale_size(r, 128) == 0


@pytest.mark.parametrize("call,kw", [
    (rows, dict(cols=64)), (rows, dict(x=None)), (rows, dict(x=ODD)), (rows, dict(act=-1)),
    (rows, dict(act=3)), (rows, dict(act=2)), (rows, dict(act=2, z=ODD)), (rows, dict(z=at(7))),
    (rows, dict(offsets=None)), (rows, dict(q=None)), (rows, dict(scale=None)),
    (rows, dict(q=ODD)), (rows, dict(scale=ODD)), (rows, dict(cq=None)), (rows, dict(cq=ODD)),
    (rows, dict(cscale=ODD)), (rows, dict(q=None, scale=None, cq=None, cscale=None)),
    (rows, dict(ws=None)), (rows, dict(ws=ODD)), (rows, dict(q=at(0))), (rows, dict(cq=at(2))),
    (rows, dict(weight=at(3))), (rows, dict(weight=ODD)), (rows, dict(src=ODD)),
    (rows, dict(offsets=ODD)), (product, dict(offsets=ODD)), (grad, dict(offsets=ODD)),
    (weights, dict(W=None)), (weights, dict(W=ODD)), (weights, dict(q=None)),
    (weights, dict(q=ODD)), (weights, dict(scale=None)), (weights, dict(q=at(0))),
    (product, dict(transposed=2)), (product, dict(q=None)), (product, dict(q=ODD)),
    (product, dict(scale=None)), (product, dict(scale=ODD)), (product, dict(wq=None)),
    (product, dict(wq=ODD)), (product, dict(wsc=None)), (product, dict(offsets=None)),
    (product, dict(out=None)), (product, dict(out=ODD)), (product, dict(out=at(0))),
    (product, dict(ws=None)), (product, dict(ws=ODD)),
    (grad, dict(x=None)), (grad, dict(x=ODD)), (grad, dict(xs=None)), (grad, dict(xs=ODD)),
    (grad, dict(dy=None)), (grad, dict(dys=ODD)), (grad, dict(offsets=None)),
    (grad, dict(dW=None)), (grad, dict(dW=ODD)), (grad, dict(dW=at(2))), (grad, dict(ws=None)),
    (back_weights, dict(W=None)), (back_weights, dict(wq=ODD)), (back_weights, dict(W=at(0))),
    (back_rows, dict(cols=64)), (back_rows, dict(q=None)), (back_rows, dict(x=ODD)),
    (back_rows, dict(x=at(0)))])
def test_fp8_arguments(lib, call, kw):
    assert call(lib, fp8(), **kw) == INVALID


def test_fp8_the_gradients_have_no_activation(lib):
    assert product(lib, fp8(silu=1), transposed=1) == UNSUPPORTED


def test_fp8_sizes(lib):
    c = fp8(R=300, K=1408, N=640, E=5)
    r = ctypes.byref(c)
    assert lib.moe_fp8_row_scale_size(r, 1408) == 300 * 12
    assert lib.moe_fp8_row_scale_size(r, 640) == 300 * 8
    assert lib.moe_fp8_row_scale_size(r, 128) == 0
    assert lib.moe_fp8_column_rows(r) == 128 * (2 + 5)
    assert lib.moe_fp8_weight_scale_size(r) == 5 * 11 * 5
    need = lib.moe_fp8_workspace_size(r)
    assert need > 0 and need % 256 == 0
    for call in (rows, product, grad):
        assert call(lib, fp8(), n=need - 1) == SMALL


# ---------------------------------------------------------------- the router's losses
def loss_cfg(**kw):
    return make(L.MoeRouterLossConfig, dict(T=64, E=8, k=2, S=1, balance=0.01, z=0.0), kw)


def loss(lib, c, **kw):
    names = "logits idx offsets mask loss counts tokens lse ws n".split()
    a = dict(zip(names, [at(0), at(1), at(2), None, at(3), at(4), at(5), at(6), at(7), BIG]))
    return lib.moe_router_loss(ctypes.byref(c), *order(names, a, kw), None)


def loss_back(lib, c, **kw):
    names = "logits offsets mask counts tokens lse dloss out".split()
    a = dict(zip(names, [at(0), at(1), None, at(2), at(3), at(4), None, at(5)]))
    return lib.moe_router_loss_backward(ctypes.byref(c), *order(names, a, kw), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(E=257), INVALID), (dict(k=0), INVALID),
    (dict(k=9), INVALID), (dict(E=32, k=17), INVALID), (dict(S=0), INVALID),
    (dict(balance=NAN), INVALID), (dict(balance=INF), INVALID), (dict(z=-INF), INVALID),
    (dict(T=(1 << 26) + 1), UNSUPPORTED), (dict(S=(1 << 20) + 1), UNSUPPORTED)])
def test_loss_configs(lib, kw, status):
    c = loss_cfg(**kw)
    assert loss(lib, c) == status and loss_back(lib, c) == status
    assert lib.moe_router_loss_workspace_size(ctypes.byref(c)) == 0


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(logits=ODD), dict(idx=None), dict(idx=ODD), dict(offsets=ODD),
    dict(loss=None), dict(loss=ODD), dict(counts=None), dict(counts=ODD), dict(tokens=None),
    dict(tokens=ODD), dict(lse=None), dict(lse=ODD), dict(ws=None), dict(ws=ODD),
    dict(loss=at(0)), dict(counts=at(3)), dict(lse=at(7))])
def test_loss_arguments(lib, kw):
    assert loss(lib, loss_cfg(), **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(logits=ODD), dict(offsets=ODD), dict(counts=None), dict(counts=ODD),
    dict(tokens=None), dict(tokens=ODD), dict(lse=None), dict(lse=ODD), dict(dloss=ODD),
    dict(out=None), dict(out=ODD), dict(out=at(0)), dict(out=at(4))])
def test_loss_backward_arguments(lib, kw):
    assert loss_back(lib, loss_cfg(), **kw) == INVALID


def test_loss_of_sequences_needs_their_offsets(lib):
    assert loss(lib, loss_cfg(S=2), offsets=None) == INVALID
    assert loss_back(lib, loss_cfg(S=2), offsets=None) == INVALID


def test_loss_workspace(lib):
    need = lib.moe_router_loss_workspace_size(ctypes.byref(loss_cfg()))
    assert need > 0 and need % 256 == 0
    assert loss(lib, loss_cfg(), n=need - 1) == SMALL


def test_backward_with_dlogits_needs_them(lib):
    from test_abi_host import cfg
    c = cfg(T=8)
    a = [at(i) for i in range(20)]
    for dlogits in (None, ODD):
        st = lib.moe_backward_with_dlogits(ctypes.byref(c), *a[:3], None, *a[3:6], BIG, a[6],
                                           dlogits, *a[7:13], BIG, None)
        assert st == INVALID


# ---------------------------------------------------------------- dropout
def drop_cfg(**kw):
    return make(L.MoeDropoutConfig, dict(T=8, d=128, dtype=1, site=0, p=0.1), kw)


def drop(lib, c, x=at(0), residual=at(1), state=at(2), out=at(3)):
    return lib.moe_dropout(ctypes.byref(c), x, residual, state, out, None)


def drop_back(lib, c, dout=at(0), state=at(2), dx=at(3)):
    return lib.moe_dropout_backward(ctypes.byref(c), dout, state, dx, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(d=0), INVALID), (dict(d=96), INVALID), (dict(dtype=2), INVALID),
    (dict(site=-1), INVALID), (dict(p=-0.1), INVALID), (dict(p=1.0), INVALID), (dict(p=NAN), INVALID),
    (dict(d=65600), UNSUPPORTED), (dict(T=(1 << 24) + 1), UNSUPPORTED)])
def test_dropout_configs(lib, kw, status):
    assert drop(lib, drop_cfg(**kw)) == status and drop_back(lib, drop_cfg(**kw)) == status


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=ODD), dict(residual=ODD), dict(state=None), dict(state=ODD),
    dict(out=None), dict(out=ODD), dict(out=V((1 << 34) + 16)), dict(out=V((2 << 34) - 16)),
    dict(state=V((4 << 34) + 8))])
def test_dropout_arguments(lib, kw):
    assert drop(lib, drop_cfg(), **kw) == INVALID


def test_dropout_backward_arguments(lib):
    for kw in (dict(dout=None), dict(dout=ODD), dict(state=None), dict(dx=None), dict(dx=ODD),
               dict(dx=V((1 << 34) + 16))):
        assert drop_back(lib, drop_cfg(), **kw) == INVALID


def test_null_configs(lib):
    assert lib.moe_fp8_product(None, 0, *[at(0)] * 7, BIG, None) == INVALID
    assert lib.moe_router_loss(None, *[at(0)] * 9, BIG, None) == INVALID
    assert lib.moe_dropout(None, *[at(0)] * 4, None) == INVALID


@pytest.mark.parametrize("tag,cls", [("moe_fp8_config", L.MoeFp8Config),
                                     ("moe_router_loss_config", L.MoeRouterLossConfig),
                                     ("moe_dropout_config", L.MoeDropoutConfig)])
def test_configs_match_the_header(tag, cls):
    from test_abi_host import struct_fields
    ctypes_of = {"int32_t": ctypes.c_int32, "float": ctypes.c_float}
    assert [(n, ctypes_of[t]) for n, t in struct_fields(tag)] == list(cls._fields_)


# ---------------------------------------------------------------- the binding
def test_binding_refuses_wrong_shapes_types_and_forms():
    import torch
    import mixture_experts_routed_gb300 as moe
    B.build()
    u8, bf, i32 = torch.uint8, torch.bfloat16, torch.int32
    c = moe.fp8_config(4, 128, 192, 2)
    ws, off = torch.zeros(1 << 16, dtype=u8), torch.zeros(3, dtype=i32)

    def refused(f, match="not"):
        with pytest.raises(moe.MoEError, match=match):
            f()

    refused(lambda: moe.fp8_quantize_weights(c, torch.zeros((2, 192, 128), dtype=bf)))
    refused(lambda: moe.fp8_quantize_weights(c, torch.zeros((2, 128, 192))))
    refused(lambda: moe.fp8_quantize_rows(c, torch.zeros((4, 64), dtype=bf), off, ws=ws))
    refused(lambda: moe.fp8_quantize_rows(c, torch.zeros((5, 128), dtype=bf), off, ws=ws))
    refused(lambda: moe.fp8_quantize_rows(c, torch.zeros((4, 128), dtype=bf), off, ws=ws,
                                          act="relu"), "act")
    refused(lambda: moe.fp8_quantize_rows(c, torch.zeros((4, 128), dtype=bf), off, ws=ws,
                                          rows=False), "neither")
    r = moe.Fp8Rows(4, 128, True, False, 0, "cpu")
    wq, wsc = torch.zeros((2, 128, 192), dtype=u8), torch.zeros((2, 1, 2), dtype=u8)
    refused(lambda: moe.fp8_product(c, r, wq, wsc, off, ws=ws, transposed=True))
    refused(lambda: moe.fp8_product(c, r, wq, wsc[:, :, :1], off, ws=ws))
    refused(lambda: moe.fp8_weight_grad(c, r, r, off, ws=ws), "form")
    refused(lambda: moe.fp8_product(c, moe.Fp8Rows(4, 128, False, True, 2, "cpu"), wq, wsc, off,
                                    ws=ws), "form")
    refused(lambda: moe.fp8_product(c, r, wq, wsc, off, ws=ws), "GPU memory")
    refused(lambda: moe.fp8_dequantize_rows(moe.fp8_config(5, 128, 192, 2), r))
    c = moe.router_loss_config(4, 8, 2)
    idx = torch.zeros((4, 2), dtype=i32)
    refused(lambda: moe.router_loss(c, torch.zeros((4, 8), dtype=bf), idx, ws=ws))
    refused(lambda: moe.router_loss(c, torch.zeros((4, 8)), idx.long(), ws=ws))
    kept = moe.RouterLoss(torch.zeros(3), torch.zeros((2, 8), dtype=i32),
                          torch.zeros(4, dtype=i32), torch.zeros(4))
    refused(lambda: moe.router_loss_backward(c, torch.zeros((4, 8)), kept))
    c = moe.dropout_config(4, 64)
    x = torch.zeros((4, 64), dtype=bf)
    refused(lambda: moe.dropout(c, x.float(), torch.zeros(2, dtype=torch.int64)))
    refused(lambda: moe.dropout(c, x, torch.zeros(2, dtype=i32)))
    refused(lambda: moe.dropout(c, x, torch.zeros(2, dtype=torch.int64)), "GPU memory")
