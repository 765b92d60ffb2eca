"""Refusals of the operators around the expert layer: status codes found on the host, before
any CUDA call (no GPU needed)."""
import ctypes

import pytest

from mixture_experts_routed_gb300 import _lib as L
from mixture_experts_routed_gb300 import build as B

P = ctypes.c_void_p(4096)    # aligned, never read: every call here is refused first
ODD = ctypes.c_void_p(4100)  # 4-byte aligned only


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def norm(**kw):
    base = dict(T=8, d=128, dtype=1, gate=0, eps=1e-6, alpha=1.0, beta=1.0)
    base.update(kw)
    return L.MoeNormConfig(*[base[n] for n, _ in L.MoeNormConfig._fields_])


def norm_forward(lib, c, x=P, b=P, w_post=P, gate=None, w_pre=P, out=P, n=P):
    return lib.moe_block_norm(ctypes.byref(c), x, b, w_post, gate, w_pre, out, n, None, None, None)


def norm_backward(lib, c, dout=P, dn=P, x=P, b=P, w_post=P, gate=None, w_pre=P, rb=P, ro=P, dx=P,
                  db=P, dw_post=P, dgate=None, dw_pre=P, ws=P, ws_bytes=1 << 40):
    return lib.moe_block_norm_backward(ctypes.byref(c), dout, dn, x, b, w_post, gate, w_pre, rb, ro,
                                       dx, db, dw_post, dgate, dw_pre, ws, ws_bytes, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), L.MOE_ERR_INVALID_ARG), (dict(d=0), L.MOE_ERR_INVALID_ARG),
    (dict(d=96), L.MOE_ERR_INVALID_ARG), (dict(dtype=2), L.MOE_ERR_INVALID_ARG),
    (dict(gate=-1), L.MOE_ERR_INVALID_ARG), (dict(gate=4), L.MOE_ERR_INVALID_ARG),
    (dict(eps=0.0), L.MOE_ERR_INVALID_ARG), (dict(eps=NAN), L.MOE_ERR_INVALID_ARG),
    (dict(eps=INF), L.MOE_ERR_INVALID_ARG), (dict(alpha=NAN), L.MOE_ERR_INVALID_ARG),
    (dict(alpha=INF), L.MOE_ERR_INVALID_ARG), (dict(beta=-INF), L.MOE_ERR_INVALID_ARG),
    (dict(d=65600), L.MOE_ERR_UNSUPPORTED)])
def test_norm_configs(lib, kw, status):
    c = norm(**kw)
    assert norm_forward(lib, c) == status
    assert norm_backward(lib, c) == status
    assert lib.moe_block_norm_backward_workspace_size(ctypes.byref(c)) == 0


def test_norm_null_config(lib):
    assert lib.moe_block_norm(None, *[P] * 9, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_block_norm_backward_workspace_size(None) == 0


@pytest.mark.parametrize("gate,kw", [
    (0, dict(x=None)), (0, dict(x=ODD)), (0, dict(b=ODD)), (0, dict(w_post=None)),
    (0, dict(w_post=ODD)), (0, dict(b=None)), (0, dict(w_pre=ODD)), (0, dict(out=None)),
    (0, dict(out=ODD)), (0, dict(n=None)), (0, dict(n=ODD)), (0, dict(w_pre=None)),
    (0, dict(b=None, w_post=None)), (0, dict(b=None, w_post=None, out=None, w_pre=None, n=None)),
    (1, dict()), (2, dict()), (2, dict(gate=ODD)), (3, dict(gate=ODD)),
    (1, dict(gate=ctypes.c_void_p(4098)))])
def test_norm_forward_arguments(lib, gate, kw):
    assert norm_forward(lib, norm(gate=gate), **kw) == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("gate,kw", [
    (0, dict(dout=None)), (0, dict(dout=ODD)), (0, dict(dn=None)), (0, dict(dn=ODD)),
    (0, dict(x=None)), (0, dict(x=ODD)), (0, dict(b=None)), (0, dict(b=ODD)),
    (0, dict(w_post=None)), (0, dict(w_pre=None)), (0, dict(rb=None)), (0, dict(ro=None)),
    (0, dict(dx=None)), (0, dict(dx=ODD)), (0, dict(db=None)), (0, dict(db=ODD)),
    (0, dict(dw_post=None)), (0, dict(dw_pre=None)), (0, dict(dw_pre=ODD)), (0, dict(dgate=P)),
    (1, dict(gate=P)), (2, dict(gate=P, dgate=ODD)), (3, dict(dgate=P)), (0, dict(ws=None)),
    (0, dict(ws=ctypes.c_void_p(4096 + 128))),
    (0, dict(b=None, w_post=None, db=None, dw_post=None, w_pre=None, dn=None, dw_pre=None))])
def test_norm_backward_arguments(lib, gate, kw):
    assert norm_backward(lib, norm(gate=gate), **kw) == L.MOE_ERR_INVALID_ARG


def test_norm_backward_of_no_rows_still_checks_what_it_reads(lib):
    for kw in (dict(w_post=None), dict(gate=None, dgate=P), dict(gate=ODD, dgate=P),
               dict(gate=P, dgate=None), dict(dw_pre=None)):
        full = dict(gate=P, dgate=P)
        full.update(kw)
        assert norm_backward(lib, norm(T=0, gate=2), **full) == L.MOE_ERR_INVALID_ARG


def test_norm_backward_workspace(lib):
    c = norm()
    need = lib.moe_block_norm_backward_workspace_size(ctypes.byref(c))
    assert need > 0 and need % 256 == 0
    assert norm_backward(lib, c, ws_bytes=need - 1) == L.MOE_ERR_WORKSPACE_TOO_SMALL


def test_norm_config_matches_the_header():
    from test_abi_host import struct_fields
    fields = struct_fields("moe_norm_config")
    ctypes_of = {"int32_t": ctypes.c_int32, "float": ctypes.c_float}
    assert [(n, ctypes_of[t]) for n, t in fields] == list(L.MoeNormConfig._fields_)


def test_norm_binding_refuses_wrong_shapes_and_types():
    import torch
    import mixture_experts_routed_gb300 as moe
    B.build()
    c = moe.norm_config(4, 64, "bf16")
    w = torch.ones(64)
    for x in (torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros((4, 64))):
        with pytest.raises(moe.MoEError, match="not"):
            moe.block_norm(c, x, w_pre=w)
    with pytest.raises(moe.MoEError, match="not contiguous"):
        moe.block_norm(c, torch.zeros((64, 4), dtype=torch.bfloat16).t(), w_pre=w)


def moe_cfg(**kw):
    from test_abi_host import cfg
    return cfg(**{"T": 8, **kw})


def few(lib, c, x=P, Wg=P, noise=None, W1=P, W2=P, out=P, ws=P, ws_bytes=1 << 40):
    return lib.moe_forward_few(ctypes.byref(c), x, Wg, None, noise, W1, W2, out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), L.MOE_ERR_INVALID_ARG), (dict(d=100), L.MOE_ERR_INVALID_ARG),
    (dict(k=9), L.MOE_ERR_INVALID_ARG), (dict(T=33), L.MOE_ERR_UNSUPPORTED),
    (dict(dtype=0), L.MOE_ERR_UNSUPPORTED), (dict(payload_fp8=1), L.MOE_ERR_UNSUPPORTED),
    (dict(output_fp8=1), L.MOE_ERR_UNSUPPORTED), (dict(keep_z=1), L.MOE_ERR_UNSUPPORTED)])
def test_few_configs(lib, kw, status):
    c = moe_cfg(**kw)
    assert few(lib, c) == status
    assert lib.moe_forward_few_workspace_size(ctypes.byref(c)) == 0


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=ODD), dict(Wg=None), dict(W1=None), dict(W1=ODD), dict(W2=None),
    dict(W2=ODD), dict(out=None), dict(out=ODD), dict(ws=None),
    dict(ws=ctypes.c_void_p(4096 + 128))])
def test_few_arguments(lib, kw):
    assert few(lib, moe_cfg(), **kw) == L.MOE_ERR_INVALID_ARG


def test_few_soft_gating_wants_its_samples(lib):
    assert few(lib, moe_cfg(router=3, E=8, k=8, tau=1.0)) == L.MOE_ERR_INVALID_ARG


def test_few_workspace(lib):
    assert L.MOE_FEW_MAX_TOKENS == 32
    for kw in (dict(T=1), dict(T=32, E=256, k=8, d=7168, f=2048), dict(T=0)):
        c = moe_cfg(**kw)
        need = lib.moe_forward_few_workspace_size(ctypes.byref(c))
        assert need > 0 and need % 256 == 0
        assert few(lib, c, ws_bytes=need - 1) == L.MOE_ERR_WORKSPACE_TOO_SMALL


def mx4(**kw):
    base = dict(R=8, K=128, N=64, E=2, dtype=1, out_dtype=1, silu=0, x_rows=8)
    base.update(kw)
    return L.MoeMx4Config(*[base[n] for n, _ in L.MoeMx4Config._fields_])


def mx4_calls(lib, c, bad=None, ws_bytes=1 << 40):
    """The five calls, each argument that `bad` = (call, position, value) names replaced."""
    r = ctypes.byref(c)
    calls = {"quantize_weights": [r, P, P, P, None],
             "quantize_rows": [r, P, None, P, P, P, P, ws_bytes, None],
             "product": [r, P, P, P, P, P, P, P, ws_bytes, None],
             "dequantize_weights": [r, P, P, P, None],
             "dequantize_rows": [r, P, P, P, P, None]}
    if bad is None:
        return [getattr(lib, "moe_mx4_" + n)(*a) for n, a in calls.items()]
    calls[bad[0]][bad[1]] = bad[2]
    return getattr(lib, "moe_mx4_" + bad[0])(*calls[bad[0]])


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), L.MOE_ERR_INVALID_ARG), (dict(K=0), L.MOE_ERR_INVALID_ARG),
    (dict(K=96), L.MOE_ERR_INVALID_ARG), (dict(N=32), L.MOE_ERR_INVALID_ARG),
    (dict(N=0), L.MOE_ERR_INVALID_ARG), (dict(E=0), L.MOE_ERR_INVALID_ARG),
    (dict(E=257), L.MOE_ERR_INVALID_ARG), (dict(dtype=2), L.MOE_ERR_INVALID_ARG),
    (dict(out_dtype=-1), L.MOE_ERR_INVALID_ARG), (dict(silu=2), L.MOE_ERR_INVALID_ARG),
    (dict(x_rows=-1), L.MOE_ERR_INVALID_ARG), (dict(K=65600), L.MOE_ERR_UNSUPPORTED),
    (dict(N=65600), L.MOE_ERR_UNSUPPORTED), (dict(R=(1 << 24) + 1), L.MOE_ERR_UNSUPPORTED)])
def test_mx4_configs(lib, kw, status):
    c = mx4(**kw)
    assert set(mx4_calls(lib, c)) == {status}
    for size in ("row_scale_size", "weight_scale_size", "workspace_size"):
        assert getattr(lib, "moe_mx4_" + size)(ctypes.byref(c)) == 0


@pytest.mark.parametrize("call,positions", [
    ("quantize_weights", (1, 2, 3)), ("quantize_rows", (1, 4, 5, 6)),
    ("product", (1, 2, 3, 4, 6, 7)), ("dequantize_weights", (1, 2, 3)),
    ("dequantize_rows", (1, 2, 4))])
def test_mx4_arguments(lib, call, positions):
    for i in positions:
        for v in (None, ODD):
            assert mx4_calls(lib, mx4(), (call, i, v)) == L.MOE_ERR_INVALID_ARG, (i, v)


def test_mx4_null_offsets_and_small_workspaces(lib):
    for call, i in (("quantize_rows", 3), ("product", 5), ("dequantize_rows", 3)):
        assert mx4_calls(lib, mx4(), (call, i, None)) == L.MOE_ERR_INVALID_ARG
    need = lib.moe_mx4_workspace_size(ctypes.byref(mx4()))
    for call, i in (("quantize_rows", 7), ("product", 8)):
        assert mx4_calls(lib, mx4(), (call, i, need - 1)) == L.MOE_ERR_WORKSPACE_TOO_SMALL


def test_mx4_scale_sizes_hold_every_split_of_the_rows(lib):
    # the row tiles of any segments: at most one partial tile per expert with rows
    import random
    rng = random.Random(0)
    for _ in range(200):
        E = rng.randint(1, 40)
        n = [rng.choice([0, 1, 127, 128, 129, rng.randint(0, 600)]) for _ in range(E)]
        c = mx4(R=sum(n), E=E, K=192)
        tiles = sum(-(-v // 128) for v in n)
        assert lib.moe_mx4_row_scale_size(ctypes.byref(c)) >= max(1, tiles) * 2 * 512 * (sum(n) > 0)
    assert lib.moe_mx4_weight_scale_size(ctypes.byref(mx4(K=192, N=192, E=3))) == 3 * 2 * 2 * 512


def test_mx4_config_matches_the_header():
    from test_abi_host import struct_fields
    assert [(n, ctypes.c_int32) for n, t in struct_fields("moe_mx4_config")] == \
        list(L.MoeMx4Config._fields_)


def test_norm_backward_wants_what_the_forward_kept():
    import torch
    import mixture_experts_routed_gb300 as moe
    B.build()
    c = moe.norm_config(4, 64, "f32")
    t, w, r = torch.zeros((4, 64)), torch.ones(64), torch.ones(4)
    with pytest.raises(moe.MoEError, match="KeptNorm"):
        moe.block_norm_backward(c, t, t, t, t, w, None, w, r, r, ws=torch.zeros(8))
