"""Python binding of the routed-MoE layer library: the same entry points as
include/moe.h, taking torch tensors.

Marshalling only: every step of the layer runs in the CUDA library. torch is
used for device memory (outputs a caller does not pass are allocated with
torch), for the current stream, and nothing else. There is no fallback: if
the library is missing, importing the first call raises.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _lib as L

__all__ = ["MoEError", "make_config", "config_from", "workspace_size", "scratch_size",
           "alloc_workspace", "route", "dispatch", "expert_ffn", "combine", "forward",
           "forward_views", "get_device_error", "clear_device_error", "kernel_count",
           "check_config", "backward", "backward_workspace_size", "forward_few",
           "few_workspace_size", "norm_config", "KeptNorm", "block_norm",
           "block_norm_backward", "block_norm_workspace_size", "alloc_norm_workspace",
           "mx4_config", "mx4_quantize_weights", "mx4_quantize_rows", "mx4_product",
           "mx4_dequantize_weights", "mx4_dequantize_rows", "alloc_mx4_workspace",
           "fp8_config", "Fp8Rows", "fp8_quantize_weights", "fp8_quantize_rows", "fp8_product",
           "fp8_weight_grad", "fp8_dequantize_weights", "fp8_dequantize_rows",
           "alloc_fp8_workspace", "router_loss_config", "RouterLoss", "router_loss",
           "router_loss_backward", "alloc_router_loss_workspace", "dropout_config", "dropout",
           "dropout_backward"]


class MoEError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = L.load().moe_strerror(status).decode()
        super().__init__(f"{what}: {msg} (status {status})" if what else msg)


_DTYPES = {"f32": L.MOE_DTYPE_F32, "fp32": L.MOE_DTYPE_F32, "bf16": L.MOE_DTYPE_BF16,
           torch.float32: L.MOE_DTYPE_F32, torch.bfloat16: L.MOE_DTYPE_BF16}


def make_config(T, d, E, k, f, dtype="bf16", router=L.MOE_ROUTER_RENORM, pre_k=8,
                payload_fp8=0, n_group=1, topk_group=1, payload_scale=0.0,
                output_fp8=0, tau=1.0, gemm_tile_n=0, x_perm_mode=0, keep_z=0) -> L.MoeConfig:
    return L.MoeConfig(int(T), int(d), int(E), int(k), int(f), _DTYPES[dtype], int(router), int(pre_k),
                       int(payload_fp8), int(n_group), int(topk_group), float(payload_scale),
                       int(output_fp8), float(tau), int(gemm_tile_n), int(x_perm_mode),
                       int(keep_z))


def config_from(c) -> L.MoeConfig:
    """From any object with T, d, E, k, f, dtype, router, pre_k, payload_fp8
    (and, optionally, n_group, topk_group, payload_scale, output_fp8, tau,
    gemm_tile_n, x_perm_mode, keep_z)."""
    if isinstance(c, L.MoeConfig):
        return c
    return make_config(c.T, c.d, c.E, c.k, c.f, c.dtype, c.router, c.pre_k, c.payload_fp8,
                       getattr(c, "n_group", 1), getattr(c, "topk_group", 1),
                       getattr(c, "payload_scale", 0.0), getattr(c, "output_fp8", 0),
                       getattr(c, "tau", 1.0), getattr(c, "gemm_tile_n", 0),
                       getattr(c, "x_perm_mode", 0), getattr(c, "keep_z", 0))


def _cfg(c):
    return ctypes.byref(config_from(c))


def _p(t):
    """Device address of a dense CUDA tensor: the C ABI takes row-major
    buffers in GPU memory, so a strided view (read with the wrong layout) or
    a host tensor (an address no kernel may touch) is refused here."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise MoEError(L.MOE_ERR_INVALID_ARG, "tensor is not contiguous")
    if not t.is_cuda:
        raise MoEError(L.MOE_ERR_INVALID_ARG, "tensor is not in GPU memory")
    return t.data_ptr()


# The current stream's handle without a Stream object in between (a call costs microseconds
# where a decode step's kernels do), where torch has the query.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _s(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:  # (called once the tensors are known to be in GPU memory)
        return _raw_stream(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def _check(st, what):
    if st != L.MOE_OK:
        raise MoEError(st, what)


def _dt(c):
    return torch.float32 if config_from(c).dtype == L.MOE_DTYPE_F32 else torch.bfloat16


def check_config(c) -> int:
    return L.load().moe_check_config(_cfg(c))


def workspace_size(c) -> int:
    return L.load().moe_workspace_size(_cfg(c))


def scratch_size(c) -> int:
    return L.load().moe_scratch_size(_cfg(c))


def kernel_count(c) -> int:
    return L.load().moe_forward_kernel_count(_cfg(c))


def backward_workspace_size(c) -> int:
    return int(L.load().moe_backward_workspace_size(_cfg(c)))


def few_workspace_size(c) -> int:
    return int(L.load().moe_forward_few_workspace_size(_cfg(c)))


def alloc_workspace(c, kind: str = "forward", device=None) -> torch.Tensor:
    """Zeroed workspace (so the device error word starts clear); kind is
    "forward", "scratch", "backward" or "few"."""
    n = {"forward": workspace_size, "scratch": scratch_size,
         "backward": backward_workspace_size, "few": few_workspace_size}[kind](c)
    if n == 0:
        raise MoEError(L.MOE_ERR_INVALID_ARG, "workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def route(c, x, Wg, bias=None, *, noise=None, topk_idx=None, topk_w=None, logits=None,
          want_logits=False, stream=None):
    """Gate + router. ``noise``: the soft router's Gumbel samples [T, E]."""
    cc = config_from(c)
    dev = x.device
    if topk_idx is None:
        topk_idx = torch.empty((cc.T, cc.k), dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty((cc.T, cc.k), dtype=torch.float32, device=dev)
    if logits is None and want_logits:
        logits = torch.empty((cc.T, cc.E), dtype=torch.float32, device=dev)
    st = L.load().moe_route(ctypes.byref(cc), _p(x), _p(Wg), _p(bias), _p(noise),
                            _p(topk_idx), _p(topk_w), _p(logits), _s(stream))
    _check(st, "moe_route")
    return topk_idx, topk_w, logits


def dispatch(c, x, topk_idx, *, ws, counts=None, offsets=None, pos=None, src=None,
             x_perm=None, x_scale=None, stream=None) -> dict:
    cc = config_from(c)
    dev = x.device
    R = cc.T * cc.k
    i32 = dict(dtype=torch.int32, device=dev)
    counts = torch.empty(cc.E, **i32) if counts is None else counts
    offsets = torch.empty(cc.E + 1, **i32) if offsets is None else offsets
    pos = torch.empty(R, **i32) if pos is None else pos
    src = torch.empty(R, **i32) if src is None else src
    soft = cc.router == L.MOE_ROUTER_SOFT_GUMBEL
    if x_perm is None and not soft:       # soft gating packs no rows
        pdt = torch.uint8 if cc.payload_fp8 else _dt(cc)
        x_perm = torch.empty((R, cc.d), dtype=pdt, device=dev)
    if x_scale is None and cc.payload_fp8:
        x_scale = torch.empty(R, dtype=torch.float32, device=dev)
    st = L.load().moe_dispatch(ctypes.byref(cc), _p(x), _p(topk_idx), _p(counts), _p(offsets),
                               _p(pos), _p(src), _p(x_perm), _p(x_scale), _p(ws),
                               ws.numel() * ws.element_size(), _s(stream))
    _check(st, "moe_dispatch")
    return {"counts": counts, "offsets": offsets, "pos": pos, "src": src, "x_perm": x_perm,
            "x_scale": x_scale}


def expert_ffn(c, x_perm, x_scale, offsets, W1, W2, *, ws, h=None, y_perm=None, stream=None):
    """Grouped FFN. With the soft router ``x_perm`` is x itself ([T, d])."""
    cc = config_from(c)
    dev = x_perm.device
    R = cc.T * cc.k
    if h is None:
        h = torch.empty((R, cc.f), dtype=_dt(cc), device=dev)
    if y_perm is None:
        y_perm = torch.empty((R, cc.d), dtype=torch.float32, device=dev)
    st = L.load().moe_expert_ffn(ctypes.byref(cc), _p(x_perm), _p(x_scale), _p(offsets),
                                 _p(W1), _p(W2), _p(h), _p(y_perm), _p(ws),
                                 ws.numel() * ws.element_size(), _s(stream))
    _check(st, "moe_expert_ffn")
    return h, y_perm


def combine(c, y_perm, pos, topk_w, *, ws, out=None, stream=None):
    cc = config_from(c)
    if out is None:
        out = torch.empty((cc.T, cc.d), dtype=_dt(cc), device=y_perm.device)
    st = L.load().moe_combine(ctypes.byref(cc), _p(y_perm), _p(pos), _p(topk_w), _p(out),
                              _p(ws), ws.numel() * ws.element_size(), _s(stream))
    _check(st, "moe_combine")
    return out


def quantize_output(c, y_perm, *, y_q=None, y_scale=None, y_zero=None, stream=None):
    """FP8 expert-output payload: (y_q uint8 [R, d], y_scale [R], y_zero [R])."""
    cc = config_from(c)
    R, dev = cc.T * cc.k, y_perm.device
    if y_q is None:
        y_q = torch.empty((R, cc.d), dtype=torch.uint8, device=dev)
    if y_scale is None:
        y_scale = torch.empty((R,), dtype=torch.float32, device=dev)
    if y_zero is None:
        y_zero = torch.empty((R,), dtype=torch.float32, device=dev)
    st = L.load().moe_quantize_output(ctypes.byref(cc), _p(y_perm), _p(y_q), _p(y_scale),
                                      _p(y_zero), _s(stream))
    _check(st, "moe_quantize_output")
    return y_q, y_scale, y_zero


def combine_fp8(c, y_q, y_scale, y_zero, pos, topk_w, *, ws, out=None, stream=None):
    cc = config_from(c)
    if out is None:
        out = torch.empty((cc.T, cc.d), dtype=_dt(cc), device=y_q.device)
    st = L.load().moe_combine_fp8(ctypes.byref(cc), _p(y_q), _p(y_scale), _p(y_zero), _p(pos),
                                  _p(topk_w), _p(out), _p(ws), ws.numel() * ws.element_size(),
                                  _s(stream))
    _check(st, "moe_combine_fp8")
    return out


def forward(c, x, Wg, bias, W1, W2, *, ws, out=None, events=None, noise=None, stream=None):
    """The whole layer. ``events``: optional list of MOE_NUM_EVENTS
    torch.cuda.Event (or None) recorded at the kernel boundaries. ``noise``:
    the soft router's Gumbel samples [T, E]."""
    cc = config_from(c)
    if out is None:
        out = torch.empty((cc.T, cc.d), dtype=_dt(cc), device=x.device)
    lib = L.load()
    nbytes = ws.numel() * ws.element_size()
    if events is None:
        st = lib.moe_forward(ctypes.byref(cc), _p(x), _p(Wg), _p(bias), _p(noise), _p(W1),
                             _p(W2), _p(out), _p(ws), nbytes, _s(stream))
    else:
        strm = stream if stream is not None else torch.cuda.current_stream()
        for e in events:
            if e is not None and not e.cuda_event:
                e.record(strm)          # torch creates its CUDA event lazily
        arr = (ctypes.c_void_p * L.MOE_NUM_EVENTS)(
            *[None if e is None else e.cuda_event for e in events])
        st = lib.moe_forward_with_events(ctypes.byref(cc), _p(x), _p(Wg), _p(bias), _p(noise),
                                         _p(W1), _p(W2), _p(out), _p(ws), nbytes, arr,
                                         len(events), _s(stream))
    _check(st, "moe_forward")
    return out


def forward_few(c, x, Wg, bias, W1, W2, *, ws, out=None, noise=None, stream=None):
    """The whole layer for at most MOE_FEW_MAX_TOKENS tokens, in one kernel. ``ws``: a
    "few" workspace."""
    cc = config_from(c)
    T, d, E, f, dt = cc.T, cc.d, cc.E, cc.f, _ndt(cc)
    if out is None:
        out = torch.empty((T, d), dtype=dt, device=x.device)
    # every tensor of the call's shape and type (named only where one is not: a decode step's
    # call costs what its kernel does)
    soft = cc.router == L.MOE_ROUTER_SOFT_GUMBEL
    if not (x.shape == out.shape == (T, d) and Wg.shape == (d, E) and W1.shape == (E, d, f)
            and W2.shape == (E, f, d) and dt is x.dtype is Wg.dtype is W1.dtype is W2.dtype
            and out.dtype is dt
            and (bias is None or bias.shape == (E,) and bias.dtype is torch.float32)) or soft:
        for name, t, shape, of in (
                ("x", x, (T, d), dt), ("Wg", Wg, (d, E), dt), ("bias", bias, (E,), torch.float32),
                ("W1", W1, (E, d, f), dt), ("W2", W2, (E, f, d), dt), ("out", out, (T, d), dt),
                ("noise", noise if soft else None, (T, E), torch.float32)):
            if t is not None and (t.shape != shape or t.dtype is not of):
                raise MoEError(L.MOE_ERR_INVALID_ARG, f"{name} is {tuple(t.shape)} {t.dtype}, not "
                                                      f"{shape} {of}")
    st = L.load().moe_forward_few(ctypes.byref(cc), _p(x), _p(Wg), _p(bias), _p(noise), _p(W1),
                                  _p(W2), _p(out), _p(ws), ws.nbytes, _s(stream))
    _check(st, "moe_forward_few")
    return out


def backward(c, x, Wg, bias, W1, W2, dout, *, fwd_ws, ws, noise=None, dlogits=None,
             stream=None) -> dict:
    """Gradients of the layer for dout = dl/dout [T, d] after a forward in
    ``fwd_ws`` on the same inputs: dx [T, d], dWg [d, E], dbias [E], dW1 [E,
    d, f], dW2 [E, f, d], all fp32. ``ws``: a backward workspace. ``dlogits`` (fp32 [T, E]): a
    gradient of the logits from elsewhere (``router_loss_backward``'s), added to the router's."""
    cc = config_from(c)
    dev = x.device
    g = {"dx": torch.empty((cc.T, cc.d), dtype=torch.float32, device=dev),
         "dWg": torch.empty((cc.d, cc.E), dtype=torch.float32, device=dev),
         "dbias": torch.empty((cc.E,), dtype=torch.float32, device=dev),
         "dW1": torch.empty((cc.E, cc.d, cc.f), dtype=torch.float32, device=dev),
         "dW2": torch.empty((cc.E, cc.f, cc.d), dtype=torch.float32, device=dev)}
    lib = L.load()
    call, more = lib.moe_backward, ()
    if dlogits is not None:
        call = lib.moe_backward_with_dlogits
        more = (_shaped("dlogits", dlogits, (cc.T, cc.E), torch.float32),)
    st = call(
        ctypes.byref(cc), _p(x), _p(Wg), _p(bias), _p(noise), _p(W1), _p(W2), _p(fwd_ws),
        fwd_ws.numel() * fwd_ws.element_size(), _p(dout), *more, _p(g["dx"]), _p(g["dWg"]),
        _p(g["dbias"]), _p(g["dW1"]), _p(g["dW2"]), _p(ws), ws.numel() * ws.element_size(),
        _s(stream))
    _check(st, "moe_backward")
    return g


def forward_views(c, ws) -> dict:
    """Tensors viewing the intermediates of the last forward in ``ws``."""
    cc = config_from(c)
    v = L.MoeForwardViews()
    _check(L.load().moe_forward_views(ctypes.byref(cc), _p(ws), ctypes.byref(v)),
           "moe_forward_views")
    base = ws.data_ptr()
    R = cc.T * cc.k

    def view(ptr, n, dtype, shape):
        if ptr is None:
            return None
        off = ptr - base
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return ws[off:off + nbytes].view(dtype).view(shape)

    pdt = torch.uint8 if cc.payload_fp8 else _dt(cc)
    return {
        "topk_idx": view(v.topk_idx, R, torch.int32, (cc.T, cc.k)),
        "topk_w": view(v.topk_w, R, torch.float32, (cc.T, cc.k)),
        "counts": view(v.counts, cc.E, torch.int32, (cc.E,)),
        "offsets": view(v.offsets, cc.E + 1, torch.int32, (cc.E + 1,)),
        "pos": view(v.pos, R, torch.int32, (R,)),
        "src": view(v.src, R, torch.int32, (R,)),
        "x_perm": view(v.x_perm, R * cc.d, pdt, (R, cc.d)) if v.x_perm else None,
        "x_scale": view(v.x_scale, R, torch.float32, (R,)) if cc.payload_fp8 else None,
        "h": view(v.h, R * cc.f, _dt(cc), (R, cc.f)),
        "y_perm": view(v.y_perm, R * cc.d, torch.float32, (R, cc.d)),
        "y_q": view(v.y_q, R * cc.d, torch.uint8, (R, cc.d)) if cc.output_fp8 else None,
        "y_scale": view(v.y_scale, R, torch.float32, (R,)) if cc.output_fp8 else None,
        "y_zero": view(v.y_zero, R, torch.float32, (R,)) if cc.output_fp8 else None,
        "z": view(v.z, R * cc.f, torch.float32, (R, cc.f)) if cc.keep_z else None,
    }


def get_device_error(ws, stream=None) -> int:
    """Synchronise, read and clear the workspace error word (a moe status)."""
    return L.load().moe_get_device_error(_p(ws), _s(stream))


def clear_device_error(ws, stream=None) -> None:
    _check(L.load().moe_clear_device_error(_p(ws), _s(stream)), "moe_clear_device_error")


# ---------------------------------------------------------------- norms around a block
_GATES = {"none": L.MOE_GATE_NONE, "token": L.MOE_GATE_TOKEN, "channel": L.MOE_GATE_CHANNEL,
          "element": L.MOE_GATE_ELEMENT}


def norm_config(T, d, dtype="bf16", gate="none", eps=1e-6, alpha=1.0, beta=1.0) -> L.MoeNormConfig:
    """gate: "none", "token", "channel", "element" or a MOE_GATE_* value."""
    return L.MoeNormConfig(int(T), int(d), _DTYPES[dtype], int(_GATES.get(gate, gate)),
                           float(eps), float(alpha), float(beta))


def _ndt(c):
    return torch.float32 if c.dtype == L.MOE_DTYPE_F32 else torch.bfloat16


def block_norm_workspace_size(c) -> int:
    return int(L.load().moe_block_norm_backward_workspace_size(ctypes.byref(c)))


def alloc_norm_workspace(c, device=None) -> torch.Tensor:
    n = block_norm_workspace_size(c)
    if n == 0:
        raise MoEError(L.MOE_ERR_INVALID_ARG, "workspace size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _shaped(name, t, shape, dtype):
    """Device address of a tensor of the call's shape and type (None stays None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype:
        raise MoEError(L.MOE_ERR_INVALID_ARG, f"{name} is {tuple(t.shape)} {t.dtype}, not "
                                              f"{tuple(shape)} {dtype}")
    if t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return _p(t)


def _gate_form(kind, T, d, dt):
    """(shape, type) of the gate, None without one."""
    if kind == L.MOE_GATE_TOKEN:
        return (T,), torch.float32
    if kind == L.MOE_GATE_CHANNEL:
        return (d,), torch.float32
    return ((T, d), dt) if kind == L.MOE_GATE_ELEMENT else None


class KeptNorm(NamedTuple):
    """What a forward with both halves keeps for the gradient through its second norm: that
    norm's 1 / root mean square [T] and x, from which (with b) out is formed again in fp32."""
    rstd: torch.Tensor
    x: torch.Tensor


def block_norm(c, x, b=None, w_post=None, gate=None, w_pre=None, *, out=None, n=None,
               rstd_post=None, rstd_pre=None, want_rstd=False, stream=None) -> dict:
    """out = alpha x + beta gate * norm(b) w_post and n = norm(out) w_pre; without ``b``
    out is x, without ``w_pre`` there is no n. ``want_rstd``: keep what the backward reads,
    under "rstd_post" (fp32 [T]) and "rstd_pre" (fp32 [T]; with both halves a ``KeptNorm`` of
    it and x, which must not change before the backward)."""
    T, d, f32 = c.T, c.d, torch.float32
    dt, td = _ndt(c), (T, d)
    post, pre = b is not None, w_pre is not None
    px = _shaped("x", x, td, dt)
    if out is not None or not post:
        po = _shaped("out", out, td, dt)
    else:
        out = torch.empty_like(x)
        po = out.data_ptr()
    if n is not None or not pre:
        pn = _shaped("n", n, td, dt)
    else:
        n = torch.empty_like(x)
        pn = n.data_ptr()
    if want_rstd and post and rstd_post is None:
        rstd_post = torch.empty(T, dtype=f32, device=x.device)
    if want_rstd and pre and rstd_pre is None:
        rstd_pre = torch.empty(T, dtype=f32, device=x.device)
    if isinstance(rstd_pre, KeptNorm):  # (one to be filled again)
        rstd_pre = rstd_pre.rstd
    form = _gate_form(c.gate, T, d, dt) if post else None
    st = L.load().moe_block_norm(
        ctypes.byref(c), px, _shaped("b", b, td, dt), _shaped("w_post", w_post, (d,), f32),
        _shaped("gate", gate, *form) if form else None, _shaped("w_pre", w_pre, (d,), f32),
        po, pn, _shaped("rstd_post", rstd_post, (T,), f32), _shaped("rstd_pre", rstd_pre, (T,), f32),
        _s(stream))
    _check(st, "moe_block_norm")
    if post and rstd_pre is not None:
        rstd_pre = KeptNorm(rstd_pre, x)
    return {"out": out, "n": n, "rstd_post": rstd_post, "rstd_pre": rstd_pre}


def block_norm_backward(c, dout, dn, y, b, w_post, gate, w_pre, rstd_post, rstd_pre, *, ws,
                        stream=None) -> dict:
    """Gradients after a ``block_norm`` of the same inputs: ``dout`` is the gradient that
    reaches its out by the residual, ``dn`` (fp32) the one of n, ``rstd_post`` and
    ``rstd_pre`` what it kept. ``y``: without ``b``, the x that was normed; with it, the
    forward's out or None: it is not read (``rstd_pre`` has what stands in for it). dx, db, an
    element gate's dgate in the config's type; dw_post, dw_pre and the other dgate fp32; None
    for what the forward left out."""
    T, d, f32 = c.T, c.d, torch.float32
    dt, td = _ndt(c), (T, d)
    post, pre = w_post is not None, w_pre is not None
    form = _gate_form(c.gate, T, d, dt) if post else None
    if post and pre:
        if not isinstance(rstd_pre, KeptNorm):
            raise MoEError(L.MOE_ERR_INVALID_ARG,
                           "rstd_pre of a forward with both halves is the KeptNorm it returned")
        if y is not None and (y.shape != td or y.dtype is not dt):
            raise MoEError(L.MOE_ERR_INVALID_ARG, f"y is {tuple(y.shape)} {y.dtype}, not {td} {dt}")
        rstd_pre, y = rstd_pre
    pd = _shaped("dout", dout, td, dt)
    g = {"dx": torch.empty_like(dout), "db": torch.empty_like(dout) if post else None,
         "dw_post": torch.empty_like(w_post) if post else None, "dgate": None,
         "dw_pre": torch.empty_like(w_pre) if pre else None}
    if form:
        g["dgate"] = torch.empty(form[0], dtype=form[1], device=dout.device)
    st = L.load().moe_block_norm_backward(
        ctypes.byref(c), pd, _shaped("dn", dn, td, f32), _shaped("y", y, td, dt) if pre else None,
        _shaped("b", b, td, dt), _shaped("w_post", w_post, (d,), f32),
        _shaped("gate", gate, *form) if form else None, _shaped("w_pre", w_pre, (d,), f32),
        _shaped("rstd_post", rstd_post, (T,), f32) if post else None,
        _shaped("rstd_pre", rstd_pre, (T,), f32) if pre else None,
        *[None if t is None else t.data_ptr() for t in g.values()], _p(ws), ws.nbytes,
        _s(stream))
    _check(st, "moe_block_norm_backward")
    return g


# ---------------------------------------------------------------- 4-bit expert products
def mx4_config(R, K, N, E, dtype="bf16", out_dtype="bf16", silu=0, x_rows=0) -> L.MoeMx4Config:
    return L.MoeMx4Config(int(R), int(K), int(N), int(E), _DTYPES[dtype], _DTYPES[out_dtype],
                          int(silu), int(x_rows))


def alloc_mx4_workspace(c, device=None) -> torch.Tensor:
    """Zeroed workspace of the 4-bit calls (one serves any configuration)."""
    n = int(L.load().moe_mx4_workspace_size(ctypes.byref(c)))
    if n == 0:
        raise MoEError(L.MOE_ERR_INVALID_ARG, "workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _scale_p(name, n, t):
    if t.dtype is not torch.uint8 or t.numel() < n or n == 0:
        raise MoEError(L.MOE_ERR_INVALID_ARG, f"{name} is {t.numel()} {t.dtype}, not {n} uint8")
    return _p(t)


def _indices(name, t, n):
    if t is not None and (t.dtype is not torch.int32 or t.numel() != n):
        raise MoEError(L.MOE_ERR_INVALID_ARG, f"{name} is {t.numel()} {t.dtype}, not {n} int32")
    return _p(t)


def _bytes(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device)


def mx4_quantize_weights(c, W, *, q=None, scale=None, stream=None):
    """W [E, K, N] -> (codes uint8 [E, N, K / 2], scales uint8 in the product's layout)."""
    lib, r = L.load(), ctypes.byref(c)
    E, K, N = c.E, c.K, c.N
    n = lib.moe_mx4_weight_scale_size(r)
    if q is None:
        q = torch.empty((E, N, K // 2), dtype=torch.uint8, device=W.device)
    if scale is None:
        scale = _bytes(n, W.device)
    st = lib.moe_mx4_quantize_weights(r, _shaped("W", W, (E, K, N), _ndt(c)),
                                      _shaped("q", q, (E, N, K // 2), torch.uint8),
                                      _scale_p("scale", n, scale), _s(stream))
    _check(st, "moe_mx4_quantize_weights")
    return q, scale


def mx4_quantize_rows(c, x, offsets, *, ws, src=None, q=None, scale=None, stream=None):
    """Rows x [R, K], or with ``src`` [R] the rows x[src] of x [x_rows, K] -> (codes uint8
    [R, K / 2], scales uint8 laid out for ``offsets``)."""
    lib, r = L.load(), ctypes.byref(c)
    R, K = c.R, c.K
    n = lib.moe_mx4_row_scale_size(r)
    if q is None:
        q = torch.empty((R, K // 2), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = _bytes(n, x.device)
    st = lib.moe_mx4_quantize_rows(
        r, _shaped("x", x, (R if src is None else c.x_rows, K), _ndt(c)),
        _indices("src", src, R), _indices("offsets", offsets, c.E + 1),
        _shaped("q", q, (R, K // 2), torch.uint8), _scale_p("scale", n, scale), _p(ws), ws.nbytes,
        _s(stream))
    _check(st, "moe_mx4_quantize_rows")
    return q, scale


def mx4_product(c, q, scale, wq, w_scale, offsets, *, ws, out=None, stream=None):
    """out[r] = rows q[r] . weights wq[e] over each expert's segment, [R, N]."""
    lib, r = L.load(), ctypes.byref(c)
    R, K, N, E = c.R, c.K, c.N, c.E
    odt = torch.float32 if c.out_dtype == L.MOE_DTYPE_F32 else torch.bfloat16
    if out is None:
        out = torch.empty((R, N), dtype=odt, device=q.device)
    st = lib.moe_mx4_product(
        r, _shaped("q", q, (R, K // 2), torch.uint8),
        _scale_p("scale", lib.moe_mx4_row_scale_size(r), scale),
        _shaped("wq", wq, (E, N, K // 2), torch.uint8),
        _scale_p("w_scale", lib.moe_mx4_weight_scale_size(r), w_scale),
        _indices("offsets", offsets, E + 1), _shaped("out", out, (R, N), odt), _p(ws), ws.nbytes,
        _s(stream))
    _check(st, "moe_mx4_product")
    return out


def mx4_dequantize_weights(c, wq, w_scale, *, W=None, stream=None):
    """The values of quantised weights, [E, K, N]."""
    lib, r = L.load(), ctypes.byref(c)
    E, K, N = c.E, c.K, c.N
    if W is None:
        W = torch.empty((E, K, N), dtype=_ndt(c), device=wq.device)
    st = lib.moe_mx4_dequantize_weights(
        r, _shaped("wq", wq, (E, N, K // 2), torch.uint8),
        _scale_p("w_scale", lib.moe_mx4_weight_scale_size(r), w_scale),
        _shaped("W", W, (E, K, N), _ndt(c)), _s(stream))
    _check(st, "moe_mx4_dequantize_weights")
    return W


def mx4_dequantize_rows(c, q, scale, offsets, *, x=None, stream=None):
    """The values of quantised rows, [R, K] (rows outside the segments are not written, and with
    offsets that fall or leave [0, R] none is)."""
    lib, r = L.load(), ctypes.byref(c)
    R, K = c.R, c.K
    if x is None:
        x = torch.empty((R, K), dtype=_ndt(c), device=q.device)
    st = lib.moe_mx4_dequantize_rows(
        r, _shaped("q", q, (R, K // 2), torch.uint8),
        _scale_p("scale", lib.moe_mx4_row_scale_size(r), scale),
        _indices("offsets", offsets, c.E + 1), _shaped("x", x, (R, K), _ndt(c)), _s(stream))
    _check(st, "moe_mx4_dequantize_rows")
    return x


# ---------------------------------------------------------------- 8-bit expert products
_ACTS = {None: L.MOE_ACT_NONE, "silu": L.MOE_ACT_SILU, "silu_grad": L.MOE_ACT_SILU_GRAD}


def fp8_config(R, K, N, E, dtype="bf16", out_dtype="bf16", silu=0, x_rows=0) -> L.MoeFp8Config:
    return L.MoeFp8Config(int(R), int(K), int(N), int(E), _DTYPES[dtype], _DTYPES[out_dtype],
                          int(silu), int(x_rows))


def alloc_fp8_workspace(c, device=None) -> torch.Tensor:
    """Zeroed workspace of the 8-bit calls (one serves any configuration)."""
    n = int(L.load().moe_fp8_workspace_size(ctypes.byref(c)))
    if n == 0:
        raise MoEError(L.MOE_ERR_INVALID_ARG, "workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _fp8_pitch(cols):
    return (-(-cols // 128) + 3) // 4 * 4


class Fp8Rows:
    """Quantised rows [R, C], uint8: codes ``q`` and scales ``scale`` [R, pitch] of blocks of 128
    along a row, codes ``cq`` [128 tiles, C] and scales ``cscale`` [tiles, ceil(C / 128), 128] of
    blocks of 128 rows of an expert; None for a form that was not asked for. Views of one buffer,
    made where they are asked for."""
    __slots__ = ("buf", "R", "C", "rows", "columns", "tiles", "at")

    def __init__(self, R, C, rows, columns, tiles, device):
        self.R, self.C, self.rows, self.columns, self.tiles = R, C, rows, columns, tiles
        # where q, scale, cq and cscale begin, and the end
        q = R * C if rows else 0
        s = q + ((R * _fp8_pitch(C) + 255) // 256 * 256 if rows else 0)
        c = s + (tiles * 128 * C if columns else 0)
        self.at = (0, q, s, c, c + (tiles * -(-C // 128) * 128 if columns else 0))
        self.buf = torch.empty(self.at[4], dtype=torch.uint8, device=device)

    def _view(self, i, *shape):
        return self.buf[self.at[i]:self.at[i + 1]][:shape[0] * shape[1]].view(shape[0], shape[1])

    @property
    def q(self):
        return self._view(0, self.R, self.C) if self.rows else None

    @property
    def scale(self):
        return self._view(1, self.R, _fp8_pitch(self.C)) if self.rows else None

    @property
    def cq(self):
        return self._view(2, self.tiles * 128, self.C) if self.columns else None

    @property
    def cscale(self):
        n = -(-self.C // 128)
        return self._view(3, self.tiles, n * 128).view(-1, n, 128) if self.columns else None

    def pointers(self, form, name, R, C, tiles=None):
        """Device addresses of a form's codes and scales, if it has that and the call's sizes."""
        if not (self.rows if form == 0 else self.columns):
            raise MoEError(L.MOE_ERR_INVALID_ARG,
                           f"{name} was not quantised in the form this takes")
        if (self.R, self.C) != (R, C) or tiles not in (None, self.tiles):
            raise MoEError(L.MOE_ERR_INVALID_ARG, f"{name} is {(self.R, self.C)}, not {(R, C)}")
        if not self.buf.is_cuda:
            raise MoEError(L.MOE_ERR_INVALID_ARG, f"{name} is not in GPU memory")
        base = self.buf.data_ptr()
        return base + self.at[2 * form], base + self.at[2 * form + 1]


def fp8_quantize_weights(c, W, *, q=None, scale=None, stream=None):
    """W [E, K, N] -> (codes uint8 [E, K, N], scales uint8 [E, ceil(K / 128), ceil(N / 128)])."""
    E, K, N = c.E, c.K, c.N
    blocks = (E, -(-K // 128), -(-N // 128))
    u8 = torch.uint8
    if q is None:
        q = torch.empty((E, K, N), dtype=u8, device=W.device)
    if scale is None:
        scale = torch.empty(blocks, dtype=u8, device=W.device)
    st = L.load().moe_fp8_quantize_weights(ctypes.byref(c), _shaped("W", W, (E, K, N), _ndt(c)),
                                           _shaped("q", q, (E, K, N), u8),
                                           _shaped("scale", scale, blocks, u8), _s(stream))
    _check(st, "moe_fp8_quantize_weights")
    return q, scale


def fp8_quantize_rows(c, x, offsets, *, ws, rows=True, columns=False, src=None, row_weight=None,
                      act=None, z=None, stream=None) -> Fp8Rows:
    """Rows x [R, K] or [R, N], or with ``src`` [R] the rows x[src] of x [x_rows, ..], times
    ``row_weight`` [R], in the forms asked for. ``act``: None, "silu" (of x) or "silu_grad" (x
    times SiLU'(z), z [R, ..])."""
    lib, r = L.load(), ctypes.byref(c)
    R, C, dt = c.R, x.shape[-1], _ndt(c)
    if act not in _ACTS:
        raise MoEError(L.MOE_ERR_INVALID_ARG, f"act is {act!r}")
    if C not in (c.K, c.N):
        raise MoEError(L.MOE_ERR_INVALID_ARG, f"x has {C} columns, not {c.K} or {c.N}")
    if not (rows or columns):
        raise MoEError(L.MOE_ERR_INVALID_ARG, "neither rows nor columns asked for")
    px = _shaped("x", x, (R if src is None else c.x_rows, C), dt)
    out = Fp8Rows(R, C, rows, columns, int(lib.moe_fp8_column_rows(r)) // 128 if columns else 0,
                  x.device)
    at, (_, o1, o2, o3, _) = out.buf.data_ptr(), out.at
    st = lib.moe_fp8_quantize_rows(
        r, C, px, None if src is None else _indices("src", src, R),
        None if row_weight is None else _shaped("row_weight", row_weight, (R,), torch.float32),
        _ACTS[act], None if z is None else _shaped("z", z, (R, C), dt),
        _indices("offsets", offsets, c.E + 1), at if rows else None, at + o1 if rows else None,
        at + o2 if columns else None, at + o3 if columns else None, _p(ws), ws.nbytes, _s(stream))
    _check(st, "moe_fp8_quantize_rows")
    return out


def _fp8_weights(c, wq, w_scale):
    return (_shaped("wq", wq, (c.E, c.K, c.N), torch.uint8),
            _shaped("w_scale", w_scale, (c.E, -(-c.K // 128), -(-c.N // 128)), torch.uint8))


def fp8_product(c, rows, wq, w_scale, offsets, *, ws, transposed=False, out=None, stream=None):
    """out[r] = rows[r] . W[e], [R, N], from rows of K columns; ``transposed``: rows[r] . W[e]^T,
    [R, K], from rows of N columns."""
    R = c.R
    length, width = (c.N, c.K) if transposed else (c.K, c.N)
    odt = torch.float32 if c.out_dtype == L.MOE_DTYPE_F32 else torch.bfloat16
    pq, ps = rows.pointers(0, "rows", R, length)
    pw, pws = _fp8_weights(c, wq, w_scale)
    if out is None:
        out = torch.empty((R, width), dtype=odt, device=wq.device)
        po = out.data_ptr()
    else:
        po = _shaped("out", out, (R, width), odt)
    st = L.load().moe_fp8_product(ctypes.byref(c), int(transposed), pq, ps, pw, pws,
                                  _indices("offsets", offsets, c.E + 1), po, _p(ws), ws.nbytes,
                                  _s(stream))
    _check(st, "moe_fp8_product")
    return out


def fp8_weight_grad(c, x, dy, offsets, *, ws, out=None, stream=None):
    """fp32 dW [E, K, N]: the sum over each expert's rows of x[r]^T dy[r], from the columns of x
    [R, K] and of dy [R, N]."""
    lib, r = L.load(), ctypes.byref(c)
    R, E, K, N = c.R, c.E, c.K, c.N
    tiles = int(lib.moe_fp8_column_rows(r)) // 128
    px, pxs = x.pointers(1, "x", R, K, tiles)
    pd, pds = dy.pointers(1, "dy", R, N, tiles)
    if out is None:
        out = torch.empty((E, K, N), dtype=torch.float32, device=x.buf.device)
    st = lib.moe_fp8_weight_grad(r, px, pxs, pd, pds, _indices("offsets", offsets, E + 1),
                                 _shaped("out", out, (E, K, N), torch.float32), _p(ws), ws.nbytes,
                                 _s(stream))
    _check(st, "moe_fp8_weight_grad")
    return out


def fp8_dequantize_weights(c, wq, w_scale, *, W=None, stream=None):
    """The values of quantised weights, [E, K, N]."""
    if W is None:
        W = torch.empty((c.E, c.K, c.N), dtype=_ndt(c), device=wq.device)
    st = L.load().moe_fp8_dequantize_weights(
        ctypes.byref(c), *_fp8_weights(c, wq, w_scale),
        _shaped("W", W, (c.E, c.K, c.N), _ndt(c)), _s(stream))
    _check(st, "moe_fp8_dequantize_weights")
    return W


def fp8_dequantize_rows(c, rows, *, x=None, stream=None):
    """The values of quantised rows, [R, C], from their ``q`` and ``scale``."""
    R, C = c.R, rows.C
    pq, ps = rows.pointers(0, "rows", R, C)
    if x is None:
        x = torch.empty((R, C), dtype=_ndt(c), device=rows.buf.device)
    st = L.load().moe_fp8_dequantize_rows(ctypes.byref(c), C, pq, ps,
                                          _shaped("x", x, (R, C), _ndt(c)), _s(stream))
    _check(st, "moe_fp8_dequantize_rows")
    return x


# ---------------------------------------------------------------- the router's losses
def router_loss_config(T, E, k, S=1, balance=0.01, z=0.0) -> L.MoeRouterLossConfig:
    """``balance`` and ``z``: the two losses' coefficients."""
    return L.MoeRouterLossConfig(int(T), int(E), int(k), int(S), float(balance), float(z))


def alloc_router_loss_workspace(c, device=None) -> torch.Tensor:
    n = int(L.load().moe_router_loss_workspace_size(ctypes.byref(c)))
    if n == 0:
        raise MoEError(L.MOE_ERR_INVALID_ARG, "workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


class RouterLoss(NamedTuple):
    """``loss`` fp32 [3]: the loss, the balance and the z loss without their coefficients;
    ``counts`` int32 [S, E]: the experts' tokens by sequence. ``tokens`` int32 [S + 2] (by
    sequence, sequences with any, all) and ``lse`` fp32 [T] are the backward's."""
    loss: torch.Tensor
    counts: torch.Tensor
    tokens: torch.Tensor
    lse: torch.Tensor


def router_loss(c, logits, topk_idx, *, ws, offsets=None, mask=None, stream=None) -> RouterLoss:
    """The router's losses of logits [T, E] and choices [T, k]. ``offsets`` int32 [S + 1]: the
    sequences' tokens (None: one of all); ``mask`` [T], bool or uint8: the tokens that count."""
    T, E, k, S = c.T, c.E, c.k, c.S
    i32, dev = torch.int32, logits.device
    r = RouterLoss(torch.empty(3, dtype=torch.float32, device=dev),
                   torch.empty((S, E), dtype=i32, device=dev),
                   torch.empty(S + 2, dtype=i32, device=dev),
                   torch.empty(T, dtype=torch.float32, device=dev))
    st = L.load().moe_router_loss(
        ctypes.byref(c), _shaped("logits", logits, (T, E), torch.float32),
        _shaped("topk_idx", topk_idx, (T, k), i32),
        None if offsets is None else _indices("offsets", offsets, S + 1),
        None if mask is None else _mask_p(mask, T), r.loss.data_ptr(), r.counts.data_ptr(),
        r.tokens.data_ptr(), r.lse.data_ptr(), _p(ws), ws.nbytes, _s(stream))
    _check(st, "moe_router_loss")
    return r


def router_loss_backward(c, logits, kept, *, dloss=None, offsets=None, mask=None, out=None,
                         stream=None):
    """fp32 [T, E]: ``dloss`` (fp32 [1]; None: 1) times the gradient of loss[0] by the logits,
    after a ``router_loss`` of the same inputs that gave ``kept``. What ``backward`` takes as
    ``dlogits``."""
    T, E, S, f32 = c.T, c.E, c.S, torch.float32
    px = _shaped("logits", logits, (T, E), f32)
    if out is None:
        out = torch.empty_like(logits)
        pout = out.data_ptr()
    else:
        pout = _shaped("out", out, (T, E), f32)
    st = L.load().moe_router_loss_backward(
        ctypes.byref(c), px, None if offsets is None else _indices("offsets", offsets, S + 1),
        None if mask is None else _mask_p(mask, T),
        _shaped("counts", kept.counts, (S, E), torch.int32),
        _shaped("tokens", kept.tokens, (S + 2,), torch.int32),
        _shaped("lse", kept.lse, (T,), f32),
        None if dloss is None else _shaped("dloss", dloss, (1,), f32), pout, _s(stream))
    _check(st, "moe_router_loss_backward")
    return out


def _mask_p(mask, T):
    if mask is not None and (mask.shape != (T,) or mask.dtype not in (torch.bool, torch.uint8)):
        raise MoEError(L.MOE_ERR_INVALID_ARG, f"mask is {tuple(mask.shape)} {mask.dtype}, not "
                                              f"{(T,)} bool or uint8")
    return _p(mask)


# ---------------------------------------------------------------- dropout of a branch
def dropout_config(T, d, dtype="bf16", p=0.1, site=0) -> L.MoeDropoutConfig:
    """``site``: which of a model's dropouts this is; each draws a mask of its own."""
    return L.MoeDropoutConfig(int(T), int(d), _DTYPES[dtype], int(site), float(p))


def dropout(c, x, state, *, residual=None, out=None, stream=None):
    """residual + x dropped and scaled, [T, d]. ``state``: int64 [2] on the GPU, the seed and the
    step; its values at the time the kernel runs are used. ``out`` may be x or residual."""
    td, dt = (c.T, c.d), _ndt(c)
    px = _shaped("x", x, td, dt)
    pr = None if residual is None else _shaped("residual", residual, td, dt)
    ps = _shaped("state", state, (2,), torch.int64)
    if out is None:
        out = torch.empty_like(x)
        po = out.data_ptr()
    else:
        po = _shaped("out", out, td, dt)
    _check(L.load().moe_dropout(ctypes.byref(c), px, pr, ps, po, _s(stream)), "moe_dropout")
    return out


def dropout_backward(c, dout, state, *, dx=None, stream=None):
    """dx [T, d] of a ``dropout`` with this config and state (the residual's gradient is dout)."""
    td, dt = (c.T, c.d), _ndt(c)
    pd = _shaped("dout", dout, td, dt)
    ps = _shaped("state", state, (2,), torch.int64)
    if dx is None:
        dx = torch.empty_like(dout)
        px = dx.data_ptr()
    else:
        px = _shaped("dx", dx, td, dt)
    _check(L.load().moe_dropout_backward(ctypes.byref(c), pd, ps, px, _s(stream)),
           "moe_dropout_backward")
    return dx
