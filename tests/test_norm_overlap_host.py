"""The norm calls refuse outputs that overlap their inputs or one another, on the host, before
any CUDA call (no GPU needed; the addresses are never read). Rows too wide for the ring are read
again after out is written, so an overlap would give wrong values without a word."""
import ctypes

import pytest

from mixture_experts_routed_gb300 import _lib as L
from mixture_experts_routed_gb300 import build as B

T, D = 4, 16448
ROWS = T * D * 4  # bytes of a [T, d] fp32 tensor
FORWARD = ["x", "b", "w_post", "gate", "w_pre", "out", "n", "rstd_post", "rstd_pre"]
BACKWARD = ["dout", "dn", "x", "b", "w_post", "gate", "w_pre", "rstd_post", "rstd_pre", "dx", "db",
            "dw_post", "dgate", "dw_pre", "ws"]


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def addresses(names):
    return {n: (i + 1) << 30 for i, n in enumerate(names)}


def status(lib, names, at):
    c = L.MoeNormConfig(T, D, 0, 3, 1e-6, 1.0, 1.0)
    args = [ctypes.c_void_p(at[n]) for n in names]
    if names is FORWARD:
        return lib.moe_block_norm(ctypes.byref(c), *args, None)
    return lib.moe_block_norm_backward(ctypes.byref(c), *args, 1 << 29, None)


@pytest.mark.parametrize("out,other,shift", [
    ("out", "x", 0), ("out", "b", 0), ("n", "x", 0), ("out", "x", ROWS - 16), ("x", "out", ROWS - 16),
    ("n", "gate", 0), ("out", "w_post", 0), ("w_pre", "n", ROWS - 16), ("n", "out", 0),
    ("rstd_post", "x", 0), ("rstd_pre", "rstd_post", 8), ("rstd_pre", "n", ROWS - 4)])
def test_forward(lib, out, other, shift):
    at = addresses(FORWARD)
    at[out] = at[other] + shift
    assert status(lib, FORWARD, at) == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("out,other,shift", [
    ("dx", "dout", 0), ("dx", "x", 0), ("db", "b", 0), ("db", "dout", ROWS - 16), ("dgate", "gate", 0),
    ("dx", "dn", 0), ("dw_pre", "w_pre", 0), ("dw_post", "w_post", 16), ("dx", "db", 0),
    ("dgate", "db", 0), ("rstd_pre", "dx", 4), ("ws", "dx", 0), ("dw_pre", "ws", 0),
    ("ws", "dn", 0)])
def test_backward(lib, out, other, shift):
    at = addresses(BACKWARD)
    at[out] = at[other] + shift
    assert status(lib, BACKWARD, at) == L.MOE_ERR_INVALID_ARG
