"""The expert half of a transformer block, run the three ways it is used.

    n = norm(x) w_pre;   b = experts(n);   out = alpha x + beta g * (norm(b) w_post)

  decode   a few tokens: the block norms around the one-kernel layer (forward_few)
  prefill  many tokens, the experts' weights and rows in 4 bits (mx4_*)
  train    a step's forward and backward: block norms, forward with kept Z, backward

The norm after one block and the norm before the next are one call, so a chain of blocks
costs one norm call a block.

    python examples/expert_block.py [--d 2048 --f 1408 --E 64 --k 2] [--tokens 4096] [--decode 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_routed_gb300 as moe  # noqa: E402


class ExpertBlock:
    """Weights of one block's expert half (synthetic), in bf16 and, for prefill, 4 bits."""

    def __init__(self, d, f, E, k, alpha=1.0, beta=1.0, seed=0, device="cuda"):
        self.d, self.f, self.E, self.k = d, f, E, k
        self.alpha, self.beta = alpha, beta
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def draw(*shape, std=1.0, dtype=torch.bfloat16):
            return (std * torch.randn(shape, generator=g, device=device)).to(dtype)

        self.Wg = draw(d, E, std=d ** -0.5)
        self.bias = draw(E, std=0.5, dtype=torch.float32)
        self.W1 = draw(E, d, f, std=d ** -0.5)
        self.W2 = draw(E, f, d, std=f ** -0.5)
        self.w_pre = 1 + draw(d, std=0.1, dtype=torch.float32)
        self.w_post = 1 + draw(d, std=0.1, dtype=torch.float32)
        self.w_next = 1 + draw(d, std=0.1, dtype=torch.float32)  # the next block's w_pre
        self.gate = torch.sigmoid(draw(d, dtype=torch.float32))  # per channel
        self._mx4 = None

    def config(self, T, **kw):
        return moe.make_config(T, self.d, self.E, self.k, self.f, "bf16",
                               pre_k=min(8, self.E), **kw)

    def norms(self, T):
        return moe.norm_config(T, self.d, "bf16", gate="channel", alpha=self.alpha, beta=self.beta)

    # ------------------------------------------------------------ decode
    def decode(self, x, ws):
        """x [T, d], T <= MOE_FEW_MAX_TOKENS; ws: alloc_workspace(config(T), "few")."""
        T = x.shape[0]
        c, nc = self.config(T), self.norms(T)
        n = moe.block_norm(nc, x, w_pre=self.w_pre)["n"]
        b = moe.forward_few(c, n, self.Wg, self.bias, self.W1, self.W2, ws=ws)
        r = moe.block_norm(nc, x, b, self.w_post, self.gate, self.w_next)
        return r["out"], r["n"]

    # ------------------------------------------------------------ prefill, 4-bit experts
    def quantize(self):
        """The experts' weights in 4 bits (once, where they are loaded)."""
        up = moe.mx4_config(1, self.d, self.f, self.E)
        down = moe.mx4_config(1, self.f, self.d, self.E)
        self._mx4 = moe.mx4_quantize_weights(up, self.W1), moe.mx4_quantize_weights(down, self.W2)
        return self

    def prefill(self, x, ws, mws):
        """ws: alloc_workspace(config(T), "scratch"); mws: alloc_mx4_workspace."""
        T = x.shape[0]
        c, nc, R = self.config(T), self.norms(T), T * self.k
        (w1, s1), (w2, s2) = self._mx4
        n = moe.block_norm(nc, x, w_pre=self.w_pre)["n"]
        idx, w, _ = moe.route(c, n, self.Wg, self.bias)
        lay = moe.dispatch(c, n, idx, ws=ws)
        off = lay["offsets"]
        up = moe.mx4_config(R, self.d, self.f, self.E, silu=1)
        down = moe.mx4_config(R, self.f, self.d, self.E, out_dtype="f32")
        q, s = moe.mx4_quantize_rows(up, lay["x_perm"], off, ws=mws)
        h = moe.mx4_product(up, q, s, w1, s1, off, ws=mws)
        q, s = moe.mx4_quantize_rows(down, h, off, ws=mws)
        y = moe.mx4_product(down, q, s, w2, s2, off, ws=mws)
        b = moe.combine(c, y, lay["pos"], w, ws=ws)
        r = moe.block_norm(nc, x, b, self.w_post, self.gate, self.w_next)
        return r["out"], r["n"]

    # ------------------------------------------------------------ training
    def train_step(self, x, dout, dnext):
        """Outputs and every gradient, given dout (of out, by the residual) and dnext (fp32,
        of the next block's input)."""
        T = x.shape[0]
        c, nc = self.config(T, keep_z=1), self.norms(T)
        ws, bws = moe.alloc_workspace(c), moe.alloc_workspace(c, "backward")
        nws = moe.alloc_norm_workspace(nc)
        pre = moe.block_norm(nc, x, w_pre=self.w_pre, want_rstd=True)
        b = moe.forward(c, pre["n"], self.Wg, self.bias, self.W1, self.W2, ws=ws)
        post = moe.block_norm(nc, x, b, self.w_post, self.gate, self.w_next, want_rstd=True)
        g = moe.block_norm_backward(nc, dout, dnext, post["out"], b, self.w_post, self.gate,
                                    self.w_next, post["rstd_post"], post["rstd_pre"], ws=nws)
        e = moe.backward(c, pre["n"], self.Wg, self.bias, self.W1, self.W2, g["db"], fwd_ws=ws,
                         ws=bws)
        first = moe.block_norm_backward(nc, g["dx"], e["dx"], x, None, None, None, self.w_pre,
                                        None, pre["rstd_pre"], ws=nws)
        grads = {"x": first["dx"], "w_pre": first["dw_pre"], "w_post": g["dw_post"],
                 "gate": g["dgate"], "w_next": g["dw_pre"], "Wg": e["dWg"], "bias": e["dbias"],
                 "W1": e["dW1"], "W2": e["dW2"]}
        return post["out"], post["n"], grads, (ws, bws)


def timed(name, f, reps=20):
    for _ in range(3):
        f()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(reps):
        f()
    b.record()
    torch.cuda.synchronize()
    print(f"{name:40s} {a.elapsed_time(b) / reps * 1e3:10.1f} us")


def main():
    ap = argparse.ArgumentParser()
    for name, v in (("d", 2048), ("f", 1408), ("E", 64), ("k", 2), ("tokens", 4096),
                    ("decode", 4)):
        ap.add_argument("--" + name, type=int, default=v)
    a = ap.parse_args()
    block = ExpertBlock(a.d, a.f, a.E, a.k).quantize()
    x = torch.randn((a.tokens, a.d), device="cuda").bfloat16()
    few = x[:a.decode].contiguous()
    fws = moe.alloc_workspace(block.config(a.decode), "few")
    sws = moe.alloc_workspace(block.config(a.tokens), "scratch")
    mws = moe.alloc_mx4_workspace(moe.mx4_config(1, a.d, a.f, a.E))
    timed(f"decode {a.decode} tokens", lambda: block.decode(few, fws))
    timed(f"prefill {a.tokens} tokens, 4-bit experts", lambda: block.prefill(x, sws, mws))
    dout, dnext = torch.randn_like(x), torch.randn((a.tokens, a.d), device="cuda")
    timed(f"train step, {a.tokens} tokens", lambda: block.train_step(x, dout, dnext), reps=3)
    for ws in (fws, sws, mws):
        if moe.get_device_error(ws) != moe.MOE_OK:
            raise SystemExit("device error")


if __name__ == "__main__":
    main()
