"""The expert half of a transformer block, run the ways it is used.

    n = norm(x) w_pre;   b = experts(n);   out = alpha x + beta g * (norm(b) w_post)

  decode   a few tokens: the block norms around the one-kernel layer (forward_few)
  prefill  many tokens, the experts' weights and rows in 4 bits (mx4_*)
  train    a step's forward and backward: block norms, forward with kept Z, backward
  train, 8-bit experts
           the same with the experts' products and their gradients in 8 bits (fp8_*), the
           router's balance loss (router_loss) and dropout of the block's output

The norm after one block and the norm before the next are one call, so a chain of blocks
costs one norm call a block.

    python examples/expert_block.py [--d 2048 --f 1408 --E 64 --k 2] [--tokens 4096] [--decode 4]
                                    [--dropout 0.1]
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
        """Outputs, every gradient and the workspaces that hold an error word (the norms' does
        not), given dout (of out, by the residual) and dnext (fp32, of the next block's input)."""
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

    def fp8_weights(self):
        """The experts' weights in 8 bits: made again after every update of theirs."""
        up = moe.fp8_config(1, self.d, self.f, self.E)
        down = moe.fp8_config(1, self.f, self.d, self.E)
        return moe.fp8_quantize_weights(up, self.W1), moe.fp8_quantize_weights(down, self.W2)

    def train_step_fp8(self, x, dout, dnext, state, p=0.1, balance=0.01, z_loss=0.001):
        """The same with the experts in 8 bits, dropout (state: int64 [2], seed and step) of
        their output and the router's losses, whose gradient joins the router's: outputs, the
        losses, every gradient, the workspaces with an error word."""
        T, d, f, E, k = x.shape[0], self.d, self.f, self.E, self.k
        R = T * k
        c, nc = self.config(T), self.norms(T)
        dc = moe.dropout_config(T, d, p=p)
        lc = moe.router_loss_config(T, E, k, balance=balance, z=z_loss)
        # each product's output where it is read next: a bf16 one by a quantiser, an fp32 one
        # by a sum over the experts
        up = moe.fp8_config(R, d, f, E, x_rows=T)
        down = moe.fp8_config(R, f, d, E, x_rows=T)
        up32 = moe.fp8_config(R, d, f, E, out_dtype="f32")
        down32 = moe.fp8_config(R, f, d, E, out_dtype="f32")
        ws, fws = moe.alloc_workspace(c, "scratch"), moe.alloc_fp8_workspace(up)
        nws, lws = moe.alloc_norm_workspace(nc), moe.alloc_router_loss_workspace(lc)
        (w1, s1), (w2, s2) = self.fp8_weights()

        pre = moe.block_norm(nc, x, w_pre=self.w_pre, want_rstd=True)
        n = pre["n"]
        idx, w, logits = moe.route(c, n, self.Wg, self.bias, want_logits=True)
        loss = moe.router_loss(lc, logits, idx, ws=lws)
        lay = moe.dispatch(c, n, idx, ws=ws)
        off, pos, src = lay["offsets"], lay["pos"], lay["src"]
        xq = moe.fp8_quantize_rows(up, n, off, ws=fws, src=src, columns=True)
        z = moe.fp8_product(up, xq, w1, s1, off, ws=fws)
        hq = moe.fp8_quantize_rows(down, z, off, ws=fws, act="silu", columns=True)
        y = moe.fp8_product(down32, hq, w2, s2, off, ws=fws)
        b = moe.dropout(dc, moe.combine(c, y, pos, w, ws=ws), state)
        post = moe.block_norm(nc, x, b, self.w_post, self.gate, self.w_next, want_rstd=True)

        g = moe.block_norm_backward(nc, dout, dnext, post["out"], b, self.w_post, self.gate,
                                    self.w_next, post["rstd_post"], post["rstd_pre"], ws=nws)
        db = moe.dropout_backward(dc, g["db"], state)
        # row r of the layout: its token's db times its routing weight
        wr = torch.empty(R, device=x.device).scatter_(0, pos.long(), w.flatten())
        dyq = moe.fp8_quantize_rows(down, db, off, ws=fws, src=src, row_weight=wr, columns=True)
        dh = moe.fp8_product(down, dyq, w2, s2, off, ws=fws, transposed=True)
        dzq = moe.fp8_quantize_rows(up, dh, off, ws=fws, act="silu_grad", z=z, columns=True)
        dxp = moe.fp8_product(up32, dzq, w1, s1, off, ws=fws, transposed=True)
        # the router: through the chosen experts' weights, and the losses' part
        dw = (db[:, None].float() * y[pos.view(T, k).long()]).sum(2)
        dL = moe.router_loss_backward(lc, logits, loss)
        dL.scatter_add_(1, idx.long(), w * (dw - (w * dw).sum(1, keepdim=True)))
        dn = dxp[pos.view(T, k).long()].sum(1) + dL @ self.Wg.float().t()
        first = moe.block_norm_backward(nc, g["dx"], dn, x, None, None, None, self.w_pre, None,
                                        pre["rstd_pre"], ws=nws)
        grads = {"x": first["dx"], "w_pre": first["dw_pre"], "w_post": g["dw_post"],
                 "gate": g["dgate"], "w_next": g["dw_pre"], "Wg": n.float().t() @ dL,
                 "bias": dL.sum(0), "W1": moe.fp8_weight_grad(up, xq, dzq, off, ws=fws),
                 "W2": moe.fp8_weight_grad(down, hq, dyq, off, ws=fws)}
        return post["out"], post["n"], loss, grads, (ws, fws, lws)


def timed(name, f, reps=20):
    """Prints a call's time; the last call's result."""
    for _ in range(3):
        f()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(reps):
        r = f()
    b.record()
    torch.cuda.synchronize()
    print(f"{name:40s} {a.elapsed_time(b) / reps * 1e3:10.1f} us")
    return r


def main():
    ap = argparse.ArgumentParser()
    for name, v in (("d", 2048), ("f", 1408), ("E", 64), ("k", 2), ("tokens", 4096),
                    ("decode", 4)):
        ap.add_argument("--" + name, type=int, default=v)
    ap.add_argument("--dropout", type=float, default=0.1)
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
    *_, step = timed(f"train step, {a.tokens} tokens", lambda: block.train_step(x, dout, dnext),
                     reps=3)
    state = torch.tensor([1, 0], dtype=torch.int64, device="cuda")
    *_, step8 = timed(f"train step, {a.tokens} tokens, 8-bit experts",
                      lambda: block.train_step_fp8(x, dout, dnext, state, p=a.dropout), reps=3)
    # every workspace with an error word; a training step makes its own and returns them
    for ws in (fws, sws, mws, *step, *step8):
        if moe.get_device_error(ws) != moe.MOE_OK:
            raise SystemExit("device error")


if __name__ == "__main__":
    main()
