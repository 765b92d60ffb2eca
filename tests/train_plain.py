"""Plain 64-bit forms of the training step's operators around the expert layer: 8-bit floating
point with a scale per block of 128, the router's losses, dropout's draws."""
import torch

F64 = torch.float64


# ---------------------------------------------------------------- 8 bits
def fp8_scales(v, rows, cols):
    """Scale bytes of the rows x cols blocks of v [r, c] in 64 bits."""
    r, c = v.shape
    nr, nc = -(-r // rows), -(-c // cols)
    pad = torch.zeros((nr * rows, nc * cols), dtype=F64, device=v.device)
    pad[:r, :c] = v.abs()
    amax = pad.view(nr, rows, nc, cols).amax(dim=(1, 3))
    # the least e with amax <= 448 2^e, from 2^e' <= amax / 256 < 2^(e' + 1)
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -200))) - 8
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= 448 * torch.exp2(e - 1), e - 1, e).clamp(min=-127)
    s = torch.where(amax == 0, torch.full_like(e, 127), e + 127)
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, 255)).to(torch.uint8)


def spread(s, rows, cols, shape):
    """Each element's scale byte."""
    return s.repeat_interleave(rows, 0).repeat_interleave(cols, 1)[:shape[0], :shape[1]]


def e4m3(m):
    """To the nearest E4M3 value, ties to the even one (|m| <= 448)."""
    step = torch.exp2(torch.floor(torch.log2(m.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(m / step) * step


def fp8_values(v, rows, cols):
    """(what v's 8-bit form stands for, its scale bytes); NaN in blocks of scale 255."""
    s = fp8_scales(v, rows, cols)
    b = spread(s, rows, cols, v.shape)
    scale = torch.exp2(b.to(F64) - 127)
    out = e4m3(torch.where(b == 255, torch.zeros_like(v), v) / scale) * scale
    return torch.where(b == 255, torch.full_like(out, float("nan")), out), s


def decode(q, s, rows, cols):
    """The values of code and scale bytes, as they lie in memory."""
    b = spread(s, rows, cols, q.shape)
    v = q.view(torch.float8_e4m3fn).to(F64) * torch.exp2(b.to(F64) - 127)
    return torch.where(b == 255, torch.full_like(v, float("nan")), v)


# ---------------------------------------------------------------- the router's losses
def router_loss(L, idx, k, offs, mask, balance, z):
    """(loss [3], counts [S, E], lse) of 64-bit logits, differentiable."""
    S, E = len(offs) - 1, L.shape[1]
    bal, zz, n, used = L.new_zeros(()), L.new_zeros(()), 0, 0
    counts = torch.zeros((S, E), dtype=torch.int64, device=L.device)
    for s in range(S):
        t = torch.arange(offs[s], offs[s + 1], device=L.device)
        if mask is not None:
            t = t[mask[t].bool()]
        if len(t) == 0:
            continue
        counts[s] = torch.bincount(idx[t].flatten().long(), minlength=E)
        f = E * counts[s].to(F64) / (k * len(t))
        bal = bal + (f * torch.softmax(L[t], 1).sum(0) / len(t)).sum()
        zz = zz + (torch.logsumexp(L[t], 1) ** 2).sum()
        n, used = n + len(t), used + 1
    bal, zz = bal / max(used, 1), zz / max(n, 1)
    return torch.stack([balance * bal + z * zz, bal, zz]), counts


def router_loss_gradient(L, idx, k, offs, mask, balance, z):
    """The formula's gradient of loss[0]."""
    S, E = len(offs) - 1, L.shape[1]
    g = torch.zeros_like(L)
    tokens = []
    for s in range(S):
        t = torch.arange(offs[s], offs[s + 1], device=L.device)
        tokens.append(t if mask is None else t[mask[t].bool()])
    n, used = sum(len(t) for t in tokens), sum(len(t) > 0 for t in tokens)
    for t in tokens:
        if len(t) == 0:
            continue
        p = torch.softmax(L[t], 1)
        f = E * torch.bincount(idx[t].flatten().long(), minlength=E).to(F64) / (k * len(t))
        g[t] = (balance / (used * len(t)) * p * (f - (p * f).sum(1, keepdim=True))
                + 2 * z / n * torch.logsumexp(L[t], 1, keepdim=True) * p)
    return g


# ---------------------------------------------------------------- dropout
def philox(c, key):
    """Philox 4x32, ten rounds, of Python integers."""
    c, key = list(c), list(key)
    low = (1 << 32) - 1
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ key[0], b & low, (a >> 32) ^ c[3] ^ key[1], a & low]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    return c


def dropout_keep(first, n, site, seed, step, p):
    """(kept, scale) of the elements [first, first + n)."""
    thr = min(int(p * 65536 + 0.5), 65535)
    low = (1 << 32) - 1
    seed &= (1 << 64) - 1
    keep, words, group = [], None, -1
    for i in range(first, first + n):
        if i // 8 != group:
            group = i // 8
            words = philox((group & low, group >> 32, site, step & low), (seed & low, seed >> 32))
        w = words[i % 8 // 2]
        keep.append(((w >> 16) if i & 1 else (w & 0xFFFF)) >= thr)
    return torch.tensor(keep), 65536 / (65536 - thr)
