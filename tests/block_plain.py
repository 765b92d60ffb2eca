"""Plain 64-bit forms of the operators around the expert layer, on the CPU, each with the sum
of absolute terms its rounding errors scale with."""
import torch

F64 = torch.float64
U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def norm_forward(x, b, w_post, gate, w_pre, kind, eps, alpha, beta):
    """dict of (value, absolute terms)."""
    r = {}
    y, ay = x, x.abs()
    if b is not None:
        rb = 1 / torch.sqrt((b * b).mean(1, keepdim=True) + eps)
        g = 1.0 if kind == "none" else (gate[:, None] if kind == "token" else gate)
        branch = beta * g * (b * rb * w_post)
        ay = (alpha * x).abs() + branch.abs()
        y = alpha * x + branch
        r["out"] = (y, ay)
        r["rstd_post"] = (rb[:, 0], rb[:, 0])
    if w_pre is not None:
        ro = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
        r["rstd_pre"] = (ro[:, 0], ro[:, 0])
        # a relative error e of rstd and the errors of y both reach n
        r["n"] = (y * ro * w_pre, (ay * ro * w_pre).abs()
                  + (y * ro * w_pre).abs() * (ay * ay).mean(1, keepdim=True) * ro * ro)
    return r


def norm_backward(dout, dn, y, b, w_post, gate, w_pre, rb, ro, kind, alpha, beta, ay=None):
    """Of (dx, db, dw_post, dgate, dw_pre): (value, absolute terms); rb, ro [T] as kept; ay: the
    absolute terms y is the sum of (its errors go by them)."""
    r = {}
    D, aD = dout, dout.abs()
    if w_pre is not None:
        yh, v = y * ro[:, None], dn * w_pre
        ah = (y.abs() if ay is None else ay) * ro[:, None]
        r["dw_pre"] = ((dn * yh).sum(0), (dn.abs() * ah).sum(0))
        D = D + ro[:, None] * (v - yh * (v * yh).mean(1, keepdim=True))
        aD = aD + ro[:, None] * (v.abs() + ah * (v.abs() * ah).mean(1, keepdim=True))
    if b is None:
        r["dx"] = (D, aD)
        return r
    r["dx"] = (alpha * D, abs(alpha) * aD)
    G, aG = beta * D, abs(beta) * aD
    bh = b * rb[:, None]
    u = bh * w_post
    if kind == "token":
        r["dgate"] = ((G * u).sum(1), (aG * u.abs()).sum(1))
    elif kind == "channel":
        r["dgate"] = ((G * u).sum(0), (aG * u.abs()).sum(0))
    elif kind == "element":
        r["dgate"] = (G * u, aG * u.abs())
    g = 1.0 if kind == "none" else (gate[:, None] if kind == "token" else gate)
    G = G * g
    aG = aG * abs(g)
    r["dw_post"] = ((G * bh).sum(0), (aG * bh.abs()).sum(0))
    v, av = G * w_post, aG * w_post.abs()
    r["db"] = (rb[:, None] * (v - bh * (v * bh).mean(1, keepdim=True)),
               rb[:, None] * (av + bh.abs() * (av * bh.abs()).mean(1, keepdim=True)))
    return r


def norm_problem(T, d, dtype, kind, post, pre, seed, device="cpu"):
    """Inputs of a norm call (fp32 draws on the CPU, rounded to dtype where the call takes it)."""
    g = torch.Generator().manual_seed(seed)

    def draw(*shape):
        return torch.randn(shape, generator=g)

    i = {"x": (1.5 * draw(T, d)).to(dtype), "b": (0.7 * draw(T, d)).to(dtype),
         "w_post": 1 + 0.2 * draw(d), "w_pre": 1 + 0.2 * draw(d), "gate": None,
         "dout": draw(T, d).to(dtype), "dn": draw(T, d)}
    if kind != "none":
        v = torch.sigmoid(draw(*{"token": (T,), "channel": (d,), "element": (T, d)}[kind]))
        i["gate"] = v.to(dtype) if kind == "element" else v
    if not post:
        i["b"] = i["w_post"] = i["gate"] = None
    if not pre:
        i["w_pre"] = i["dn"] = None
    return {k: None if v is None else v.to(device) for k, v in i.items()}


# ---------------------------------------------------------------- the layer for a few tokens
def choose(L, router, k, pre_k, n_group, topk_group, noise=None, tau=1.0):
    """ids [T, k] and weights of 64-bit logits, and each token's distance to another choice."""
    T, E = L.shape
    if router == 3:
        w = torch.softmax((L + noise) / tau, 1)
        return torch.arange(E, device=L.device).expand(T, E), w, torch.full((T,), 1.0)
    gap = torch.full((T,), float("inf"), dtype=F64, device=L.device)
    if router == 2:
        score = torch.softmax(L, 1).view(T, n_group, -1).sum(2)
        s, order = torch.sort(score, dim=1, descending=True, stable=True)
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, order[:, :topk_group], True)
        if topk_group < n_group:
            gap = (s[:, topk_group - 1] - s[:, topk_group]) / s[:, 0]
        L = L.masked_fill(~keep.repeat_interleave(E // n_group, 1), -float("inf"))
    v, i = torch.sort(L, dim=1, descending=True, stable=True)
    if k < E:
        gap = torch.minimum(gap, (v[:, k - 1] - v[:, k]).abs())
    if k > 1:
        gap = torch.minimum(gap, (v[:, :k - 1] - v[:, 1:k]).min(1).values)
    ex = torch.exp(v[:, :pre_k if router == 1 else k] - v[:, :1])
    return i[:, :k], ex[:, :k] / ex.sum(1, keepdim=True), gap.cpu()


def few_layer(c, i):
    """(out, its tolerance without the last rounding, gap) of the layer: c a config, i its
    inputs. Sums of n products on the tensor cores add 16 at a time in fp32: n / 8 + 64 half
    steps of the absolute terms cover the additions and the joining of partial sums; h is
    carried to 2^-17; the logits' errors reach the routing weights twice."""
    x = i["x"].to(F64)
    Wg = i["Wg"].to(F64)
    noise = i.get("gumbel")
    L = x @ Wg + i["bias"].to(F64)
    idx, w, gap = choose(L, c.router, c.k, c.pre_k, c.n_group, c.topk_group,
                         None if noise is None else noise.to(F64), c.tau)
    e_l = ((c.d / 64 + 128) * U32 * (x.abs() @ Wg.abs()).max(1).values / c.tau)[:, None]
    c1, c2 = (c.d / 8 + 64) * U32, (c.f / 8 + 64) * U32
    out, tol = torch.zeros_like(x), torch.zeros_like(x)
    for e in sorted(set(idx.flatten().tolist())):
        t, j = (idx == e).nonzero(as_tuple=True)
        W1, W2 = i["W1"][e].to(F64), i["W2"][e].to(F64)
        z = x[t] @ W1
        h = z * torch.sigmoid(z)
        dh = 1.1 * c1 * (x[t].abs() @ W1.abs()) + (2.0 ** -17 + 8 * U32) * h.abs()
        y, ya = h @ W2, h.abs() @ W2.abs()
        we = w[t, j][:, None]
        out[t] += we * y
        tol[t] += we * (c2 * ya + dh @ W2.abs() + (2 * e_l[t] + 64 * U32) * y.abs())
    return out, tol, gap


# ---------------------------------------------------------------- microscaled 4-bit values
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64)


def mx4_quantize(v):
    """[n, K] in 64 bits -> codes [n, K] and scale bytes [n, K / 32], by nearest grid value."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(2)
    fin = torch.isfinite(b).all(2)
    s = torch.frexp(torch.where(fin & (amax > 0), amax, torch.ones_like(amax))).exponent - 1 - 2
    s = s.clamp(min=-127) + 127
    s = torch.where(amax == 0, torch.full_like(s, 127), s)
    s = torch.where(fin, s, torch.full_like(s, 255))
    m = torch.where(fin[..., None], b.abs(), torch.zeros_like(b)) * torch.exp2(
        127.0 - s[..., None].to(F64))
    dist = (m.clamp(max=6.0)[..., None] - GRID.to(v.device)).abs()
    near = dist == dist.amin(-1, keepdim=True)
    # of two equally near codes the even one
    code = torch.arange(8, device=v.device)
    pick = torch.where(near, 8 * (code % 2) + code, torch.full_like(code, 99)).amin(-1) % 8
    pick = pick + 8 * torch.signbit(b).long()
    return pick.reshape(v.shape), s.to(torch.uint8)


def mx4_values(code, s):
    code = code.long()
    v = GRID.to(code.device)[code & 7] * (1 - 2 * (code >> 3))
    sc = torch.where(s == 255, torch.full(s.shape, float("nan"), dtype=F64, device=s.device),
                     torch.exp2(s.to(F64) - 127))
    return (v.reshape(code.shape[0], -1, 32) * sc[..., None]).reshape(code.shape)


def unpack_codes(q):
    """[..., K / 2] bytes -> [..., K] codes, the even k in the low half."""
    return torch.stack([q & 15, q >> 4], -1).flatten(-2)


def scales_of_tiles(scale, tiles, K):
    """Chunk bytes -> [tiles * 128, K / 32] scale bytes."""
    kc = -(-K // 128)
    c = scale[:tiles * kc * 512].reshape(tiles, kc, 32, 4, 4)   # i % 32, i / 32, block
    return c.permute(0, 3, 2, 1, 4).reshape(tiles * 128, kc * 4)[:, :K // 32]
