"""Measured cases of three operators around the routed expert layer, with their
plain forms:

  few    the whole layer (gate, router, expert FFN, combine) for a few tokens
  norm   RMS norms before and after a block, fused with the block's gate and
         the residual scale, forward and backward
  mx4    microscaled 4-bit floating point (E2M1 elements, one power-of-two
         scale per 32 along the contraction): quantisation of rows and of
         expert weights, and the expert-grouped product of the two

`own` selects the plain form (False) or the framework's calls (True).
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def _moe():
    import mixture_experts_routed_gb300 as moe
    return moe


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, std=1.0, dtype=torch.float32):
    t = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if std != 1.0:
        t.mul_(std)
    return t.to(dtype)


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


# ------------------------------------------------------------------ the cases
def listed():
    few, norm, mx4 = {"op": "few"}, {"op": "norm"}, {"op": "mx4"}
    return [
        # one token of a decode step through the 64-expert layer: latency
        {**few, "name": "few_1_many_expert", "T": 1, "d": 2048, "E": 64, "k": 2, "f": 1408,
         "router": 1, "n_group": 1, "topk_group": 1},
        # one token through the fine-grained 256-expert layer: eight experts' weights
        {**few, "name": "few_1_fine_grained", "T": 1, "d": 7168, "E": 256, "k": 8, "f": 2048,
         "router": 0, "n_group": 1, "topk_group": 1},
        # a small odd decode batch over eight wide experts
        {**few, "name": "few_7_balanced", "T": 7, "d": 4096, "E": 8, "k": 2, "f": 11008,
         "router": 0, "n_group": 1, "topk_group": 1},
        # the largest few-token batch, group-limited, every expert active
        {**few, "name": "few_32_grouped", "T": 32, "d": 7168, "E": 32, "k": 8, "f": 2048,
         "router": 2, "n_group": 8, "topk_group": 4},
        # one token between two blocks of a decode step
        {**norm, "name": "norm_1_decode", "T": 1, "d": 7168, "dtype": "bf16", "gate": "token",
         "post": True, "pre": True, "train": False, "alpha": 1.0, "beta": 1.0},
        # a prefill batch between two blocks, per-channel branch scale
        {**norm, "name": "norm_prefill", "T": 16384, "d": 5120, "dtype": "bf16",
         "gate": "channel", "post": True, "pre": True, "train": False, "alpha": 1.0,
         "beta": 0.5},
        # a training step's norms, forward and backward, odd token count
        {**norm, "name": "norm_train", "T": 8191, "d": 7168, "dtype": "bf16", "gate": "token",
         "post": True, "pre": True, "train": True, "alpha": 0.75, "beta": 1.0},
        # the tiny fp32 layer's norms in training, one gate value per element
        {**norm, "name": "norm_train_f32", "T": 255, "d": 128, "dtype": "f32",
         "gate": "element", "post": True, "pre": True, "train": True, "alpha": 1.25,
         "beta": 1.0},
        # one token, two experts: reads two experts' 4-bit weights
        {**mx4, "name": "mx4_1_token", "what": "product", "R": 2, "K": 4096, "N": 11008, "E": 8,
         "zipf": 0.0, "out": "bf16"},
        # the up projection of a ragged many-expert batch, some experts empty
        {**mx4, "name": "mx4_ragged", "what": "product", "R": 2047, "K": 2048, "N": 1408,
         "E": 64, "zipf": 1.9, "out": "bf16"},
        # the up projection of a fine-grained skewed batch: the largest product
        {**mx4, "name": "mx4_skewed", "what": "product", "R": 16384, "K": 7168, "N": 2048,
         "E": 32, "zipf": 1.1, "out": "f32"},
        # expert weights into 4 bits and back
        {**mx4, "name": "mx4_weights", "what": "weights", "R": 1, "K": 1536, "N": 5120, "E": 16,
         "zipf": 0.0, "out": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["few", "norm", "mx4"])
    if op == "few":
        while True:
            c = {"op": "few", "T": _log_uniform(rng, 1, 32), "d": 64 * _log_uniform(rng, 2, 112),
                 "E": _log_uniform(rng, 2, 256), "f": 64 * _log_uniform(rng, 1, 172),
                 "router": rng.choice([0, 0, 1, 2]), "n_group": 1, "topk_group": 1}
            c["k"] = rng.randint(1, min(8, c["E"]))
            if c["router"] == 2:
                divs = [g for g in range(1, 33) if c["E"] % g == 0]
                c["n_group"] = rng.choice(divs)
                c["topk_group"] = rng.randint(1, c["n_group"])
                c["k"] = min(c["k"], c["topk_group"] * (c["E"] // c["n_group"]))
            if (c["E"] * c["d"] * c["f"] <= 3 << 30
                    and work(c)["bytes"] <= 32 * 7168 * 2048 * 4):
                return c
    if op == "norm":
        while True:
            c = {"op": "norm", "T": _log_uniform(rng, 1, 16384),
                 "d": 64 * _log_uniform(rng, 1, 160), "dtype": rng.choice(["bf16", "bf16", "f32"]),
                 "gate": rng.choice(["none", "token", "channel", "element"]),
                 "alpha": rng.choice([1.0, 0.5, 1.25]), "beta": rng.choice([1.0, 0.3]),
                 "train": rng.random() < 0.5}
            c["post"], c["pre"] = rng.choice([(True, True), (True, False), (False, True)])
            if work(c)["bytes"] <= 8191 * 7168 * 22:
                return c
    while True:
        c = {"op": "mx4", "what": rng.choice(["product"] * 4 + ["weights"]),
             "R": _log_uniform(rng, 1, 16384), "K": 64 * _log_uniform(rng, 1, 112),
             "N": 64 * _log_uniform(rng, 1, 172), "E": _log_uniform(rng, 1, 64),
             "zipf": rng.choice([0.0, 1.1, 1.9]), "out": rng.choice(["bf16", "f32"])}
        cap = 2 * 16384 * 7168 * 2048
        if (c["E"] * c["K"] * c["N"] <= 512 << 20 and 2 * c["R"] * c["K"] * c["N"] <= cap
                and (c["what"] == "product" or c["E"] * c["K"] * c["N"] <= 16 * 1536 * 5120)):
            return c


def _counts(c):
    """Rows per popularity rank: shares r^-zipf by largest remainder."""
    s = [(r + 1) ** -c["zipf"] for r in range(c["E"])]
    tot = sum(s)
    quota = [c["R"] * v / tot for v in s]
    n = [int(q) for q in quota]
    order = sorted(range(c["E"]), key=lambda i: (-(quota[i] - n[i]), i))
    for i in order[:c["R"] - sum(n)]:
        n[i] += 1
    return n


def work(c):
    if c["op"] == "few":
        T, d, E, k, f = (c[v] for v in ("T", "d", "E", "k", "f"))
        # experts that T tokens of k choices among E reach, uniform choices
        active = min(E, max(k, round(E * (1 - (1 - k / E) ** T))))
        return {"bytes": active * d * f * 4 + d * E * 2 + E * 4 + T * d * 4,
                "flops": 4 * T * k * d * f + 2 * T * d * E}
    if c["op"] == "norm":
        T, d, s = c["T"], c["d"], 2 if c["dtype"] == "bf16" else 4
        g = {"none": 0, "token": T * 4, "channel": d * 4, "element": T * d * s}[c["gate"]]
        post, pre = c["post"], c["pre"]
        by = T * d * s + pre * (T * d * s + d * 4) + post * (2 * T * d * s + d * 4 + g)
        fl = T * d * (4 * pre + 7 * post)
        if c["train"]:
            # dout in, dx out; dn (fp32) and the normed rows; b in, db out
            by += 2 * T * d * s + pre * (T * d * (4 + s) + 2 * d * 4)
            by += post * (2 * T * d * s + 2 * d * 4 + 2 * g)
            fl += T * d * (10 * pre + 14 * post)
        return {"bytes": by, "flops": fl}
    R, K, N, E = (c[v] for v in ("R", "K", "N", "E"))
    if c["what"] == "weights":
        # the weights in, their values out (the packed form stays inside)
        return {"bytes": E * K * N * 4, "flops": E * K * N * 4}
    active = sum(1 for v in _counts(c) if v)
    o = 2 if c["out"] == "bf16" else 4
    return {"bytes": R * K * 2 + active * N * (K // 2 + K // 32) + R * N * o + (E + 1) * 4,
            "flops": 2 * R * K * N}


# ------------------------------------------------------------------ the inputs
def _few_inputs(c, seed):
    g = _gen(seed)
    T, d, E, f = c["T"], c["d"], c["E"], c["f"]
    bf = torch.bfloat16
    x = _randn(g, (T, d), 1.0, bf)
    Wg = _randn(g, (d, E), d ** -0.5, bf)
    bias = _randn(g, (E,), 0.5 ** 0.5)
    W1 = torch.empty((E, d, f), dtype=bf, device=DEV)
    W2 = torch.empty((E, f, d), dtype=bf, device=DEV)
    for e in range(E):
        W1[e] = _randn(g, (d, f), d ** -0.5, bf)
        W2[e] = _randn(g, (f, d), f ** -0.5, bf)
    return {"x": x, "Wg": Wg, "bias": bias, "W1": W1, "W2": W2}


def _norm_inputs(c, seed):
    g = _gen(seed)
    T, d, dt = c["T"], c["d"], _dtype(c["dtype"])
    i = {"x": _randn(g, (T, d), 1.5, dt), "b": _randn(g, (T, d), 0.7, dt),
         "w_post": 1 + _randn(g, (d,), 0.2), "w_pre": 1 + _randn(g, (d,), 0.2)}
    shape = {"none": None, "token": (T,), "channel": (d,), "element": (T, d)}[c["gate"]]
    i["gate"] = None
    if shape is not None:
        v = torch.sigmoid(_randn(g, shape))
        i["gate"] = v.to(dt) if c["gate"] == "element" else v
    i["dout"] = _randn(g, (T, d), 1.0, dt)
    i["dn"] = _randn(g, (T, d), 1.0)
    if not c["post"]:
        i["b"] = i["w_post"] = i["gate"] = None
    if not c["pre"]:
        i["w_pre"] = i["dn"] = None
    return i


def _mx4_inputs(c, seed):
    g = _gen(seed)
    bf = torch.bfloat16
    R, K, N, E = (c[v] for v in ("R", "K", "N", "E"))
    W = torch.empty((E, K, N), dtype=bf, device=DEV)
    for e in range(E):
        W[e] = _randn(g, (K, N), K ** -0.5, bf)
    if c["what"] == "weights":
        return {"W": W}
    x = _randn(g, (R, K), 1.0, bf)
    # activations' outliers
    hit = torch.rand((R, K), generator=g, device=DEV) < 1e-3
    x = torch.where(hit, torch.sign(x.float()).to(bf) * 20, x)
    perm = torch.randperm(E, generator=g, device=DEV).tolist()
    n = _counts(c)
    offs = [0]
    for e in range(E):
        offs.append(offs[-1] + n[perm[e]])
    return {"W": W, "x": x, "offs": offs}


def prepare(case, seed):
    c = dict(case)
    st = {"c": c}
    if c["op"] == "few":
        st.update(_few_inputs(c, seed))
        if own:
            moe = _moe()
            st["cfg"] = moe.make_config(c["T"], c["d"], c["E"], c["k"], c["f"], "bf16",
                                        router=c["router"], pre_k=min(8, c["E"]),
                                        n_group=c["n_group"], topk_group=c["topk_group"])
            st["ws"] = moe.alloc_workspace(st["cfg"], "few")
        return st
    if c["op"] == "norm":
        st.update(_norm_inputs(c, seed))
        if own:
            moe = _moe()
            st["cfg"] = moe.norm_config(c["T"], c["d"], c["dtype"], gate=c["gate"], eps=EPS,
                                        alpha=c["alpha"], beta=c["beta"])
            st["ws"] = moe.alloc_norm_workspace(st["cfg"]) if c["train"] else None
        return st
    st.update(_mx4_inputs(c, seed))
    if c["what"] == "product":
        W = st.pop("W")
        st["offsets"] = torch.tensor(st["offs"], dtype=torch.int32, device=DEV)
        if own:
            moe = _moe()
            st["cfg"] = moe.mx4_config(c["R"], c["K"], c["N"], c["E"], out_dtype=c["out"])
            st["wq"], st["wsc"] = moe.mx4_quantize_weights(st["cfg"], W)
            st["ws"] = moe.alloc_mx4_workspace(st["cfg"])
        else:
            # one byte per element here: sign and magnitude code, and the exponents
            st["wq"] = torch.empty((c["E"], c["N"], c["K"]), dtype=torch.uint8, device=DEV)
            st["we"] = torch.empty((c["E"], c["N"], c["K"] // 32), dtype=torch.int8, device=DEV)
            for e in range(c["E"]):
                st["wq"][e], st["we"][e] = _mx4_codes(W[e].float().t())
    elif own:
        st["cfg"] = _moe().mx4_config(1, c["K"], c["N"], c["E"], out_dtype=c["out"])
    return st


# ------------------------------------------------------------------ plain forms
def _choose(c, L):
    """The chosen experts' ids [T, k] and weights of logits L (64 bits): larger
    logit first, the lower id on ties."""
    k = c["k"]
    if c["router"] == 2:
        p = torch.exp(L - L.max(1, keepdim=True).values)
        p = p.view(L.shape[0], c["n_group"], -1)
        order = torch.sort(p.sum(2), dim=1, descending=True, stable=True).indices
        keep = torch.zeros(p.shape[:2], dtype=torch.bool, device=L.device)
        keep.scatter_(1, order[:, :c["topk_group"]], True)
        L = torch.where(keep.unsqueeze(2).expand_as(p).reshape(L.shape), L,
                        torch.full_like(L, -math.inf))
    v, i = torch.sort(L, dim=1, descending=True, stable=True)
    n = min(8, c["E"]) if c["router"] == 1 else k
    ex = torch.exp(v[:, :n] - v[:, :1])
    return i[:, :k], ex[:, :k] / ex.sum(1, keepdim=True)


def _silu(z):
    return z / (1 + torch.exp(-z))


def _few_plain(st):
    c = st["c"]
    # the choice in 64 bits: logits next to one another decide experts
    idx, w = _choose(c, st["x"].double() @ st["Wg"].double() + st["bias"].double())
    x, w = st["x"].float(), w.float()
    T, k, E = c["T"], c["k"], c["E"]
    if E <= 2 * T * k:
        by = torch.zeros((T, E), device=DEV).scatter_(1, idx, w)
        out = torch.zeros_like(x)
        for e in range(E):
            out += by[:, e:e + 1] * (_silu(x @ st["W1"][e].float()) @ st["W2"][e].float())
    else:
        out = torch.zeros_like(x)
        for j in range(k):
            h = _silu(torch.bmm(x.unsqueeze(1), st["W1"][idx[:, j]].float()))
            out += w[:, j:j + 1] * torch.bmm(h, st["W2"][idx[:, j]].float()).squeeze(1)
    return out.to(torch.bfloat16)


def _norm_plain(st):
    c = st["c"]
    dt = _dtype(c["dtype"])
    d, al, be = c["d"], c["alpha"], c["beta"]
    res, y = {}, st["x"].float()
    if c["post"]:
        b = st["b"].float()
        rb = torch.rsqrt((b * b).mean(1, keepdim=True) + EPS)
        u = b * rb * st["w_post"]                 # the normed branch
        g = st["gate"]
        g = 1.0 if g is None else (g.unsqueeze(1) if c["gate"] == "token" else g.float())
        y = al * y + be * g * u
        res["out"] = y.to(dt)
    if c["pre"]:
        ry = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        res["n"] = (y * ry * st["w_pre"]).to(dt)
    if not c["train"]:
        return res
    D = st["dout"].float()
    if c["pre"]:
        yh, v = y * ry, st["dn"] * st["w_pre"]
        res["dw_pre"] = (st["dn"] * yh).double().sum(0).float()
        D = D + ry * (v - yh * (v * yh).mean(1, keepdim=True))
    res["dx"] = ((al if c["post"] else 1.0) * D).to(dt)
    if c["post"]:
        G = be * D
        bh = b * rb
        if c["gate"] == "token":
            res["dgate"] = (G * u).sum(1)
        elif c["gate"] == "channel":
            res["dgate"] = (G * u).double().sum(0).float()
        elif c["gate"] == "element":
            res["dgate"] = (G * u).to(dt)
        G = G * g
        res["dw_post"] = (G * bh).double().sum(0).float()
        v = G * st["w_post"]
        res["db"] = (rb * (v - bh * (v * bh).mean(1, keepdim=True))).to(dt)
    return res


def _mx4_codes(v):
    """fp32 [n, K] -> codes [n, K] (sign bit 3, magnitude code 0..7) and the
    blocks' exponents [n, K / 32]: 2^floor(log2 amax) / 4, 1 for a zero block."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(2)
    ex = torch.frexp(amax).exponent - 3
    ex = torch.where(amax == 0, torch.zeros_like(ex), ex.clamp(-127, 127))
    m = torch.ldexp(b.abs(), -ex.unsqueeze(2))
    lo, mid, hi = torch.round(m * 2), torch.round(m) + 2, torch.round(m / 2) + 4
    code = torch.where(m < 2, lo, torch.where(m < 4, mid, hi)).clamp(max=7).to(torch.uint8)
    code |= torch.signbit(b).to(torch.uint8) << 3
    return code.reshape(v.shape), ex.to(torch.int8)


def _mx4_values(code, ex):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    table = torch.cat([table, -table])
    v = table[code.int()].reshape(code.shape[0], -1, 32)
    return torch.ldexp(v, ex.int().unsqueeze(2)).reshape(code.shape)


def _mx4_plain(st):
    c = st["c"]
    if c["what"] == "weights":
        out = torch.empty_like(st["W"])
        for e in range(c["E"]):
            out[e] = _mx4_values(*_mx4_codes(st["W"][e].float().t())).t().to(torch.bfloat16)
        return out
    a = _mx4_values(*_mx4_codes(st["x"].float()))
    out = torch.empty((c["R"], c["N"]), dtype=_dtype(c["out"]), device=DEV)
    for e in range(c["E"]):
        lo, hi = st["offs"][e], st["offs"][e + 1]
        if hi > lo:
            out[lo:hi] = (a[lo:hi] @ _mx4_values(st["wq"][e], st["we"][e]).t()).to(out.dtype)
    return out


# ------------------------------------------------------------------ the framework's calls
def _few_own(st):
    return _moe().forward_few(st["cfg"], st["x"], st["Wg"], st["bias"], st["W1"], st["W2"],
                              ws=st["ws"])


def _norm_own(st):
    moe, c = _moe(), st["c"]
    r = moe.block_norm(st["cfg"], st["x"], st["b"], st["w_post"], st["gate"], st["w_pre"],
                       want_rstd=c["train"])
    res = {k: r[k] for k, on in (("out", c["post"]), ("n", c["pre"])) if on}
    if c["train"]:
        g = moe.block_norm_backward(st["cfg"], st["dout"], st["dn"],
                                    r["out"] if c["post"] else st["x"], st["b"], st["w_post"],
                                    st["gate"], st["w_pre"], r["rstd_post"], r["rstd_pre"],
                                    ws=st["ws"])
        res.update({k: v for k, v in g.items() if v is not None})
    return res


def _mx4_own(st):
    moe, c = _moe(), st["c"]
    if c["what"] == "weights":
        q, s = moe.mx4_quantize_weights(st["cfg"], st["W"])
        return moe.mx4_dequantize_weights(st["cfg"], q, s)
    q, s = moe.mx4_quantize_rows(st["cfg"], st["x"], st["offsets"], ws=st["ws"])
    return moe.mx4_product(st["cfg"], q, s, st["wq"], st["wsc"], st["offsets"], ws=st["ws"])


def run(state):
    op = state["c"]["op"]
    if own:
        return {"few": _few_own, "norm": _norm_own, "mx4": _mx4_own}[op](state)
    return {"few": _few_plain, "norm": _norm_plain, "mx4": _mx4_plain}[op](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _few_exact(c, i):
    x = i["x"].double()
    logits = x @ i["Wg"].double() + i["bias"].double()
    out = torch.zeros_like(x)
    for t in range(c["T"]):
        row = logits[t].tolist()
        ids = list(range(c["E"]))
        if c["router"] == 2:
            top, gs = max(row), c["E"] // c["n_group"]
            score = [sum(math.exp(v - top) for v in row[q * gs:(q + 1) * gs])
                     for q in range(c["n_group"])]
            best = sorted(range(c["n_group"]), key=lambda q: (-score[q], q))[:c["topk_group"]]
            ids = [e for e in ids if e // gs in best]
        ids.sort(key=lambda e: (-row[e], e))
        n = min(8, c["E"]) if c["router"] == 1 else c["k"]
        den = sum(math.exp(row[e] - row[ids[0]]) for e in ids[:n])
        for e in ids[:c["k"]]:
            z = x[t] @ i["W1"][e].double()
            h = z * torch.sigmoid(z)
            out[t] += math.exp(row[e] - row[ids[0]]) / den * (h @ i["W2"][e].double())
    return out


def _norm_exact(c, i):
    """The gradients by differentiating the forward in 64 bits."""
    t = {k: None if v is None else v.double() for k, v in i.items()}
    leaves = [k for k in ("x", "b", "w_post", "gate", "w_pre") if t[k] is not None]
    for k in leaves:
        t[k].requires_grad_(c["train"])

    def normed(v, w):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * w

    y, res = t["x"], {}
    if c["post"]:
        u = c["beta"] * normed(t["b"], t["w_post"])
        if t["gate"] is not None:
            u = u * (t["gate"][:, None] if c["gate"] == "token" else t["gate"])
        y = c["alpha"] * y + u
        res["out"] = y.detach()
    loss = (y * t["dout"]).sum()
    if c["pre"]:
        n = normed(y, t["w_pre"])
        res["n"] = n.detach()
        loss = loss + (n * t["dn"]).sum()
    if c["train"]:
        grads = dict(zip(leaves, torch.autograd.grad(loss, [t[k] for k in leaves])))
        for k, name in (("w_pre", "dw_pre"), ("x", "dx"), ("gate", "dgate"),
                        ("w_post", "dw_post"), ("b", "db")):
            if k in grads:
                res[name] = grads[k]
    return res


def _mx4_exact_values(v):
    """v [n, K] in 64 bits -> the values its 4-bit form stands for."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(2, keepdim=True)
    scale = torch.where(amax == 0, torch.ones_like(amax),
                        torch.exp2(torch.floor(torch.log2(amax)) - 2))
    m = b.abs() / scale
    code = torch.zeros_like(m, dtype=torch.int64)
    for i, border in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        # a tie goes to the even code
        code += (m >= border) if i % 2 else (m > border)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    return (torch.sign(b) * grid[code] * scale).reshape(v.shape)


def _mx4_exact(c, i):
    if c["what"] == "weights":
        return torch.stack([_mx4_exact_values(w.double().t()).t() for w in i["W"]])
    a = _mx4_exact_values(i["x"].double())
    out = torch.zeros((c["R"], c["N"]), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        lo, hi = i["offs"][e], i["offs"][e + 1]
        if hi > lo:
            out[lo:hi] = a[lo:hi] @ _mx4_exact_values(i["W"][e].double().t()).t()
    return out


def exact(case, seed):
    c = dict(case)
    if c["op"] == "few":
        return _few_exact(c, _few_inputs(c, seed))
    if c["op"] == "norm":
        return _norm_exact(c, _norm_inputs(c, seed))
    return _mx4_exact(c, _mx4_inputs(c, seed))
