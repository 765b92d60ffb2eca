"""Measured cases of three operators of a training step around the routed expert layer, with
their plain forms:

  fp8      expert products in 8-bit floating point (E4M3) with one power-of-two scale per
           block of 128: along a row for rows, 128 x 128 for weights, 128 rows of one expert
           for weight gradients; quantisation, the product, the gradient of its rows and of
           its weights
  balance  the router's balance loss, per sequence or over the batch, its z loss and the
           experts' counts, with the gradient of the logits
  dropout  dropout of a block's branch before the residual sum, its mask drawn from a
           counter-based generator (Philox 4x32, ten rounds) forward and backward

`own` selects the plain form (False) or the framework's calls (True).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF = torch.bfloat16


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
    return {"bf16": BF, "f32": torch.float32}[name]


# ------------------------------------------------------------------ the cases
def listed():
    fp8, bal, drop = {"op": "fp8"}, {"op": "balance"}, {"op": "dropout"}
    return [
        # two experts of a decode step: their weights are read, little else
        {**fp8, "name": "fp8_decode", "what": "product", "R": 2, "K": 4096, "N": 11008, "E": 8,
         "zipf": 0.0, "out": "bf16"},
        # the up projection of a ragged many-expert batch, some experts empty
        {**fp8, "name": "fp8_ragged", "what": "product", "R": 2047, "K": 2048, "N": 1408,
         "E": 64, "zipf": 1.9, "out": "bf16"},
        # the up projection of a fine-grained skewed batch
        {**fp8, "name": "fp8_skewed", "what": "product", "R": 16384, "K": 7168, "N": 2048,
         "E": 32, "zipf": 1.1, "out": "bf16"},
        # forward and both gradients of a projection, few wide experts: the largest
        {**fp8, "name": "fp8_train_wide", "what": "train", "R": 16384, "K": 5120, "N": 1536,
         "E": 16, "zipf": 0.0, "out": "bf16"},
        # the same of a ragged many-expert batch, rows' gradient in fp32
        {**fp8, "name": "fp8_train_ragged", "what": "train", "R": 8191, "K": 1408, "N": 2048,
         "E": 64, "zipf": 1.1, "out": "f32"},
        # expert weights into 8 bits and back
        {**fp8, "name": "fp8_weights", "what": "weights", "R": 1, "K": 1536, "N": 5120, "E": 16,
         "zipf": 0.0, "out": "bf16"},
        # the tiny layer's router
        {**bal, "name": "balance_tiny", "T": 256, "E": 8, "k": 2, "S": 1, "masked": False},
        # a padded batch of ragged sequences through the 64-expert layer
        {**bal, "name": "balance_sequences", "T": 8192, "E": 64, "k": 2, "S": 17, "masked": True},
        # a whole batch through the 256-expert layer: the largest
        {**bal, "name": "balance_fine_grained", "T": 16384, "E": 256, "k": 8, "S": 1,
         "masked": False},
        # the tiny fp32 layer's branch
        {**drop, "name": "dropout_tiny", "T": 256, "d": 128, "dtype": "f32", "p": 0.25,
         "residual": True},
        # a training batch's branch, with its residual
        {**drop, "name": "dropout_residual", "T": 16384, "d": 5120, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # the same without one, an odd number of rows
        {**drop, "name": "dropout_alone", "T": 8191, "d": 7168, "dtype": "bf16", "p": 0.5,
         "residual": False},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fp8", "fp8", "balance", "dropout"])
    if op == "balance":
        E = _log_uniform(rng, 1, 256)
        return {"op": op, "T": _log_uniform(rng, 1, 16384), "E": E,
                "k": rng.randint(1, min(8, E)), "S": _log_uniform(rng, 1, 64),
                "masked": rng.random() < 0.5}
    if op == "dropout":
        while True:
            c = {"op": op, "T": _log_uniform(rng, 1, 16384), "d": 64 * _log_uniform(rng, 1, 160),
                 "dtype": rng.choice(["bf16", "bf16", "f32"]),
                 "p": rng.choice([0.0, 0.1, 0.25, 0.5, 0.9]), "residual": rng.random() < 0.5}
            if c["T"] * c["d"] <= 16384 * 5120:
                return c
    while True:
        c = {"op": op, "what": rng.choice(["product", "product", "train", "train", "weights"]),
             "R": _log_uniform(rng, 1, 16384), "K": 64 * _log_uniform(rng, 1, 112),
             "N": 64 * _log_uniform(rng, 1, 172), "E": _log_uniform(rng, 1, 64),
             "zipf": rng.choice([0.0, 1.1, 1.9]), "out": rng.choice(["bf16", "f32"])}
        if (c["E"] * c["K"] * c["N"] <= 16 * 5120 * 1536
                and work(c)["flops"] <= 6 * 16384 * 5120 * 1536):
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
    if c["op"] == "balance":
        T, E, k, S = (c[v] for v in ("T", "E", "k", "S"))
        # logits in, their gradient out, the choices, one statistic a token, the counts
        return {"bytes": T * (8 * E + 4 * k + 4 + c["masked"]) + 4 * S * E,
                "flops": 12 * T * E}
    if c["op"] == "dropout":
        n, s = c["T"] * c["d"], 2 if c["dtype"] == "bf16" else 4
        # forward: the branch and the residual in, the sum out; backward: one in, one out
        return {"bytes": n * s * (4 + c["residual"]), "flops": n * (3 + c["residual"])}
    R, K, N, E = (c[v] for v in ("R", "K", "N", "E"))
    up = (-(-K // 128)) * (-(-N // 128))
    if c["what"] == "weights":
        # the weights in, their values out (the packed form stays inside)
        return {"bytes": E * K * N * 4, "flops": E * K * N * 4}
    active = sum(1 for v in _counts(c) if v)
    o = 2 if c["out"] == "bf16" else 4
    w = active * (K * N + up)
    if c["what"] == "product":
        return {"bytes": R * K * 2 + w + R * N * o + (E + 1) * 4, "flops": 2 * R * K * N}
    return {"bytes": 2 * R * (K + N) + w + R * (N + K) * o + E * K * N * 4 + (E + 1) * 4,
            "flops": 6 * R * K * N}


# ------------------------------------------------------------------ the inputs
def _spiky(g, shape):
    """bf16 activations: normal values and one large in a thousand."""
    v = _randn(g, shape)
    hit = torch.rand(shape, generator=g, device=DEV) < 1e-3
    return torch.where(hit, torch.sign(v) * 20, v).to(BF)


def _fp8_inputs(c, seed):
    g = _gen(seed)
    R, K, N, E = (c[v] for v in ("R", "K", "N", "E"))
    i = {"W": torch.empty((E, K, N), dtype=BF, device=DEV)}
    for e in range(E):
        i["W"][e] = _randn(g, (K, N), K ** -0.5, BF)
    if c["what"] == "weights":
        return i
    i["x"] = _spiky(g, (R, K))
    if c["what"] == "train":
        # gradients: small, and of another size in every row
        i["dy"] = (_spiky(g, (R, N)).float() *
                   torch.exp2(torch.randint(-12, -4, (R, 1), generator=g, device=DEV).float())
                   ).to(BF)
    perm = torch.randperm(E, generator=g, device=DEV).tolist()
    n = _counts(c)
    i["offs"] = [0]
    for e in range(E):
        i["offs"].append(i["offs"][-1] + n[perm[e]])
    return i


def _balance_inputs(c, seed):
    g = _gen(seed)
    T, E, k, S = (c[v] for v in ("T", "E", "k", "S"))
    # some experts are liked more than others
    logits = _randn(g, (T, E)) + _randn(g, (1, E), 0.5)
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    i = {"logits": logits, "idx": idx, "offsets": None, "mask": None,
         "dloss": torch.rand((1,), generator=g, device=DEV) + 0.5}
    if c["masked"] or S > 1:
        # sequences of any length, some of none; masked: the batch's end is padding, and one
        # token in sixteen inside it
        end = T - T // 8 if c["masked"] else T
        cut = torch.randint(0, end + 1, (S - 1,), generator=g, device=DEV)
        i["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV),
                                  torch.sort(cut).values,
                                  torch.full((1,), end, device=DEV)]).to(torch.int32)
    if c["masked"]:
        i["mask"] = (torch.rand((T,), generator=g, device=DEV) >= 1 / 16).to(torch.uint8)
    return i


def _dropout_inputs(c, seed):
    g = _gen(seed)
    T, d, dt = c["T"], c["d"], _dtype(c["dtype"])
    i = {"x": _randn(g, (T, d), 1.0, dt), "dout": _randn(g, (T, d), 1.0, dt), "residual": None,
         # what the generator is keyed by: a 64-bit seed and the step
         "state": torch.randint(0, 1 << 31, (2,), generator=g, device=DEV, dtype=torch.int64)}
    i["state"][0] *= 2654435761
    if c["residual"]:
        i["residual"] = _randn(g, (T, d), 2.0, dt)
    return i


BALANCE, Z = 0.01, 0.001  # the two losses' coefficients
SITE = 5                  # which of a model's dropouts this is


def prepare(case, seed):
    c = dict(case)
    st = {"c": c}
    moe = _moe() if own else None
    if c["op"] == "balance":
        st.update(_balance_inputs(c, seed))
        if own:
            st["cfg"] = moe.router_loss_config(c["T"], c["E"], c["k"], S=c["S"], balance=BALANCE,
                                               z=Z)
            st["ws"] = moe.alloc_router_loss_workspace(st["cfg"])
        return st
    if c["op"] == "dropout":
        st.update(_dropout_inputs(c, seed))
        if own:
            st["cfg"] = moe.dropout_config(c["T"], c["d"], c["dtype"], p=c["p"], site=SITE)
        return st
    st.update(_fp8_inputs(c, seed))
    if own:
        st["cfg"] = moe.fp8_config(c["R"], c["K"], c["N"], c["E"], out_dtype=c["out"])
    if c["what"] == "weights":
        return st
    W = st.pop("W")
    st["offsets"] = torch.tensor(st["offs"], dtype=torch.int32, device=DEV)
    if own:
        st["wq"], st["wsc"] = moe.fp8_quantize_weights(st["cfg"], W)
        st["ws"] = moe.alloc_fp8_workspace(st["cfg"])
    else:
        st["wq"] = torch.empty(W.shape, dtype=torch.float8_e4m3fn, device=DEV)
        st["we"] = []
        for e in range(c["E"]):
            st["wq"][e], ex = _weight_codes(W[e])
            st["we"].append(ex)
    return st


# ------------------------------------------------------------------ plain forms
def _exponent(amax):
    """The least e of at least -127 with amax <= 448 2^e (0 for amax = 0)."""
    f = torch.frexp(amax)
    e = f.exponent - 9 + (f.mantissa > 0.875).int()
    return torch.where(amax == 0, torch.zeros_like(e), e.clamp(min=-127))


def _padded(v, rows, cols):
    r, n = v.shape
    return torch.nn.functional.pad(v, (0, -n % cols, 0, -r % rows))


def _codes(v, rows, cols):
    """fp32 [r, n] in blocks of rows x cols -> (E4M3 codes [r, n], exponents of the blocks)."""
    r, n = v.shape
    b = _padded(v, rows, cols)
    b = b.view(b.shape[0] // rows, rows, b.shape[1] // cols, cols)
    e = _exponent(b.abs().amax(dim=(1, 3)))
    q = torch.ldexp(b, -e[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(b.shape[0] * rows, -1)[:r, :n], e


def _values(q, e, rows, cols):
    """What codes stand for, in fp32."""
    up = e.repeat_interleave(rows, 0).repeat_interleave(cols, 1)[:q.shape[0], :q.shape[1]]
    return torch.ldexp(q.float(), up)


def _weight_codes(w):
    return _codes(w.float(), 128, 128)


def _fp8_plain(st):
    c = st["c"]
    if c["what"] == "weights":
        out = torch.empty_like(st["W"])
        for e in range(c["E"]):
            out[e] = _values(*_weight_codes(st["W"][e]), 128, 128).to(BF)
        return out
    odt = _dtype(c["out"])
    train = c["what"] == "train"
    R, K, N, E = (c[v] for v in ("R", "K", "N", "E"))
    res = {"y": torch.empty((R, N), dtype=odt, device=DEV)}
    x = _values(*_codes(st["x"].float(), 1, 128), 1, 128)
    if train:
        res["dx"] = torch.empty((R, K), dtype=odt, device=DEV)
        res["dW"] = torch.zeros((E, K, N), device=DEV)
        dy = _values(*_codes(st["dy"].float(), 1, 128), 1, 128)
    for e in range(E):
        lo, hi = st["offs"][e], st["offs"][e + 1]
        if hi == lo:
            continue
        w = _values(st["wq"][e], st["we"][e], 128, 128)
        res["y"][lo:hi] = (x[lo:hi] @ w).to(odt)
        if train:
            res["dx"][lo:hi] = (dy[lo:hi] @ w.t()).to(odt)
            xc = _values(*_codes(st["x"][lo:hi].float(), 128, 1), 128, 1)
            dc = _values(*_codes(st["dy"][lo:hi].float(), 128, 1), 128, 1)
            res["dW"][e] = xc.t() @ dc
    return res


def _sequence_of(T, offsets):
    """Each token's sequence, -1 for the tokens of none."""
    if offsets is None:
        return torch.zeros((T,), dtype=torch.int64, device=DEV)
    t = torch.arange(T, device=DEV)
    s = torch.searchsorted(offsets.long(), t, right=True) - 1
    return torch.where((t >= offsets[0]) & (t < offsets[-1]), s, torch.full_like(s, -1))


def _balance_plain(st):
    c = st["c"]
    T, E, k, S = (c[v] for v in ("T", "E", "k", "S"))
    seq = _sequence_of(T, st["offsets"])
    on = seq >= 0
    if st["mask"] is not None:
        on = on & (st["mask"] != 0)
    # the tokens that count, one row of S flags each
    member = (seq[:, None] == torch.arange(S, device=DEV)) & on[:, None]
    n = member.sum(0)
    rows, used = n.sum(), (n > 0).sum()
    L = st["logits"]
    top = L.max(1, keepdim=True).values
    lse = (top + torch.log(torch.exp(L - top).sum(1, keepdim=True)))
    p = torch.exp(L - lse)
    chosen = torch.zeros((T, E), device=DEV).scatter_add_(1, st["idx"].long(),
                                                          torch.ones((T, k), device=DEV))
    m = member.double()
    counts = (m.t() @ chosen.double())
    per = n.clamp(min=1).double()[:, None]
    f = counts * E / (k * per)
    P = (m.t() @ p.double()) / per
    some, all_ = used.clamp(min=1).double(), rows.clamp(min=1).double()
    balance = (f * P).sum() / some
    z = (torch.where(on, lse[:, 0].double(), 0.0) ** 2).sum() / all_
    loss = torch.stack([BALANCE * balance + Z * z, balance, z]).float()
    ft = (m @ (f / per)).float() * (BALANCE / some).float()
    g = p * (ft - (p * ft).sum(1, keepdim=True)) + p * lse * (2 * Z / all_).float()
    g = torch.where(on[:, None], g * st["dloss"], torch.zeros_like(g))
    return {"loss": loss, "counts": counts.to(torch.int32), "dlogits": g}


_M0, _M1, _W0, _W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85
_LOW = 0xFFFFFFFF


def _mul32(a, m):
    """(high, low) 32 bits of a m, a in int64 below 2^32: 16 bits of a at a time."""
    t = (a >> 16) * m + ((a & 0xFFFF) * m >> 16)
    return t >> 16, (a * m) & _LOW


def _dropout_mask(c, state):
    """Truth values [T, d] that are kept, and the scale of those."""
    n = c["T"] * c["d"]
    thr = min(int(round(c["p"] * 65536)), 65535)
    g = torch.arange(n // 8, device=DEV)
    k0, k1 = state[0] & _LOW, (state[0] >> 32) & _LOW
    w = [g & _LOW, g >> 32, torch.full_like(g, SITE), (state[1] & _LOW).expand_as(g)]
    for r in range(10):
        h0, l0 = _mul32(w[0], _M0)
        h1, l1 = _mul32(w[2], _M1)
        w = [h1 ^ w[1] ^ ((k0 + r * _W0) & _LOW), l1, h0 ^ w[3] ^ ((k1 + r * _W1) & _LOW), l0]
    u = torch.stack([v for x in w for v in (x & 0xFFFF, x >> 16)], dim=1)
    return (u >= thr).view(c["T"], c["d"]), 65536 / (65536 - thr)


def _dropout_plain(st):
    c = st["c"]
    dt = _dtype(c["dtype"])
    keep, scale = _dropout_mask(c, st["state"])
    out = torch.where(keep, st["x"].float() * scale, 0.0)
    if c["residual"]:
        out = out + st["residual"].float()
    return {"out": out.to(dt),
            "dx": torch.where(keep, st["dout"].float() * scale, 0.0).to(dt)}


# ------------------------------------------------------------------ the framework's calls
def _fp8_own(st):
    moe, c, cfg = _moe(), st["c"], st["cfg"]
    if c["what"] == "weights":
        return moe.fp8_dequantize_weights(cfg, *moe.fp8_quantize_weights(cfg, st["W"]))
    off, ws = st["offsets"], st["ws"]
    if c["what"] == "product":
        rows = moe.fp8_quantize_rows(cfg, st["x"], off, ws=ws)
        return {"y": moe.fp8_product(cfg, rows, st["wq"], st["wsc"], off, ws=ws)}
    x = moe.fp8_quantize_rows(cfg, st["x"], off, ws=ws, columns=True)
    dy = moe.fp8_quantize_rows(cfg, st["dy"], off, ws=ws, columns=True)
    return {"y": moe.fp8_product(cfg, x, st["wq"], st["wsc"], off, ws=ws),
            "dx": moe.fp8_product(cfg, dy, st["wq"], st["wsc"], off, ws=ws, transposed=True),
            "dW": moe.fp8_weight_grad(cfg, x, dy, off, ws=ws)}


def _balance_own(st):
    moe, cfg = _moe(), st["cfg"]
    r = moe.router_loss(cfg, st["logits"], st["idx"], offsets=st["offsets"], mask=st["mask"],
                        ws=st["ws"])
    g = moe.router_loss_backward(cfg, st["logits"], r, dloss=st["dloss"],
                                 offsets=st["offsets"], mask=st["mask"])
    return {"loss": r.loss, "counts": r.counts, "dlogits": g}


def _dropout_own(st):
    moe, cfg = _moe(), st["cfg"]
    return {"out": moe.dropout(cfg, st["x"], st["state"], residual=st["residual"]),
            "dx": moe.dropout_backward(cfg, st["dout"], st["state"])}


def run(state):
    op = state["c"]["op"]
    if own:
        return {"fp8": _fp8_own, "balance": _balance_own, "dropout": _dropout_own}[op](state)
    return {"fp8": _fp8_plain, "balance": _balance_plain, "dropout": _dropout_plain}[op](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_values(v, along, size):
    """v in 64 bits -> what its 8-bit form stands for, blocks of `size` along each of the
    dimensions `along`."""
    amax = v.abs()
    for dim in along:
        n = amax.shape[dim]
        parts = [s.amax(dim, keepdim=True) for s in amax.split(size, dim)]
        amax = torch.cat(parts, dim).repeat_interleave(size, dim).narrow(dim, 0, n)
    scale = torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(min=-127))
    # (log2 near a whole number may land on either side of it)
    scale = torch.where(amax > 448 * scale, 2 * scale, scale)
    scale = torch.where((amax <= 224 * scale) & (scale > 2.0 ** -127), scale / 2, scale)
    scale = torch.where(amax == 0, torch.ones_like(scale), scale)
    m = v / scale
    # eight values to a power of two, down to 2^-6, then evenly: ties to the even one
    grid = torch.exp2(torch.floor(torch.log2(m.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(m / grid) * grid * scale


def _fp8_exact(c, i):
    if c["what"] == "weights":
        return torch.stack([_exact_values(w.double(), (0, 1), 128) for w in i["W"]])
    R, K, N, E = (c[v] for v in ("R", "K", "N", "E"))
    f64 = dict(dtype=torch.float64, device=DEV)
    x = _exact_values(i["x"].double(), (1,), 128)
    res = {"y": torch.zeros((R, N), **f64)}
    if c["what"] == "train":
        dy = _exact_values(i["dy"].double(), (1,), 128)
        res["dx"], res["dW"] = torch.zeros((R, K), **f64), torch.zeros((E, K, N), **f64)
    for e in range(E):
        rows = slice(i["offs"][e], i["offs"][e + 1])
        if rows.start == rows.stop:
            continue
        w = _exact_values(i["W"][e].double(), (0, 1), 128)
        res["y"][rows] = x[rows] @ w
        if c["what"] == "train":
            res["dx"][rows] = dy[rows] @ w.t()
            res["dW"][e] = (_exact_values(i["x"][rows].double(), (0,), 128).t()
                            @ _exact_values(i["dy"][rows].double(), (0,), 128))
    return res


def _balance_exact(c, i):
    """The gradient by differentiating the loss in 64 bits."""
    T, E, k, S = (c[v] for v in ("T", "E", "k", "S"))
    L = i["logits"].double().requires_grad_(True)
    offs = [0, T] if i["offsets"] is None else i["offsets"].tolist()
    balance, z, rows, used = 0.0, 0.0, 0, 0
    counts = torch.zeros((S, E), dtype=torch.float64, device=DEV)
    for s in range(S):
        t = torch.arange(offs[s], offs[s + 1], device=DEV)
        if i["mask"] is not None:
            t = t[i["mask"][t] != 0]
        if not len(t):
            continue
        counts[s] = torch.bincount(i["idx"][t].flatten().long(), minlength=E).double()
        balance = balance + (counts[s] * (E / (k * len(t)))
                             * torch.softmax(L[t], 1).mean(0)).sum()
        z = z + torch.logsumexp(L[t], 1).square().sum()
        rows, used = rows + len(t), used + 1
    if not rows:
        zero = torch.zeros((), dtype=torch.float64, device=DEV)
        return {"loss": torch.stack([zero] * 3), "counts": None, "dlogits": torch.zeros_like(L)}
    balance, z = balance / used, z / rows
    loss = BALANCE * balance + Z * z
    g, = torch.autograd.grad(loss * i["dloss"].double()[0], [L])
    return {"loss": torch.stack([loss, balance, z]).detach(), "counts": None, "dlogits": g}


def _dropout_exact(c, i):
    n = c["T"] * c["d"]
    seed, step = (int(v) & ((1 << 64) - 1) for v in i["state"].tolist())
    u64 = np.uint64
    low, half = u64(_LOW), u64(32)
    g = np.arange(n // 8, dtype=u64)
    x0, x1 = g & low, g >> half
    x2, x3 = np.full_like(g, SITE), np.full_like(g, step & _LOW)
    key = [seed & _LOW, seed >> 32]
    for _ in range(10):
        a, b = x0 * u64(0xD2511F53), x2 * u64(0xCD9E8D57)
        x0, x1, x2, x3 = ((b >> half) ^ x1 ^ u64(key[0]), b & low,
                          (a >> half) ^ x3 ^ u64(key[1]), a & low)
        key = [(key[0] + 0x9E3779B9) & _LOW, (key[1] + 0xBB67AE85) & _LOW]
    words = np.stack([x0, x1, x2, x3], axis=1).astype("<u4")
    # two 16-bit draws to a word, the lower first
    draws = words.view("<u2").reshape(c["T"], c["d"])
    thr = min(int(round(c["p"] * 65536)), 65535)
    keep = torch.from_numpy((draws >= thr).astype(np.float64)).to(DEV) * (65536 / (65536 - thr))
    out = i["x"].double() * keep
    if c["residual"]:
        out = out + i["residual"].double()
    return {"out": out, "dx": i["dout"].double() * keep}


def exact(case, seed):
    c = dict(case)
    if c["op"] == "balance":
        return _balance_exact(c, _balance_inputs(c, seed))
    if c["op"] == "dropout":
        return _dropout_exact(c, _dropout_inputs(c, seed))
    return _fp8_exact(c, _fp8_inputs(c, seed))
