"""Cases of the router's training operators (include/moe_router.h) and of the product with 4-bit weights (include/moe_w4.h),
each with a plain form in elementary torch operations.

kind "loss":   the router's balance loss and z-loss of every sequence with the slots per expert, then the gradient of
               the logits from both losses and from the gate's weights.
kind "router": the gradients of the router's product: of the hidden states, of the router's weight and of its bias.
kind "w4":     rows times 4-bit expert weights with a scale (and perhaps a zero point) for each group of values, grouped by
               expert, with or without the SwiGLU of both halves of the result.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def _loss(name, T, E, k, B, dtype, masked=0.0, skew=0.5):
    return {"name": name, "kind": "loss", "T": T, "E": E, "k": k, "B": B, "dtype": dtype, "masked": masked, "skew": skew}


def _router(name, T, E, D, dtype, bias):
    return {"name": name, "kind": "router", "T": T, "E": E, "D": D, "dtype": dtype, "bias": bias}


def _w4(name, T, E, e0, e1, k, N, K, G, scale="bf16", zeros=False, swiglu=False, skew=0.0):
    return {"name": name, "kind": "w4", "T": T, "E": E, "e0": e0, "e1": e1, "k": k, "N": N, "K": K, "G": G, "scale": scale,
            "zeros": zeros, "swiglu": swiglu, "skew": skew}


def listed():
    return [
        # a training step of a tiny model: launch latency
        _loss("losses tiny", 48, 64, 8, 1, "fp32"),
        # short packed sequences of different lengths, a tenth of the tokens padding, rows that end inside a 16-byte piece
        _loss("losses packed odd", 5003, 61, 3, 17, "bf16", masked=0.1, skew=1.0),
        # a training step over a batch of sequences with a few hot experts
        _loss("losses train", 16384, 384, 8, 8, "fp32", skew=1.0),
        # the same layer over a long batch, balanced as a whole
        _loss("losses long batch", 131072, 384, 8, 1, "fp32"),
        # the router of a tiny model
        _router("router grad tiny", 300, 64, 256, "bf16", False),
        # fp32 gradients with the bias's, odd numbers of tokens and experts
        _router("router grad odd", 5003, 61, 1088, "fp32", True),
        # a training step over a long batch
        _router("router grad train", 16384, 384, 4096, "bf16", False),
        # one generated token: the down matrix of its eight experts out of 64
        _w4("w4 one token", 1, 64, 0, 64, 8, 4096, 2560, 128),
        # one generated token through a dense projection
        _w4("w4 one row", 1, 1, 0, 1, 1, 5120, 4096, 64, scale="fp16", zeros=True),
        # a decode batch on one of four expert-parallel ranks: gate and up matrix with the activation, fine groups
        _w4("w4 decode share", 64, 384, 0, 96, 8, 5120, 4096, 32, zeros=True, swiglu=True),
        # a batch with hot experts, sizes that end inside tiles
        _w4("w4 skewed odd", 1001, 60, 0, 60, 3, 1002, 2592, 32, scale="fp16", skew=1.0),
        # prefill on one of four expert-parallel ranks
        _w4("w4 prefill share", 4096, 384, 0, 96, 8, 5120, 4096, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["loss", "router", "w4"])
    k = rng.choice([1, 2, 3, 4, 6, 8])
    E = max(k, _log(rng, 1, 384))
    if kind == "loss":
        T = _log(rng, 1, 131072)
        return {"kind": kind, "T": T, "E": E, "k": k, "B": min(T, _log(rng, 1, 64)), "dtype": rng.choice(["bf16", "fp32"]),
                "masked": rng.choice([0.0, 0.1, 0.5]), "skew": rng.choice([0.0, 0.5, 1.0])}
    if kind == "router":
        return {"kind": kind, "T": _log(rng, 1, 16384), "E": E, "D": 64 * _log(rng, 1, 64),
                "dtype": rng.choice(["bf16", "fp32"]) if E * 3 <= 384 * 2 else "bf16", "bias": rng.random() < 0.5}
    G = rng.choice([32, 64, 128])
    swiglu = rng.random() < 0.4
    if rng.random() < 0.25:
        E = k = 1
    e0 = rng.randrange(E) if rng.random() < 0.4 else 0
    e1 = min(e0 + 96, rng.randrange(e0 + 1, E + 1) if e0 else E)
    T = _log(rng, 1, 2048)
    return {"kind": kind, "T": T, "E": E, "e0": e0, "e1": e1, "k": min(k, max(1, 8192 // T)), "N": 2 * _log(rng, 32, 2560),
            "K": G * _log(rng, 1, 4096 // G), "G": G, "scale": rng.choice(["bf16", "fp16"]), "zeros": rng.random() < 0.5,
            "swiglu": swiglu, "skew": rng.choice([0.0, 0.5, 1.0])}


def work(c):
    T, E = c["T"], c["E"]
    if c["kind"] == "loss":
        k, B, es = c["k"], c["B"], 2 if c["dtype"] == "bf16" else 4
        forward = T * E * es + 4 * T * k + T + 4 * T + B * (8 * E + 12)
        backward = T * E * (es + 4) + 12 * T * k + 4 * T + B * (4 * E + 12)
        return {"bytes": forward + backward, "flops": 20 * T * E}
    if c["kind"] == "router":
        D, es = c["D"], 2 if c["dtype"] == "bf16" else 4
        return {"bytes": (2 + es) * (T + E) * D + 4 * T * E + (4 * E if c["bias"] else 0), "flops": 4 * T * E * D}
    n, N, K, G = c["e1"] - c["e0"], c["N"], c["K"], c["G"]
    S = max(1, int(T * c["k"] * n / E + 0.5))
    used = n * (1 - (1 - 1 / n) ** S)  # experts that have rows, for an even routing
    weight = N * K // 2 + N * (K // G) * (3 if c["zeros"] else 2)
    out = 2 * S * (N // 2 if c["swiglu"] else N)
    return {"bytes": int(used * weight) + 2 * min(S, T) * K + out + 12 * T * c["k"], "flops": 2 * S * N * K}


# ---------------------------------------------------------------- inputs

def _randn(shape, dtype, gen, sigma=1.0):
    return (torch.randn(shape, device=DEV, generator=gen) * sigma).to(dtype)


def _logits(T, E, skew, gen):
    """Logits of a router with popular experts: `skew` raises low-numbered ones of a random order."""
    bias = -skew * torch.log1p(torch.arange(E, device=DEV, dtype=torch.float32))
    return torch.randn((T, E), device=DEV, generator=gen) * 1.5 + bias[torch.randperm(E, device=DEV, generator=gen)]


def _lengths(T, B, gen):
    """[B + 1] starts of B sequences over T tokens, some of them perhaps empty."""
    cut = torch.randint(0, T + 1, (B - 1,), device=DEV, generator=gen).sort().values
    return torch.cat([torch.zeros(1, device=DEV, dtype=torch.int64), cut, torch.full((1,), T, device=DEV)]).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"c": c}
    T, E = c["T"], c["E"]
    if c["kind"] == "loss":
        k, B = c["k"], c["B"]
        dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["logits"] = _logits(T, E, c["skew"], gen).to(dtype)
        top = s["logits"].float().topk(k, dim=1)
        s["idx"], s["w"] = top.indices.to(torch.int32), torch.softmax(top.values, dim=1)
        s["dw"] = _randn((T, k), torch.float32, gen, 1e-3)
        s["valid"] = None
        if c["masked"]:
            s["valid"] = torch.rand(T, device=DEV, generator=gen) >= c["masked"]
            s["idx"][~s["valid"]] = -1  # padding has no expert, and whatever in its row
            s["logits"][~s["valid"]] = float("nan")
        s["seq"] = _lengths(T, B, gen) if B > 1 else None
        s["d_balance"] = torch.rand(B, device=DEV, generator=gen) * 0.01 + 0.005
        s["d_z"] = torch.rand(B, device=DEV, generator=gen) * 0.001 + 0.0005
        return s
    if c["kind"] == "router":
        D = c["D"]
        s["h"], s["wr"] = _randn((T, D), torch.bfloat16, gen), _randn((E, D), torch.bfloat16, gen, 0.02)
        # what logits_grad returns: a dense part from the losses, larger values at the chosen experts
        g = _randn((T, E), torch.float32, gen, 1e-6)
        chosen = torch.randint(0, E, (T, min(8, E)), device=DEV, generator=gen)
        s["d_logits"] = g.scatter_add_(1, chosen, _randn(chosen.shape, torch.float32, gen, 1e-3))
        return s
    k, N, K, G, n = c["k"], c["N"], c["K"], c["G"], c["e1"] - c["e0"]
    if E == 1:
        s["idx"], s["counts"] = None, [T]
    else:
        s["idx"] = _logits(T, E, c["skew"], gen).topk(k, dim=1).indices.to(torch.int32)
        local = s["idx"] - c["e0"]
        local = torch.where((local >= 0) & (local < n), local, n)
        s["counts"] = torch.bincount(local.flatten(), minlength=n + 1)[:n].tolist()  # the host's own view of the batch
    s["S"] = sum(s["counts"])
    s["x"] = _randn((T, K), torch.bfloat16, gen)
    s["out"] = torch.zeros((T * k, N // 2 if c["swiglu"] else N), dtype=torch.bfloat16, device=DEV)
    # a checkpoint: codes of values 2 i and 2 i + 1 in a byte, the even one's in the low half
    s["codes"] = torch.randint(0, 256, (n, N, K // 2), device=DEV, generator=gen, dtype=torch.uint8)
    scale = torch.rand((n, N, K // G), device=DEV, generator=gen) * 0.004 + 0.002
    s["scales"] = scale.to(torch.bfloat16 if c["scale"] == "bf16" else torch.float16)
    s["zeros"] = None
    if c["zeros"]:
        s["zeros"] = torch.randint(4, 12, (n, N, K // G), device=DEV, generator=gen, dtype=torch.uint8)
    if own:  # laid out once, as a loader does
        import block_scaled_moe_amd as moe
        s["weights"] = moe.pack_w4(s["codes"], s["scales"], s["zeros"])
    return s


# ---------------------------------------------------------------- plain forms

def _sequence_of(seq, T):
    if seq is None:
        return torch.zeros(T, dtype=torch.int64, device=DEV)
    return torch.searchsorted(seq[1:].contiguous(), torch.arange(T, device=DEV, dtype=torch.int32), right=True)


def _plain_loss(s):
    c = s["c"]
    T, E, k, B = c["T"], c["E"], c["k"], c["B"]
    at = _sequence_of(s["seq"], T)
    counted = torch.ones(T, dtype=torch.bool, device=DEV) if s["valid"] is None else s["valid"]
    logits = torch.where(counted[:, None], s["logits"].float(), 0.0)
    top = logits.amax(1, keepdim=True)
    ex = torch.exp(logits - top)
    total = ex.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    p = ex / total * counted[:, None]
    of = at[None, :] == torch.arange(B, device=DEV)[:, None]  # [B, T]: the tokens of each sequence
    tokens = (of & counted).sum(1).to(torch.int32)
    slot = torch.where((s["idx"] >= 0) & (s["idx"] < E) & counted[:, None], s["idx"].long(), E) + at[:, None] * (E + 1)
    counts = torch.bincount(slot.flatten(), minlength=B * (E + 1)).view(B, E + 1)[:, :E].to(torch.int32).contiguous()
    # long sums in 64 bits
    sums = of.double() @ p.double()
    squares = of.double() @ torch.where(counted, lse, 0.0).double() ** 2
    m = tokens.clamp(min=1).double()
    balance = (counts * sums).sum(1) * E / (k * m * m)
    a = s["d_balance"][:, None] * counts * (E / (k * m * m)).float()[:, None]
    a, b = a[at], (2.0 * s["d_z"] / m.float())[at] * lse
    d = p * (a - (a * p).sum(1, keepdim=True)) + b[:, None] * p
    here = (s["idx"] >= 0) & (s["idx"] < E)
    w = s["w"] * here
    gate = w * (s["dw"] - (w * s["dw"]).sum(1, keepdim=True))
    d = d.scatter_add(1, torch.where(here, s["idx"].long(), 0), gate)
    lse = torch.where(counted, lse, -math.inf)
    return {"balance": balance.float(), "z": (squares / m).float(), "counts": counts, "tokens": tokens,
            "prob_sums": sums.float(), "lse": lse, "d_logits": d}


def _plain_router(s):
    c = s["c"]
    dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    g = s["d_logits"]
    r = {"dh": (g @ s["wr"].float()).to(dtype), "dwr": (g.t() @ s["h"].float()).to(dtype)}
    if c["bias"]:
        r["dbias"] = g.sum(0)
    return r


def _order(s):
    """The slots of every local expert, ascending, one expert after the other."""
    c = s["c"]
    n = c["e1"] - c["e0"]
    e = s["idx"].flatten() - c["e0"]
    return torch.sort(torch.where((e >= 0) & (e < n), e, n), stable=True)[1][:s["S"]]


def _dequantised(s, e):
    """Expert e's (or an index's) weights in fp32."""
    q = s["codes"][e]
    q = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2).float()
    q = q.view(q.shape[:-1] + (q.shape[-1] // s["c"]["G"], s["c"]["G"]))
    z = 8.0 if s["zeros"] is None else s["zeros"][e].float()[..., None]
    return ((q - z) * s["scales"][e].float()[..., None]).flatten(-2)


def _plain_w4(s):
    c = s["c"]
    rows = s["x"].float()
    if s["idx"] is not None:
        rows = rows[_order(s) // c["k"]]
    y = torch.empty((s["S"], c["N"]), device=DEV)
    used = [e for e, m in enumerate(s["counts"]) if m]
    if s["S"] < 32 * len(s["counts"]) and len(used) > 1:  # small groups, padded to the longest: one product for some experts at a time
        counts = torch.tensor(s["counts"], device=DEV)
        first = torch.cumsum(counts, 0) - counts
        at = torch.arange(max(s["counts"]), device=DEV)
        some = max(1, (1 << 28) // (c["N"] * c["K"]))
        for a in range(0, len(used), some):
            u = torch.tensor(used[a:a + some], device=DEV)
            have = at[None, :] < counts[u][:, None]
            place = torch.where(have, first[u][:, None] + at[None, :], 0)
            y[place[have]] = torch.bmm(rows[place] * have[:, :, None], _dequantised(s, u).transpose(1, 2).contiguous())[have]
    else:
        o = 0
        for e in used:
            m = s["counts"][e]
            y[o:o + m] = rows[o:o + m] @ _dequantised(s, e).t()
            o += m
    if c["swiglu"]:
        g, u = y[:, :c["N"] // 2], y[:, c["N"] // 2:]
        y = g / (1.0 + torch.exp(-g)) * u
    s["out"][:s["S"]] = y
    return s["out"]


# ---------------------------------------------------------------- the framework's operators

def _own(s):
    import block_scaled_moe_amd as moe
    c = s["c"]
    if c["kind"] == "loss":
        l = moe.router_losses(s["logits"], s["idx"], valid=s["valid"], seq=s["seq"])
        d = moe.logits_grad(s["logits"], s["idx"], losses=l, d_balance=s["d_balance"], d_z=s["d_z"], topk_w=s["w"],
                            d_topk_w=s["dw"])
        return {"balance": l.balance, "z": l.z, "counts": l.counts, "tokens": l.tokens, "prob_sums": l.prob_sums,
                "lse": l.lse, "d_logits": d}
    if c["kind"] == "router":
        dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        dh, dwr, dbias = moe.route_backward(s["h"], s["wr"], s["d_logits"], dh_dtype=dtype, dwr_dtype=dtype,
                                            want_bias=c["bias"])
        return {"dh": dh, "dwr": dwr, "dbias": dbias} if c["bias"] else {"dh": dh, "dwr": dwr}
    if s["idx"] is None:
        return moe.w4_product(s["x"], s["weights"], swiglu=c["swiglu"], out=s["out"])
    g = moe.sort_tokens(s["idx"], c["E"], c["e0"], c["e1"])
    return moe.w4_product(s["x"], s["weights"], g, by_token=True, swiglu=c["swiglu"], out=s["out"])


def run(s):
    if own:
        return _own(s)
    return {"loss": _plain_loss, "router": _plain_router, "w4": _plain_w4}[s["c"]["kind"]](s)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_loss(s):
    c = s["c"]
    T, E, k, B = c["T"], c["E"], c["k"], c["B"]
    starts = [0, T] if s["seq"] is None else s["seq"].tolist()
    valid = torch.ones(T, dtype=torch.bool, device=DEV) if s["valid"] is None else s["valid"]
    balance, z = (torch.zeros(B, dtype=torch.float64, device=DEV) for _ in range(2))
    sums = torch.zeros((B, E), dtype=torch.float64, device=DEV)
    lse = torch.full((T,), -math.inf, dtype=torch.float64, device=DEV)
    d = torch.zeros((T, E), dtype=torch.float64, device=DEV)
    for b in range(B):
        t = torch.arange(starts[b], starts[b + 1], device=DEV)
        t = t[valid[t]]
        m = len(t)
        if m == 0:
            continue
        l = s["logits"][t].double()
        lse[t] = torch.logsumexp(l, 1)
        p = torch.softmax(l, 1)
        sums[b] = p.sum(0)
        chosen = s["idx"][t].flatten()
        f = torch.bincount(chosen[(chosen >= 0) & (chosen < E)].long(), minlength=E).double() * E / (k * m)
        balance[b], z[b] = (f * sums[b]).sum() / m, (lse[t] ** 2).mean()
        d[t] = p * (f - (p * f).sum(1, keepdim=True)) * (s["d_balance"][b].double() / m)
        d[t] += p * (lse[t][:, None] * s["d_z"][b].double() * 2 / m)
    for j in range(k):  # the softmax over the chosen, one weight at a time
        here = (s["idx"][:, j] >= 0) & (s["idx"][:, j] < E)
        dots = sum(torch.where((s["idx"][:, i] >= 0) & (s["idx"][:, i] < E), s["w"][:, i].double() * s["dw"][:, i].double(), 0.0)
                   for i in range(k))
        t = here.nonzero()[:, 0]
        d[t, s["idx"][t, j].long()] += s["w"][t, j].double() * (s["dw"][t, j].double() - dots[t])
    return {"balance": balance, "z": z, "counts": None, "tokens": None, "prob_sums": sums, "lse": lse, "d_logits": d}


def _exact_w4(s):
    c = s["c"]
    k, G, out = c["k"], c["G"], torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    o = 0
    for e in range(c["e1"] - c["e0"]):
        rows = s["x"] if s["idx"] is None else s["x"][(s["idx"].flatten() == e + c["e0"]).nonzero()[:, 0] // k]
        if not len(rows):
            continue
        w = torch.empty((c["N"], c["K"]), dtype=torch.float64, device=DEV)
        w[:, 0::2], w[:, 1::2] = (s["codes"][e] % 16).double(), (s["codes"][e] // 16).double()
        z = torch.full_like(s["scales"][e], 8.0).double() if s["zeros"] is None else s["zeros"][e].double()
        w = (w - z.repeat_interleave(G, 1)) * s["scales"][e].double().repeat_interleave(G, 1)
        y = rows.double() @ w.t()
        if c["swiglu"]:
            g, u = y.chunk(2, dim=1)
            y = g * torch.sigmoid(g) * u
        out[o:o + len(rows)] = y
        o += len(rows)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["c"]["kind"] == "loss":
        return _exact_loss(s)
    if s["c"]["kind"] == "w4":
        return _exact_w4(s)
    g = s["d_logits"].double()
    dwr = torch.zeros(s["wr"].shape, dtype=torch.float64, device=DEV)
    dh = torch.empty(s["h"].shape, dtype=torch.float64, device=DEV)
    wr = s["wr"].double()
    for a in range(0, s["c"]["T"], 4096):
        dh[a:a + 4096] = g[a:a + 4096] @ wr
        dwr += g[a:a + 4096].t() @ s["h"][a:a + 4096].double()
    return {"dh": dh, "dwr": dwr, "dbias": g.sum(0)} if s["c"]["bias"] else {"dh": dh, "dwr": dwr}
