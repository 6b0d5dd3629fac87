"""Cases of the token-grouping and block-scaled product operators (include/moe_ops.h), each with a
plain form in elementary torch operations.

kind "sort":          moe_sort, moe_gather and moe_combine: the tokens' rows grouped by expert, and the
                      experts' rows weighted and summed back per token.
kind "sort_grad":     the same pass followed by the gradients of both directions.
kind "product":       x quantised to E4M3 with a scale for each row's 128 values, multiplied with E4M3
                      expert weights holding a scale for each 128 x 128 block, grouped by expert.
kind "product_grad":  the gradients of that product: dy quantised by rows and by columns, x by columns,
                      the gradient of the input rows and the gradient of every expert's weight.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128


# ---------------------------------------------------------------- cases

def _sort(name, T, E, e0, e1, k, D, dtype, skew=0.0, pad=0.0, grad=False):
    return {"name": name, "kind": "sort_grad" if grad else "sort", "T": T, "E": E, "e0": e0, "e1": e1, "k": k, "D": D,
            "dtype": dtype, "skew": skew, "pad": pad}


def _product(name, T, E, e0, e1, k, N, K, skew=0.0, grad=False):
    return {"name": name, "kind": "product_grad" if grad else "product", "T": T, "E": E, "e0": e0, "e1": e1, "k": k,
            "N": N, "K": K, "skew": skew}


def listed():
    return [
        # one generated token through all 384 experts of a layer: launch latency
        _sort("sort one token", 1, 384, 0, 384, 8, 4096, "bf16"),
        # a decode batch, a quarter of it padding (no expert)
        _sort("sort decode batch", 64, 384, 0, 384, 8, 4096, "fp32", pad=0.25),
        # prefill on one of four expert-parallel ranks
        _sort("sort prefill share", 8192, 384, 0, 96, 8, 4096, "bf16"),
        # a training step of a small model, rows that end inside a 16-byte piece
        _sort("sort train odd", 517, 60, 0, 60, 3, 1001, "fp32", skew=1.0, grad=True),
        # a training step over a long batch with a few hot experts
        _sort("sort train", 16384, 384, 0, 384, 8, 4096, "bf16", skew=1.0, grad=True),
        # one generated token: the first matrix of its eight experts out of 64
        _product("product one token", 1, 64, 0, 64, 8, 5120, 4096),
        # a decode batch on one of four expert-parallel ranks
        _product("product decode share", 64, 384, 0, 96, 8, 5120, 4096),
        # prefill on one of four expert-parallel ranks
        _product("product prefill share", 8192, 384, 0, 96, 8, 5120, 4096),
        # the down matrix over a long skewed batch: groups of very different sizes
        _product("product skewed share", 16384, 384, 96, 192, 8, 4096, 2560, skew=1.0),
        # a dense projection (a single group) over an odd number of rows
        _product("product dense", 8191, 1, 0, 1, 1, 5120, 4096),
        # a training step of a tiny model
        _product("product train tiny", 300, 64, 0, 64, 8, 256, 128, grad=True),
        # a training step of the down matrix on one of four expert-parallel ranks
        _product("product train share", 8192, 384, 0, 96, 8, 4096, 2560, skew=0.5, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["sort", "sort_grad", "product", "product_grad"])
    k = rng.choice([1, 2, 3, 4, 6, 8])
    E = max(k, _log(rng, 1, 384))
    e0 = rng.randrange(E) if rng.random() < 0.4 else 0
    e1 = rng.randrange(e0 + 1, E + 1) if e0 else E
    skew = rng.choice([0.0, 0.5, 1.0])
    if kind.startswith("sort"):
        D = _log(rng, 32, 4096)
        if rng.random() < 0.7:
            D = max(64, D // 64 * 64)
        dtype = rng.choice(["bf16", "fp32"])
        T = _log(rng, 1, 16384 if dtype == "bf16" else 8192)
        return {"kind": kind, "T": T, "E": E, "e0": e0, "e1": e1, "k": k, "D": D, "dtype": dtype,
                "skew": skew, "pad": rng.choice([0.0, 0.1])}
    N, K = 128 * _log(rng, 1, 40), 128 * _log(rng, 1, 32)
    e1 = min(e1, e0 + 96)
    T = _log(rng, 1, 8192)
    if kind == "product_grad":
        N, K = 128 * _log(rng, 1, 32), 128 * _log(rng, 1, 20)
    k = min(k, max(1, 16384 // T))
    return {"kind": kind, "T": T, "E": E, "e0": e0, "e1": e1, "k": k, "N": N, "K": K, "skew": skew}


def _expected_slots(c):
    return int(c["T"] * c["k"] * (c["e1"] - c["e0"]) / c["E"] * (1 - c.get("pad", 0.0)) + 0.5)


def work(c):
    S, T, k = max(1, _expected_slots(c)), c["T"], c["k"]
    n = c["e1"] - c["e0"]
    used = n * (1 - (1 - 1 / n) ** S)  # experts that have rows, for an even routing
    order = 4 * (3 * T * k + n + 1)
    if c["kind"].startswith("sort"):
        es, D = (2 if c["dtype"] == "bf16" else 4), c["D"]
        fwd = order + 4 * T * k + (T * D + 2 * S * D + T * D) * es
        if c["kind"] == "sort":
            return {"bytes": fwd, "flops": 2 * S * D}
        return {"bytes": fwd + (2 * S * D + 2 * T * D) * es + 4 * T * k, "flops": 2 * S * D + S * D + 3 * S * D}
    N, K = c["N"], c["K"]
    scales = 4 * (N // BLOCK) * (K // BLOCK)
    if c["kind"] == "product":
        return {"bytes": order + 2 * min(S, T) * K + used * (N * K + scales) + 2 * S * N, "flops": 2 * S * N * K}
    return {"bytes": order + 2 * S * N + 2 * min(S, T) * K + used * (N * K + scales) + 2 * S * K + 2 * n * N * K,
            "flops": 4 * S * N * K}


# ---------------------------------------------------------------- inputs

def _routing(c, gen):
    """Distinct experts per token, [T, k] int32; `skew` makes low-numbered experts of a random order popular;
    a share `pad` of the tokens has no expert (-1)."""
    T, E, k = c["T"], c["E"], c["k"]
    bias = -c["skew"] * torch.log1p(torch.arange(E, device=DEV, dtype=torch.float32))
    bias = bias[torch.randperm(E, device=DEV, generator=gen)]
    noise = torch.rand((T, E), device=DEV, generator=gen).clamp_(1e-9, 1 - 1e-7)
    idx = (bias - torch.log(-torch.log(noise))).topk(k, dim=1).indices.to(torch.int32)
    if c.get("pad", 0.0):
        idx[torch.rand(T, device=DEV, generator=gen) < c["pad"]] = -1
    w = torch.softmax(torch.randn((T, k), device=DEV, generator=gen), dim=1)
    return idx, w


def _randn(shape, dtype, gen, sigma=1.0):
    return (torch.randn(shape, device=DEV, generator=gen) * sigma).to(dtype)


def _packed_weights(n, N, K, gen):
    """E4M3 expert weights as a checkpoint's loader lays them out once: codes [n, N/32, K/64, 4, 32, 16] (blocks of 32 rows
    and 64 columns, each block's four 16-column quarters apart), scales fp32 [n, N/128, K/128]."""
    codes = torch.empty((n, N // 32, K // 64, 4, 32, 16), dtype=torch.uint8, device=DEV)
    scales = torch.empty((n, N // BLOCK, K // BLOCK), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, n, step):
        m = min(step, n - e)
        w = torch.randn((m, N // BLOCK, BLOCK, K // BLOCK, BLOCK), device=DEV, generator=gen) * 0.02
        s = w.abs().amax((2, 4)) / 448.0
        q = (w / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[e:e + m] = q.view(m, N // 32, 32, K // 64, 4, 16).permute(0, 1, 3, 4, 2, 5)
        scales[e:e + m] = s
    return codes, scales


def prepare(case, seed):
    """Buffers of sorted rows have room for every slot; rows past the local slots keep what they hold, here zeros."""
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"c": c}
    T, k = c["T"], c["k"]
    if c["kind"] == "product" and c["E"] == 1:
        s["idx"], s["counts"] = None, [T]
    else:
        s["idx"], s["w"] = _routing(c, gen)
        local = s["idx"] - c["e0"]
        n = c["e1"] - c["e0"]
        local = torch.where((local >= 0) & (local < n), local, n)
        s["counts"] = torch.bincount(local.flatten(), minlength=n + 1)[:n].tolist()  # the host's own view of the batch
    S = s["S"] = sum(s["counts"])
    if c["kind"].startswith("sort"):
        dt, D = (torch.bfloat16 if c["dtype"] == "bf16" else torch.float32), c["D"]
        s["x"] = _randn((T, D), dt, gen)
        s["y"] = _randn((T * k, D), dt, gen)  # the experts' outputs, in sorted order
        s["rows"] = torch.zeros((T * k, D), dtype=dt, device=DEV)
        if c["kind"] == "sort_grad":
            s["dout"] = _randn((T, D), dt, gen)
            s["drows"] = _randn((T * k, D), dt, gen)
            s["dy"] = torch.zeros((T * k, D), dtype=dt, device=DEV)
        return s
    s["x"] = _randn((T, c["K"]), torch.bfloat16, gen)
    width = c["K"] if c["kind"] == "product_grad" else c["N"]
    s["out"] = torch.zeros((T * k, width), dtype=torch.bfloat16, device=DEV)
    s["codes"], s["scales"] = _packed_weights(c["e1"] - c["e0"], c["N"], c["K"], gen)
    if c["kind"] == "product_grad":
        s["dy"] = _randn((T * k, c["N"]), torch.bfloat16, gen, 0.1)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_order(s):
    """offsets, the local slots in sorted order (-1 behind them) and each slot's position (-1: not local)."""
    c = s["c"]
    n, S = c["e1"] - c["e0"], s["S"]
    e = s["idx"].flatten() - c["e0"]
    key = torch.where((e >= 0) & (e < n), e, n)
    sorted_key, order = torch.sort(key, stable=True)
    slots = order[:S]
    offsets = torch.searchsorted(sorted_key, torch.arange(n + 1, device=DEV, dtype=sorted_key.dtype))
    pos = torch.full((key.numel(),), -1, dtype=torch.int64, device=DEV)
    pos[slots] = torch.arange(S, device=DEV)
    return offsets, slots, pos


def _per_slot(rows, pos, c):
    """rows in slot order [T, k, D] in fp32, zero where the slot is not local."""
    if rows.shape[0] == 0:
        return torch.zeros((c["T"], c["k"], rows.shape[1]), device=DEV)
    got = rows[pos.clamp(min=0)].float() * (pos >= 0)[:, None]
    return got.view(c["T"], c["k"], -1)


def _plain_sort(s):
    c = s["c"]
    k, S = c["k"], s["S"]
    offsets, slots, pos = _plain_order(s)
    x, y, w = s["x"], s["y"][:S], s["w"]
    s["rows"][:S] = x[slots // k]
    per_slot = _per_slot(y, pos, c)
    out = (per_slot * w[:, :, None]).sum(1).to(x.dtype)
    sorted_slot = torch.full((c["T"] * k,), -1, dtype=torch.int32, device=DEV)
    sorted_slot[:S] = slots
    r = {"offsets": offsets.int(), "sorted_slot": sorted_slot, "slot_pos": pos.int().view(c["T"], k), "rows": s["rows"],
         "out": out}
    if c["kind"] == "sort_grad":
        dout = s["dout"].float()
        r["dx"] = _per_slot(s["drows"][:S], pos, c).sum(1).to(x.dtype)
        s["dy"][:S] = dout[slots // k] * w.flatten()[slots][:, None]
        r["dy"] = s["dy"]
        r["dw"] = (per_slot * dout[:, None, :]).sum(2)
    return r


def _e4m3(x, amax):
    """x at the nearest values that E4M3 codes with the scale amax / 448 hold."""
    # a division by a tensor: one by a number may be a product with its reciprocal, an ulp away
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    return (x / scale).to(torch.float8_e4m3fn).float() * scale


def _quantised_rows(x):
    b = x.float().view(x.shape[0], x.shape[1] // BLOCK, BLOCK)
    return _e4m3(b, b.abs().amax(2, keepdim=True)).view(x.shape)


def _quantised_columns(x, s, offsets):
    """x [S, C] with a scale for each column of each 128 rows of a group, counted from the group's first row."""
    counts = offsets[1:] - offsets[:-1]
    blocks = (counts + BLOCK - 1) // BLOCK
    first = torch.cumsum(blocks, 0) - blocks
    at = torch.arange(x.shape[0], device=DEV)
    e = torch.searchsorted(offsets[1:], at, right=True)
    at = first[e] * BLOCK + at - offsets[e]
    total = sum((n + BLOCK - 1) // BLOCK for n in s["counts"])
    b = torch.zeros((total * BLOCK, x.shape[1]), device=DEV)
    b[at] = x.float()
    b = b.view(total, BLOCK, x.shape[1])
    return _e4m3(b, b.abs().amax(1, keepdim=True)).view(total * BLOCK, x.shape[1])[at]


def _weights(s, chosen):
    """The experts `chosen` (an index) as fp32 [.., N, K]."""
    c = s["c"]
    N, K = c["N"], c["K"]
    q = s["codes"][chosen].view(torch.float8_e4m3fn).float()
    q = q.movedim(-2, -4).reshape(q.shape[:-5] + (N // BLOCK, BLOCK, K // BLOCK, BLOCK))
    return (q * s["scales"][chosen][..., :, None, :, None]).reshape(q.shape[:-4] + (N, K))


def _few(s):
    return s["S"] < 32 * len(s["counts"])


def _padded(s, offsets, rows, used):
    """rows of the groups `used`, each padded with zeros to the longest: [len(used), most, C]."""
    most = max(s["counts"])
    at = torch.arange(most, device=DEV)
    have = at[None, :] < (offsets[used + 1] - offsets[used])[:, None]
    at = torch.where(have, offsets[used][:, None] + at[None, :], 0)
    return rows[at] * have[:, :, None], at, have


def _plain_grouped(s, offsets, rows, transposed):
    """rows of each group times its expert's weights: one batched product over the experts that have rows when the groups
    are small, otherwise one product for each group."""
    c = s["c"]
    out = torch.empty((rows.shape[0], c["K"] if transposed else c["N"]), dtype=torch.float32, device=DEV)
    if _few(s):
        used = torch.tensor([e for e, n in enumerate(s["counts"]) if n], device=DEV)
        if len(used):
            w = _weights(s, used)
            x, at, have = _padded(s, offsets, rows, used)
            out[at[have]] = torch.bmm(x, w if transposed else w.transpose(1, 2).contiguous())[have]
        return out
    o = 0
    for e, n in enumerate(s["counts"]):
        if n:
            w = _weights(s, e)
            torch.mm(rows[o:o + n], w if transposed else w.t(), out=out[o:o + n])
            o += n
    return out


def _plain_product(s):
    c = s["c"]
    if s["idx"] is None:
        s["out"].copy_(_plain_grouped(s, None, _quantised_rows(s["x"]), False))
        return s["out"]
    offsets, slots, _ = _plain_order(s)
    s["out"][:s["S"]] = _plain_grouped(s, offsets, _quantised_rows(s["x"])[slots // c["k"]], False)
    return s["out"]


def _plain_product_grad(s):
    c, S = s["c"], s["S"]
    offsets, slots, _ = _plain_order(s)
    dy = s["dy"][:S]
    s["out"][:S] = _plain_grouped(s, offsets, _quantised_rows(dy), True)
    g = _quantised_columns(dy, s, offsets)
    x = _quantised_columns(s["x"][slots // c["k"]], s, offsets)
    if _few(s) and S:
        every = torch.arange(len(s["counts"]), device=DEV)
        gp, _, _ = _padded(s, offsets, g, every)
        xp, _, _ = _padded(s, offsets, x, every)
        dw = torch.bmm(gp.transpose(1, 2).contiguous(), xp).to(torch.bfloat16)
    else:
        dw = torch.zeros((len(s["counts"]), c["N"], c["K"]), dtype=torch.bfloat16, device=DEV)
        o = 0
        for e, n in enumerate(s["counts"]):
            if n:
                dw[e] = torch.mm(g[o:o + n].t(), x[o:o + n])
                o += n
    return {"dx": s["out"], "dw": dw}


# ---------------------------------------------------------------- the framework's operators

def _own(s):
    import block_scaled_moe_amd as moe
    c = s["c"]
    if s["idx"] is None:
        w = moe.BlockWeights(1, c["N"], c["K"], s["codes"], s["scales"])
        return moe.block_product(moe.quantize_block(s["x"]), w, out=s["out"])
    g = moe.sort_tokens(s["idx"], c["E"], c["e0"], c["e1"])
    if c["kind"].startswith("sort"):
        r = {"offsets": g.offsets, "sorted_slot": g.sorted_slot, "slot_pos": g.slot_pos}
        r["rows"] = moe.gather(g, s["x"], out=s["rows"])
        r["out"] = moe.combine(g, s["y"], s["w"], out_dtype=s["x"].dtype)
        if c["kind"] == "sort_grad":
            r["dx"] = moe.gather_backward(g, s["drows"])
            r["dy"], r["dw"] = moe.combine_backward(g, s["dout"], s["y"], s["w"], dy=s["dy"])
        return r
    w = moe.BlockWeights(c["e1"] - c["e0"], c["N"], c["K"], s["codes"], s["scales"])
    if c["kind"] == "product":
        return moe.block_product(moe.quantize_block(s["x"]), w, g, by_token=True, out=s["out"])
    dyq, dyc = moe.quantize_block_both(s["dy"], g)
    xc = moe.quantize_block_columns(s["x"], g, by_token=True)
    return {"dx": moe.block_product_grad(dyq, w, g, out=s["out"]), "dw": moe.block_weight_grad(dyc, xc, g)}


def run(s):
    if own:
        return _own(s)
    kind = s["c"]["kind"]
    if kind.startswith("sort"):
        return _plain_sort(s)
    return _plain_product(s) if kind == "product" else _plain_product_grad(s)


# ---------------------------------------------------------------- the definition in 64 bits

def _nearest_e4m3(v):
    """The nearest E4M3 value, ties to the even one: three mantissa bits from 2^-6 up, steps of 2^-9 below."""
    exponent = (torch.frexp(v)[1] - 1).clamp(min=-6)
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_quantised(x, dim):
    top = x.abs().amax(dim, keepdim=True)
    # the scale and the quotient are 32-bit numbers by definition
    scale = torch.where(top > 0, (top / 448.0).float().double(), torch.ones_like(top))
    return _nearest_e4m3((x / scale).float().double()) * scale


def _exact_groups(s):
    """For every expert, the slots that chose it, in ascending order."""
    c = s["c"]
    if s["idx"] is None:
        return [torch.arange(c["T"], device=DEV)]
    flat = s["idx"].flatten()
    return [torch.nonzero(flat == e).flatten() for e in range(c["e0"], c["e1"])]


def _exact_weight(s, e):
    c = s["c"]
    w = torch.empty((c["N"], c["K"]), dtype=torch.float64, device=DEV)
    blocks = s["codes"][e].view(torch.float8_e4m3fn).double()  # [N/32, K/64, 4, 32, 16]
    for quarter in range(4):
        piece = blocks[:, :, quarter].transpose(1, 2).reshape(c["N"], c["K"] // 64, 16)
        w.view(c["N"], c["K"] // 64, 64)[:, :, 16 * quarter:16 * quarter + 16] = piece
    return w * s["scales"][e].double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    k = c["k"]
    groups = _exact_groups(s)
    if c["kind"].startswith("sort"):
        slots = torch.cat(groups) if groups else torch.empty(0, dtype=torch.int64, device=DEV)
        tokens = slots // k
        w = s["w"].double().flatten()[slots]
        out = torch.zeros((c["T"], c["D"]), dtype=torch.float64, device=DEV)
        dx, dw = torch.zeros_like(out), torch.zeros(c["T"] * k, dtype=torch.float64, device=DEV)
        dy = torch.zeros((c["T"] * k if c["kind"] == "sort_grad" else 0, c["D"]), dtype=torch.float64, device=DEV)
        for a in range(0, len(slots), 16384):
            b = min(len(slots), a + 16384)
            y = s["y"][a:b].double()
            out.index_add_(0, tokens[a:b], y * w[a:b, None])
            if c["kind"] == "sort_grad":
                d = s["dout"][tokens[a:b]].double()
                dx.index_add_(0, tokens[a:b], s["drows"][a:b].double())
                dy[a:b] = d * w[a:b, None]
                dw[slots[a:b]] = (d * y).sum(1)
        rows = torch.zeros((c["T"] * k, c["D"]), dtype=torch.float64, device=DEV)
        rows[:len(slots)] = s["x"][tokens].double()
        r = {"offsets": None, "sorted_slot": None, "slot_pos": None, "rows": rows, "out": out}
        if c["kind"] == "sort_grad":
            r.update(dx=dx, dy=dy, dw=dw.view(c["T"], k))
        return r
    N, K = c["N"], c["K"]
    y = torch.zeros((c["T"] * k, K if c["kind"] == "product_grad" else N), dtype=torch.float64, device=DEV)
    dw = torch.zeros((len(groups), N, K), dtype=torch.float64, device=DEV) if c["kind"] == "product_grad" else None
    o = 0
    for e, slots in enumerate(groups):
        n = len(slots)
        if not n:
            continue
        x = s["x"][slots // k].double()
        if dw is None:
            q = _exact_quantised(x.view(n, K // BLOCK, BLOCK), 2).view(n, K)
            y[o:o + n] = q @ _exact_weight(s, e).t()
        else:
            g = s["dy"][o:o + n].double()
            q = _exact_quantised(g.view(n, N // BLOCK, BLOCK), 2).view(n, N)
            y[o:o + n] = q @ _exact_weight(s, e)
            for a in range(0, n, BLOCK):
                dw[e] += _exact_quantised(g[a:a + BLOCK], 0).t() @ _exact_quantised(x[a:a + BLOCK], 0)
        o += n
    return y if dw is None else {"dx": y, "dw": dw}
