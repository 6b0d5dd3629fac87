"""Plain 64-bit forms of the operators of include/moe_router.h, in numpy on the host, written from their definitions, with how
far the operators' fp32 results may be from them."""
from __future__ import annotations

import numpy as np

U24 = 2.0 ** -24   # half a step of fp32, relative
U_BF16 = 2.0 ** -8  # half a step of bf16, relative (its largest)
INF = np.inf


def starts(seq, T):
    return np.array([0, T]) if seq is None else np.clip(np.asarray(seq, np.int64), 0, T)


def sequence_of(seq, T):
    """Number of each token's sequence, -1 for none."""
    of = np.full(T, -1)
    s = starts(seq, T)
    for b in range(len(s) - 1):
        of[s[b]:s[b + 1]] = b
    return of


# Relative error of one exponential: two units of the last place from the function itself, and the argument l - m (or l - lse),
# a difference rounded once: off by U24 of its size.
def exp_error(x):
    return 4 * U24 + U24 * np.abs(np.where(np.isfinite(x), x, 0.0))


ADDS = 64 + 6 + 8  # additions of a row's sum at most: 64 values in a lane, six exchanges; of a run's: 64 rows, two exchanges, eight waves


def losses(logits, idx, valid, seq, k):
    """Every output of moe_router_losses and {name: bound}. logits are taken as given (fp32 or bf16 values)."""
    T, E = logits.shape
    l = np.asarray(logits, np.float64)
    of = sequence_of(seq, T)
    B = len(starts(seq, T)) - 1
    with np.errstate(all="ignore"):
        top = np.nanmax(np.where(np.isnan(l), -INF, l), axis=1)
        m = np.where(top == -INF, 0.0, top)
        x = l - m[:, None]
        ex = np.exp(x)
        total = ex.sum(1)
        counted = (of >= 0) & (total != 0) & (np.ones(T, bool) if valid is None else np.asarray(valid) != 0)
        lse = np.where(counted, m + np.log(total), -INF)
        p = np.where(counted[:, None], ex / total[:, None], 0.0)
        e_sum = (np.where(ex > 0, ex * exp_error(x), 0.0).sum(1) / total + ADDS * U24)      # of the total, relative
        e_lse = e_sum + 4 * U24 * (np.abs(np.log(total)) + 1) + 2 * U24 * np.abs(lse)
        e_p = p * (exp_error(x) + e_sum[:, None] + 3 * U24)
    counts = np.zeros((B, E), np.int64)
    sums, e_sums = np.zeros((B, E)), np.zeros((B, E))
    tokens = np.zeros(B, np.int64)
    z, balance, e_z, e_balance = (np.zeros(B) for _ in range(4))
    for b in range(B):
        t = np.nonzero(counted & (of == b))[0]
        n = tokens[b] = len(t)
        if n == 0:
            continue
        chosen = idx[t].reshape(-1).astype(np.int64)
        chosen = chosen[(chosen >= 0) & (chosen < E)]
        counts[b] = np.bincount(chosen, minlength=E)
        sums[b] = p[t].sum(0)
        e_sums[b] = e_p[t].sum(0) + ADDS * U24 * sums[b]
        with np.errstate(all="ignore"):
            z[b] = (lse[t] ** 2).mean()
            e_z[b] = (2 * np.abs(lse[t]) * e_lse[t]).mean() + (ADDS + 2) * U24 * z[b]
            balance[b] = (counts[b] * sums[b]).sum() * E / (k * n * n)
            e_balance[b] = (counts[b] * e_sums[b]).sum() * E / (k * n * n) + 2 * U24 * balance[b]
    return (dict(balance=balance, z=z, counts=counts, tokens=tokens, prob_sums=sums, lse=lse),
            dict(balance=e_balance, z=e_z, prob_sums=e_sums + U24 * sums, lse=e_lse), of, counted)


def logits_grad(logits, idx, got, d_balance, d_z, w, dw, seq, k):
    """d_logits and its bound, from the operator's own counts, tokens and lse (got, as numpy) or, with got None, of the gate
    alone. Rows of no sequence are NaN: not to be compared."""
    T, E = logits.shape
    d, bound = np.zeros((T, E)), np.zeros((T, E))
    if got is not None:
        of = sequence_of(seq, T)
        l, lse = np.asarray(logits, np.float64), np.asarray(got["lse"], np.float64)
        live = (of >= 0) & (lse != -INF)
        with np.errstate(all="ignore"):
            x = l - lse[:, None]
            p = np.where(live[:, None], np.exp(x), 0.0)
            e_p = exp_error(x)
            n = np.maximum(got["tokens"].astype(np.float64), 1)
            a = np.zeros((len(n), E)) if d_balance is None else (d_balance * E / (k * n * n))[:, None] * got["counts"]
            b = np.zeros(len(n)) if d_z is None else 2 * d_z / n
            a, b = a[of], (b[of] * lse)[:, None]
            pa = np.where(p > 0, p * np.abs(a), 0.0)
            dot = np.where(p > 0, p * a, 0.0).sum(1, keepdims=True)
            e_dot = np.where(p > 0, pa * (e_p + 3 * U24), 0.0).sum(1, keepdims=True) + ADDS * U24 * pa.sum(1, keepdims=True)
            inner = np.abs(a) + np.abs(dot) + np.abs(b)
            own = p * (a - dot + b)
            d[live], bound[live] = own[live], (p * ((e_p + 8 * U24) * inner + e_dot))[live]
        d[of < 0] = np.nan
    if w is not None:
        for t in range(T):
            if got is not None and of[t] < 0:
                continue
            here = [j for j in range(k) if 0 <= idx[t, j] < E]
            g = {j: float(w[t, j]) * (float(dw[t, j]) - sum(float(w[t, i]) * float(dw[t, i]) for i in here)) for j in here}
            size = {j: abs(float(w[t, j])) * (abs(float(dw[t, j])) + sum(abs(float(w[t, i]) * float(dw[t, i])) for i in here)) for j in here}
            for j in here:  # eight products and sums, a difference, a product, the sum over a token's equal slots
                d[t, idx[t, j]] += g[j]
                bound[t, idx[t, j]] += 24 * U24 * size[j]
    with np.errstate(all="ignore"):
        return d, bound + 2 * U24 * np.abs(d) + 1e-37  # exponentials below the normal numbers are cut off


def close(got, want, bound, what):
    """got within bound of want; NaN and infinities in the same places, where a value past fp32's largest (by half a step or
    more) is an infinity in fp32."""
    got, want, bound = np.asarray(got, np.float64), np.asarray(want, np.float64), np.broadcast_to(bound, np.shape(want))
    want = np.where(np.abs(want) >= 2.0 ** 128 * (1 - U24 / 2), np.copysign(INF, want), want)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    err = np.abs(got[fine] - want[fine])
    assert (err <= bound[fine]).all(), f"{what}: off by {err.max()}, at most {(err / np.maximum(bound[fine], 1e-300)).max()} of the bound"


def product(a, b, out_bf16, pieces, parts=1):
    """a @ b in 64 bits with the bound of one result and of the root mean square: a (fp32) is cut to `pieces` times 8 bits; the MFMA's
    sums are fp32, one step (2 U24, should it cut off) of a partial sum for each of the pieces' products."""
    y, size = a @ b, np.abs(a) @ np.abs(b)
    cut = 2.0 ** -15 if pieces == 2 else 0.0
    n = pieces * a.shape[1] + parts
    bound = (cut + n * 2 * U24) * size
    bound = bound + (U_BF16 * (np.abs(y) + bound) if out_bf16 else U24 * np.abs(y)) + 1e-37
    # signs in the mean: n roundings of partial sums no larger than a result, cuts of single products
    rms = np.sqrt((y ** 2).mean())
    size2 = np.sqrt((a ** 2 @ b ** 2).mean())
    mean = np.sqrt(n * (2 * U24 * rms) ** 2 + (cut * size2) ** 2 + ((U_BF16 if out_bf16 else U24) ** 2 / 3) * rms ** 2)
    return y, bound, 1.1 * mean
