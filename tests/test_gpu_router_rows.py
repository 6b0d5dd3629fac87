"""Gradient of the router's losses on the GPU from the logits alone (the softmax of a row in 64 bits, not from what the losses
returned): rows far from zero or of the type's lowest value, where a sum's logarithm has no bits left beside the row's maximum; and
tokens that lie in no sequence."""
import numpy as np
import pytest
import torch

import block_scaled_moe_amd as moe
import router_ref as ref
from gpu_util import host

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
U24 = ref.U24


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def num(t):
    return host(t.float() if t.dtype == BF16 else t)


def slots(rng, T, E, k):
    return np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)


def gradient(logits, idx, valid, seq, k, db, dz):
    """d_logits of both losses and its bound, rows that do not count 0: softmax, sums and counts from the logits, in 64 bits."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    values, bounds, of, counted = ref.losses(logits, idx, valid, seq, k)
    with np.errstate(all="ignore"):
        l = np.where(counted[:, None], l, 0.0)  # whatever is in the other rows
        m = l.max(1)[:, None]
        ex = np.where(counted[:, None], np.exp(l - m), 0.0)
        total = np.where(counted, ex.sum(1), 1.0)[:, None]
        p = ex / total
        # an exponent is a difference rounded once; what the row's sum is off by
        e = np.where(p > 0, ref.exp_error(np.where(p > 0, l, m) - m - np.log(total)), 0.0)
        e_p = e + (p * e).sum(1, keepdims=True) + (ref.ADDS + 3) * U24
    n = np.maximum(values["tokens"], 1).astype(np.float64)
    a = ((db * E / (k * n * n))[:, None] * values["counts"])[of]
    lse = np.where(counted, values["lse"], 0.0)[:, None]
    b = (2 * dz / n)[of][:, None]
    dot, size = (p * a).sum(1, keepdims=True), (p * np.abs(a)).sum(1, keepdims=True)
    e_dot = (p * np.abs(a) * (e_p + 4 * U24)).sum(1, keepdims=True) + ref.ADDS * U24 * size
    d = p * (a - dot + b * lse)
    inner = np.abs(a) + np.abs(dot) + np.abs(b * lse)
    bound = p * ((e_p + 8 * U24) * inner + e_dot + np.abs(b) * np.where(counted, bounds["lse"], 0.0)[:, None])
    return np.where(counted[:, None], d, 0.0), np.where(counted[:, None], bound, 0.0) + 2 * U24 * np.abs(d) + 1e-37, of


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("E", [60, 61, 384, 700, 2100])
@pytest.mark.parametrize("balance,z", [(1.0, 0.0), (0.0, 1.0), (1.0, 0.01)])
def test_gradient_of_rows_far_from_zero(dtype, E, balance, z):
    rng = np.random.default_rng(E)
    offsets = np.repeat([0.0, 30.0, -1000.0, 1000.0, 5000.0, 3.0e4, 1.0e6, -1.0e8, 1.0e12], 5)
    T, k = len(offsets), 4
    x = rng.standard_normal((T, E)).astype(np.float32) * 2 + offsets[:, None].astype(np.float32)
    t, idx = dev(x, dtype), slots(rng, T, E, k)
    seq = [0, 20, T]
    db, dz = balance * rng.standard_normal(2).astype(np.float32), z * rng.standard_normal(2).astype(np.float32)
    l = moe.router_losses(t, dev(idx), seq=dev(np.array(seq, np.int32)))
    d = moe.logits_grad(t, dev(idx), l, dev(db) if balance else None, dev(dz) if z else None, out=torch.empty((T, E), device="cuda"))
    want, bound, _ = gradient(num(t), idx, None, seq, k, db.astype(np.float64), dz.astype(np.float64))
    ref.close(num(d), want, bound, "d_logits")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("low", ["min", -1e30])
def test_gradient_of_rows_of_the_lowest_value(dtype, low):
    """All experts masked by the same lowest value are as likely as each other; beside one finite value they are not likely at all."""
    rng = np.random.default_rng(2)
    T, E, k = 24, 70, 3
    x = np.full((T, E), torch.finfo(dtype).min if low == "min" else low, np.float32)
    x[8:16, ::2] = rng.standard_normal((8, 35))
    x[16:, 5] = 3.0
    t, idx = dev(x, dtype), slots(rng, T, E, k)
    db = np.array([0.7])
    l = moe.router_losses(t, dev(idx))
    d = moe.logits_grad(t, dev(idx), l, dev(db.astype(np.float32)))
    want, bound, _ = gradient(num(t), idx, None, None, k, db.astype(np.float32).astype(np.float64), np.zeros(1))
    ref.close(num(d), want, bound, "d_logits")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("z", [0.0, 1e-3])
def test_gradient_of_masked_and_extreme_logits(dtype, z):
    """Experts that may not be chosen, rows of nothing else, one finite value, large and lowest values, and anything in rows that do
    not count, with the gate's gradient."""
    rng = np.random.default_rng(4)
    T, E, k = 40, 70, 3
    x = rng.standard_normal((T, E)).astype(np.float32) * 2
    x[0] = -np.inf
    x[1, 1:] = -np.inf
    x[2, ::2] = -np.inf
    x[3] = 3.0e4
    x[4, 5] = 80.0
    x[5] = -1e30
    x[6] = -np.inf
    x[6, 69] = -1e30
    x[7, 3:] = -100.0
    x[8] += 5.0e3
    valid = np.ones(T, bool)
    valid[[10, 11, 12, 13]] = False
    x[10], x[11], x[12, 4], x[13] = np.nan, np.inf, np.nan, -np.inf
    t, idx = dev(x, dtype), slots(rng, T, E, k)
    w, dw = rng.random((T, k)).astype(np.float32), rng.standard_normal((T, k)).astype(np.float32)
    db, dz = rng.standard_normal(1).astype(np.float32), (z * rng.standard_normal(1)).astype(np.float32)
    l = moe.router_losses(t, dev(idx), valid=dev(valid))
    assert int(l.tokens[0]) == T - 5 and host(l.lse)[0] == -np.inf
    d = moe.logits_grad(t, dev(idx), l, dev(db), dev(dz) if z else None, dev(w), dev(dw))
    want, bound, _ = gradient(num(t), idx, valid, None, k, db.astype(np.float64), dz.astype(np.float64))
    gate, off = ref.logits_grad(num(t), idx, None, None, None, w, dw, None, k)
    ref.close(num(d), want + gate, bound + off + 2 * U24 * np.abs(want + gate), "d_logits")


@pytest.mark.parametrize("offset", [0.0, 1000.0, 3.0e4, -1e30])
def test_gradient_of_equal_counts_is_nothing(offset):
    """Where every expert has as many slots, a[e] is the same for all and the gradient of the balance is 0 but for roundings."""
    T, E, k = 96, 48, 4
    rng = np.random.default_rng(3)
    idx = (np.arange(T * k) % E).reshape(T, k).astype(np.int32)
    x = (rng.standard_normal((T, E)) + offset).astype(np.float32)
    l = moe.router_losses(dev(x), dev(idx))
    d = num(moe.logits_grad(dev(x), dev(idx), l, torch.ones(1, device="cuda")))
    _, bound, _ = gradient(x, idx, None, None, k, np.ones(1), np.zeros(1))
    assert (np.abs(d) <= bound).all() and np.abs(d).max() <= 500 * U24 / T


@pytest.mark.parametrize("E", [60, 384, 4095])
def test_log_sum_exp_is_rounded_once(E):
    """Half a step of the result, beside what the row's sum is off by (a relative error of the sum is one of its logarithm's value)."""
    rng = np.random.default_rng(E)
    x = (rng.standard_normal((400, E)) * 3 + rng.choice([0.0, -9.0, 40.0], (400, 1))).astype(np.float32)
    got = num(moe.router_losses(dev(x), dev(slots(rng, 400, E, 2))).lse).astype(np.float64)
    l = x.astype(np.float64)
    m = l.max(1, keepdims=True)
    ex = np.exp(l - m)
    want = m[:, 0] + np.log(ex.sum(1))
    # a lane's values, their exchanges; log(f) of f in 1/2 .. 1 is below one: a unit and a half of its last place at most
    off = (ex * ref.exp_error(l - m)).sum(1) / ex.sum(1) + ((E + 63) // 64 + 6) * U24 + 2 * U24
    assert (np.abs(got - want) <= off + U24 * np.exp2(np.ceil(np.log2(np.abs(want))))).all()


def poison(*shapes):
    """Leaves NaN in memory that the allocator will hand out next."""
    kept = [torch.full(s, float("nan"), device="cuda") for s in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del kept


OUTSIDE = {"both": (700, [90, 300, 300, 610]), "behind": (1000, [0, 400, 940]), "before": (300, [299, 300, 300]), "one": (200, [150, 190]),
           "one small": (14, [3, 9]), "one of none": (100, [40, 40]), "small of none": (12, [5, 5]), "none": (50, [0, 0, 0]), "end": (60, [60, 60, 60]),
           "many": (5000, sorted(np.random.default_rng(0).integers(700, 4200, 300).tolist())), "outside": (80, [-5, 20, 95]), "long": (70000, [33000, 33100, 66000])}


@pytest.mark.parametrize("name", OUTSIDE)
@pytest.mark.parametrize("E,dtype", [(60, FP32), (61, BF16), (384, FP32), (1100, FP32)])
@pytest.mark.parametrize("with_gate", [False, True])
def test_tokens_in_no_sequence(name, E, dtype, with_gate):
    """They count nowhere: lse is -inf, and their rows of a new gradient are the gate's alone, or zeros."""
    T, seq = OUTSIDE[name]
    k = 4
    rng = np.random.default_rng(T + E)
    x = rng.standard_normal((T, E)).astype(np.float32) * 2
    of = ref.sequence_of(seq, T)
    x[of < 0] = np.nan  # not looked at
    t, idx = dev(x, dtype), slots(rng, T, E, k)
    B = len(seq) - 1
    db, dz = rng.standard_normal(B).astype(np.float32), rng.standard_normal(B).astype(np.float32)
    w, dw = (rng.random((T, k)).astype(np.float32), rng.standard_normal((T, k)).astype(np.float32)) if with_gate else (None, None)
    opt = lambda a: None if a is None else dev(a)
    args = (t, dev(idx), dev(np.array(seq, np.int32)), dev(db), dev(dz), opt(w), opt(dw))
    poison((T,), (T, E), (4 * T + 64 * E,))
    l = moe.router_losses(args[0], args[1], seq=args[2])
    d = moe.logits_grad(args[0], args[1], l, *args[3:])
    values, bounds, _, _ = ref.losses(np.where(of[:, None] < 0, 0.0, num(t)), idx, None, seq, k)
    assert np.isneginf(host(l.lse)[of < 0]).all()
    ref.close(host(l.lse), values["lse"], np.where(of < 0, 0.0, bounds["lse"]), "lse")
    assert np.array_equal(host(l.counts), values["counts"]) and np.array_equal(host(l.tokens), values["tokens"])
    for n in ("balance", "z", "prob_sums"):
        ref.close(host(getattr(l, n)), values[n], bounds[n], n)
    want, bound, _ = gradient(np.where(of[:, None] < 0, 0.0, num(t)), idx, None, seq, k, db.astype(np.float64), dz.astype(np.float64))
    if with_gate:
        gate, off = ref.logits_grad(np.zeros((T, E)), idx, None, None, None, w, dw, None, k)
        want, bound = want + gate, bound + off + 2 * U24 * np.abs(want + gate)
    else:
        assert not host(d)[of < 0].any()
    ref.close(host(d), want, bound, "d_logits")
    kept = torch.full((T, E), 77.0, device="cuda")  # a given buffer keeps those rows
    assert moe.logits_grad(args[0], args[1], l, *args[3:], out=kept) is kept
    assert (host(kept)[of < 0] == 77.0).all() and torch.equal(kept[dev(of >= 0)], d[dev(of >= 0)])


def test_router_gradient_of_a_padded_batch():
    """router_losses, logits_grad, route_backward: padding before the first and behind the last sequence adds nothing."""
    rng = np.random.default_rng(9)
    T, E, D, k, seq = 300, 48, 128, 3, [20, 100, 250]
    h, wr = dev(rng.standard_normal((T, D)).astype(np.float32), BF16), dev(rng.standard_normal((E, D)).astype(np.float32), BF16)
    x, idx = dev(rng.standard_normal((T, E)).astype(np.float32)), dev(slots(rng, T, E, k))
    ones = torch.ones(2, device="cuda")
    poison((T,), (T, E), (4 * T + 16 * E,))
    l = moe.router_losses(x, idx, seq=dev(np.array(seq, np.int32)))
    d = moe.logits_grad(x, idx, l, ones, ones)
    dh, dwr, dbias = moe.route_backward(h, wr, d, dh_dtype=FP32, want_bias=True)
    d64 = num(d).astype(np.float64)
    assert not d64[:20].any() and not d64[250:].any() and not dh[:20].any() and not dh[250:].any()
    y, bound, _ = ref.product(np.ascontiguousarray(d64[20:250].T), num(h)[20:250].astype(np.float64), False, 3, 256)
    ref.close(num(dwr), y, bound, "dwr")
    assert np.isfinite(num(dbias)).all()


def test_sequences_that_move_between_calls():
    """The starts are read when the calls run: a token that left its sequence has no lse and no gradient of the losses any more."""
    rng = np.random.default_rng(10)
    T, E = 400, 64
    x, idx = dev(rng.standard_normal((T, E)).astype(np.float32)), dev(slots(rng, T, E, 2))
    seq = dev(np.array([0, 200, 400], np.int32))
    l, ones = moe.router_losses(x, idx, seq=seq), torch.ones(2, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.router_losses(x, idx, out=l)
        d = moe.logits_grad(x, idx, l, ones, ones)
    for starts in ([0, 200, 400], [100, 150, 300], [0, 0, 50], [390, 400, 400], [0, 399, 400]):
        seq.copy_(dev(np.array(starts, np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in (d, l.lse, l.balance, l.counts)]
        again = moe.router_losses(x, idx, seq=seq)
        eager = [moe.logits_grad(x, idx, again, ones, ones), again.lse, again.balance, again.counts]
        assert all(torch.equal(a, b) for a, b in zip(kept, eager)), starts
        assert bool(torch.isneginf(l.lse[:starts[0]]).all()) and bool(torch.isneginf(l.lse[starts[2]:]).all())
