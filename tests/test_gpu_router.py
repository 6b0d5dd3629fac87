"""The operators of include/moe_router.h on the GPU against plain forms in 64 bits (router_ref.py): the router's losses, the
gradients of its logits and of its product, at the sizes, masks and values where they can go wrong; gradients against
differences; a training step of them together; streams and graph replays."""
import numpy as np
import pytest
import torch

import block_scaled_moe_amd as moe
import router_ref as ref
from gpu_util import host

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def num(t):
    return host(t.float() if t.dtype == BF16 else t)


def routing(rng, T, E, k, kind="dup"):
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "wild":
        bad = rng.choice(np.array([-1, -7, E, E + 5, -2 ** 31, 2 ** 31 - 1], np.int64), (T, k)).astype(np.int32)
        idx = np.where(rng.random((T, k)) < 0.4, bad, idx)
    if kind == "one":
        idx[:] = E - 1
    if kind == "none":
        idx[:] = -1
    return idx


def gate(rng, T, k):
    w = rng.random((T, k)).astype(np.float32) + 0.1
    return w / w.sum(1, keepdims=True), rng.standard_normal((T, k)).astype(np.float32)


def check(logits, idx, valid=None, seq=None, seed=0, balance=True, z=True, with_gate=True, tail=True):
    """Losses and gradient of device logits against the reference; returns the losses."""
    T, E = logits.shape
    k = idx.shape[1]
    rng = np.random.default_rng(seed)
    l = moe.router_losses(logits, dev(idx), None if valid is None else dev(valid), None if seq is None else dev(np.asarray(seq, np.int32)),
                          out=None)
    got = {n: num(getattr(l, n)) for n in ("balance", "z", "counts", "tokens", "prob_sums", "lse")}
    want, bound, of, counted = ref.losses(num(logits), idx, valid, seq, k)
    assert np.array_equal(got["counts"], want["counts"]) and np.array_equal(got["tokens"], want["tokens"])
    for n in ("balance", "z", "prob_sums"):
        ref.close(got[n], want[n], bound[n], n)
    ref.close(got["lse"][of >= 0], want["lse"][of >= 0], bound["lse"][of >= 0], "lse")
    B = len(got["tokens"])
    db, dz = rng.standard_normal(B).astype(np.float32) if balance else None, rng.standard_normal(B).astype(np.float32) if z else None
    w, dw = gate(rng, T, k) if with_gate else (None, None)
    out = torch.full((T, E), 77.0, device="cuda")
    opt = lambda a: None if a is None else dev(a)
    d = moe.logits_grad(logits, dev(idx), l, opt(db), opt(dz), opt(w), opt(dw), out=out)
    assert d is out
    want_d, bound_d = ref.logits_grad(num(logits), idx, got, db, dz, w, dw, seq, k)
    inside = of >= 0
    ref.close(num(d)[inside], want_d[inside], bound_d[inside], "d_logits")
    assert (num(d)[~inside] == 77.0).all()
    return l


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 384, 8), (2, 64, 8), (31, 61, 3), (64, 8, 2), (65, 65, 1), (300, 128, 4), (129, 129, 5),
                                   (1000, 256, 8), (777, 257, 2), (2049, 384, 8), (515, 512, 6), (100, 513, 8), (333, 1024, 3),
                                   (70, 1026, 8), (40, 2048, 1), (37, 4095, 8), (9, 4096, 4)])
def test_losses_and_gradient(T, E, k, dtype):
    rng = np.random.default_rng(T * E)
    logits = dev(rng.standard_normal((T, E)).astype(np.float32) * 3, dtype)
    check(logits, routing(rng, T, E, k, "wild" if T % 2 else "dup"), seed=E)


@pytest.mark.parametrize("kind", ["dup", "wild", "one", "none"])
@pytest.mark.parametrize("balance,z,with_gate", [(True, True, True), (True, False, False), (False, True, True), (False, False, True), (True, True, False)])
def test_parts_of_the_gradient(kind, balance, z, with_gate):
    rng = np.random.default_rng(3)
    check(dev(rng.standard_normal((150, 62)).astype(np.float32)), routing(rng, 150, 62, 5, kind), balance=balance, z=z, with_gate=with_gate)


SEQS = {
    "even": (1000, [0, 250, 500, 750, 1000]), "ragged": (1000, [0, 1, 1, 3, 700, 701, 1000]), "empty": (60, [0, 0, 0, 60, 60]),
    "middle": (500, [100, 130, 400]), "none": (50, [0, 0, 0]), "ends": (90, [0, 90]), "singles": (70, list(range(71))),
    "many": (5000, sorted(np.random.default_rng(0).integers(0, 5001, 300).tolist())), "outside": (80, [-5, 20, 95]),
    "late": (300, [299, 300, 300]), "one late": (200, [150, 200]), "one of none": (100, [40, 40]),
}


@pytest.mark.parametrize("name", SEQS)
@pytest.mark.parametrize("E,dtype", [(60, FP32), (61, BF16), (384, FP32), (700, BF16)])
def test_packed_sequences(name, E, dtype):
    T, seq = SEQS[name]
    rng = np.random.default_rng(T + E)
    logits = dev(rng.standard_normal((T, E)).astype(np.float32) * 2, dtype)
    valid = (rng.random(T) < 0.8).astype(np.uint8) if T % 20 == 0 else None
    l = check(logits, routing(rng, T, E, 4, "wild"), valid=valid, seq=seq)
    assert l.balance.shape == (len(seq) - 1,)


def test_runs_of_a_long_batch():
    """Several runs a sequence, runs of more than one sweep, sequences that begin inside a run."""
    rng = np.random.default_rng(1)
    T, E = 40000, 24
    logits = dev(rng.standard_normal((T, E)).astype(np.float32))
    idx = routing(rng, T, E, 2)
    for seq in (None, [0, 17, 12345, 39999, 40000]):
        check(logits, idx, seq=seq, with_gate=False)
    l = moe.router_losses(logits, dev(idx))
    again = moe.router_losses(logits, dev(idx))
    assert all(torch.equal(getattr(l, n), getattr(again, n)) for n in ("balance", "z", "prob_sums", "lse", "counts"))


def test_even_routing_has_balance_one():
    """Logits all equal and every expert chosen equally often: exactly the value that the loss has at its least."""
    T, E, k = 96, 48, 4
    idx = (np.arange(T * k) % E).reshape(T, k).astype(np.int32)
    l = moe.router_losses(torch.zeros((T, E), device="cuda"), dev(idx))
    assert abs(float(l.balance[0]) - 1.0) <= 80 * ref.U24 and abs(float(l.z[0]) - np.log(E) ** 2) <= 1e-5
    assert (host(l.counts) == T * k // E).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_masked_and_extreme_logits(dtype):
    """-inf for experts that may not be chosen, rows of nothing else, the type's lowest value, a single finite value, large
    values, NaN and infinities in rows that do not count."""
    rng = np.random.default_rng(4)
    T, E = 40, 70
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
    x[10], x[11], x[12, 4] = np.nan, np.inf, np.nan
    x[13] = -np.inf
    t = dev(x, dtype)
    idx = routing(rng, T, E, 3)
    l = check(t, idx, valid=valid, z=False)
    assert int(l.tokens[0]) == T - 5 and host(l.lse)[0] == -np.inf
    lowest = torch.full((3, E), torch.finfo(dtype).min, device="cuda", dtype=dtype)
    l = moe.router_losses(lowest, dev(idx[:3]))
    assert torch.allclose(l.prob_sums, torch.full((1, E), 3 / E, device="cuda"), rtol=1e-5) and torch.isinf(l.z).all()
    d = moe.logits_grad(lowest, dev(idx[:3]), l, d_balance=torch.ones(1, device="cuda"))
    assert torch.isfinite(d).all()


def test_all_rows_masked():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((30, 20)).astype(np.float32)
    l = check(dev(x), routing(rng, 30, 20, 2), valid=np.zeros(30, np.uint8))
    assert not l.balance.any() and not l.z.any() and not l.prob_sums.any() and torch.isneginf(l.lse).all()


def test_non_finite_values_stay_in_their_sequence():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((100, 33)).astype(np.float32)
    seq, idx = [0, 40, 60, 100], routing(rng, 100, 33, 3)
    clean = moe.router_losses(dev(x), dev(idx), seq=dev(np.array(seq, np.int32)))
    ones = torch.ones(3, device="cuda")
    g0 = moe.logits_grad(dev(x), dev(idx), clean, ones, ones)
    for bad in (np.nan, np.inf):
        y = x.copy()
        y[50, 7] = bad
        l = moe.router_losses(dev(y), dev(idx), seq=dev(np.array(seq, np.int32)))
        for n in ("balance", "z", "prob_sums"):
            a, b = getattr(l, n), getattr(clean, n)
            assert torch.equal(a[[0, 2]], b[[0, 2]]) and not torch.isfinite(a[1]).any()
        assert int(l.tokens[1]) == 20
        g = moe.logits_grad(dev(y), dev(idx), l, ones, ones)
        other = [t for t in range(100) if t != 50]
        assert torch.equal(g[other], g0[other]) and torch.isnan(g[50]).any()


def test_no_tokens():
    logits, idx = torch.empty((0, 16), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    for seq in (None, torch.zeros(4, dtype=torch.int32, device="cuda")):
        l = moe.router_losses(logits, idx, seq=seq)
        assert not l.balance.any() and not l.z.any() and not l.counts.any() and not l.tokens.any() and not l.prob_sums.any()
        assert moe.logits_grad(logits, idx, l, torch.ones_like(l.balance)).shape == (0, 16)


def test_gradient_against_differences():
    """The gradient of the two losses (with the counts held) by central differences in 64 bits, and of the gate's weights as
    the softmax over the chosen logits."""
    rng = np.random.default_rng(7)
    T, E, k = 12, 10, 3
    x = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.argsort(-x, axis=1)[:, :k].astype(np.int32)
    seq = [0, 5, 12]
    l = moe.router_losses(dev(x), dev(idx), seq=dev(np.array(seq, np.int32)))
    db, dz = np.array([0.7, -1.3], np.float32), np.array([0.2, 0.4], np.float32)
    top = np.take_along_axis(x, idx.astype(np.int64), 1)
    w = np.exp(top - top.max(1, keepdims=True))
    w = (w / w.sum(1, keepdims=True)).astype(np.float32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    g = num(moe.logits_grad(dev(x), dev(idx), l, dev(db), dev(dz), dev(w), dev(dw)))
    counts = host(l.counts).astype(np.float64)

    def f(v):
        total = 0.0
        for b in range(2):
            r = v[seq[b]:seq[b + 1]]
            n = len(r)
            e = np.exp(r)
            total += db[b] * E / (k * n * n) * (counts[b] * (e / e.sum(1, keepdims=True)).sum(0)).sum()
            total += dz[b] * (np.log(e.sum(1)) ** 2).mean()
        e = np.exp(np.take_along_axis(v, idx.astype(np.int64), 1))
        return total + (dw * e / e.sum(1, keepdims=True)).sum()

    h = 1e-5  # the third derivative is of order one: h^2 of truncation, 1e-16 / h of rounding
    x64 = x.astype(np.float64)
    for t in range(T):
        for e in range(E):
            up, down = x64.copy(), x64.copy()
            up[t, e] += h
            down[t, e] -= h
            assert abs((f(up) - f(down)) / (2 * h) - g[t, e]) <= 1e-6


def test_gradient_of_the_gate_alone():
    rng = np.random.default_rng(8)
    for T, E, k, kind in ((200, 100, 8, "wild"), (77, 61, 3, "one"), (1, 4096, 8, "dup"), (5, 3, 8, "dup")):
        idx, (w, dw) = routing(rng, T, E, k, kind), gate(rng, T, k)
        logits = torch.full((T, E), float("nan"), device="cuda")  # not read
        d = moe.logits_grad(logits, dev(idx), topk_w=dev(w), d_topk_w=dev(dw))
        want, bound = ref.logits_grad(np.zeros((T, E)), idx, None, None, None, w, dw, None, k)
        ref.close(num(d), want, bound, "gate")


def test_summed_counts_of_several_batches():
    """The gradient goes by the counts and tokens that the losses hold when it is asked for."""
    rng = np.random.default_rng(9)
    x, idx = rng.standard_normal((90, 40)).astype(np.float32), routing(rng, 90, 40, 2)
    l = moe.router_losses(dev(x), dev(idx))
    other = moe.router_losses(dev(x[::-1].copy()), dev(routing(rng, 90, 40, 2)))
    l.counts.add_(other.counts)
    l.tokens += other.tokens
    got = {n: num(getattr(l, n)) for n in ("counts", "tokens", "lse")}
    d = moe.logits_grad(dev(x), dev(idx), l, d_balance=torch.ones(1, device="cuda"))
    want, bound = ref.logits_grad(x, idx, got, np.ones(1), None, None, None, None, 2)
    ref.close(num(d), want, bound, "d_logits")


# ---------------------------------------------------------------- the router's product

def grads(rng, T, E):
    g = rng.standard_normal((T, E)).astype(np.float32) * 1e-4
    hot = rng.random((T, E)) < 0.05
    return np.where(hot, g * 1000, g).astype(np.float32)


def bf16(rng, shape):
    return dev(rng.standard_normal(shape).astype(np.float32), BF16)


@pytest.mark.parametrize("T,E,D", [(1, 1, 64), (1, 384, 4096), (2, 8, 128), (31, 33, 192), (32, 32, 256), (33, 64, 320), (128, 128, 256), (129, 127, 576),
                                   (300, 60, 1088), (1000, 61, 64), (257, 384, 512), (2049, 129, 256), (5003, 40, 128), (70, 1025, 192)])
@pytest.mark.parametrize("kinds", [(BF16, BF16, False), (FP32, FP32, True), (BF16, FP32, True), (FP32, BF16, False), (BF16, BF16, True)], ids=str)
def test_route_backward(T, E, D, kinds):
    dh_t, dwr_t, bias = kinds
    rng = np.random.default_rng(T + E + D)
    g, h, wr = grads(rng, T, E), bf16(rng, (T, D)), bf16(rng, (E, D))
    dh, dwr, dbias = moe.route_backward(h, wr, dev(g), dh_dtype=dh_t, dwr_dtype=dwr_t, want_bias=bias)
    g = g.astype(np.float64)
    for name, got, a, b, t in (("dh", dh, g, num(wr), dh_t), ("dwr", dwr, np.ascontiguousarray(g.T), num(h), dwr_t)):
        assert got.dtype == t
        y, bound, mean = ref.product(a, b.astype(np.float64), t == BF16, 2 if t == BF16 else 3, 256)
        ref.close(num(got), y, bound, name)
        err = np.sqrt(((num(got) - y) ** 2).mean())
        assert got.numel() < 4096 or err <= mean, f"{name}: rms {err}, expected up to {mean}"
    if bias:
        y, bound, _ = ref.product(np.ascontiguousarray(g.T), np.ones((T, 1)), False, 3, 256)
        ref.close(num(dbias), y[:, 0], bound[:, 0], "dbias")
    else:
        assert dbias is None


def test_route_backward_in_parts():
    """Either output alone has the bits that it has beside the other; given buffers and a workspace that held other values."""
    rng = np.random.default_rng(11)
    g, h, wr = dev(grads(rng, 700, 90)), bf16(rng, (700, 384)), bf16(rng, (90, 384))
    dh, dwr, _ = moe.route_backward(h, wr, g)
    ws = moe.route_backward_workspace(700, 384, 90).fill_(255)
    one, none, _ = moe.route_backward(h, wr, g, dh=torch.full_like(dh, float("nan")), want_dwr=False, workspace=ws)
    assert none is None and torch.equal(one, dh)
    none, two, _ = moe.route_backward(h, wr, g, dwr=torch.full_like(dwr, float("nan")), want_dh=False, workspace=ws.fill_(255))
    assert none is None and torch.equal(two, dwr)
    a, b, c = moe.route_backward(h[:0], wr, g[:0], want_bias=True)
    assert a.shape == (0, 384) and not b.any() and not c.any() and b.shape == (90, 384)


def test_route_backward_of_extreme_gradients():
    """Values next to the type's largest and far below one come through; zeros give zeros; a NaN stays in its row and column."""
    T, E, D = 40, 20, 64
    h, wr, g = torch.zeros((T, D), dtype=BF16, device="cuda"), torch.zeros((E, D), dtype=BF16, device="cuda"), torch.zeros((T, E), device="cuda")
    wr[:, 0], h[:, 0] = 0.5, 0.5
    g[0, 0], g[1, 1], g[2, 2], g[3, 3] = torch.finfo(FP32).max, 2.0 ** -100 * (1 + 2.0 ** -23), -3.0, 1 + 2.0 ** -23
    for t in (BF16, FP32):
        dh, dwr, _ = moe.route_backward(h, wr, g, dh_dtype=t, dwr_dtype=t)
        for got in (num(dh)[:4, 0], num(dwr)[:4, 0]):
            want = num(g)[[0, 1, 2, 3], [0, 1, 2, 3]].astype(np.float64) / 2
            assert (np.abs(got - want) <= np.abs(want) * (ref.U_BF16 + 2.0 ** -15 if t == BF16 else ref.U24)).all()
        assert not num(dh)[4:].any() and not num(dh)[:, 1:].any() and not num(dwr)[4:].any()
    rng = np.random.default_rng(1)
    g, h, wr = dev(grads(rng, T, E)), bf16(rng, (T, D)), bf16(rng, (E, D))
    a, b, _ = moe.route_backward(h, wr, g)
    g[7, 3] = float("nan")
    c, d, _ = moe.route_backward(h, wr, g)
    assert torch.isnan(c[7]).all() and torch.isnan(d[3]).all()
    assert torch.equal(c[[i for i in range(T) if i != 7]], a[[i for i in range(T) if i != 7]])
    assert torch.equal(d[[i for i in range(E) if i != 3]], b[[i for i in range(E) if i != 3]])


def test_training_step():
    """route, losses, sort, combine, and all the way back: the gradients of h and of the router's weight against autograd in 64
    bits on the CPU, where the choice of experts and the counts are held."""
    rng = np.random.default_rng(12)
    T, D, E, k, seq = 200, 256, 24, 4, [0, 90, 200]
    h, wr = bf16(rng, (T, D)), (bf16(rng, (E, D)).float() * 0.1).to(BF16)
    idx, w, logits, _ = moe.route(h, wr, top_k=k, want_logits=True)
    l = moe.router_losses(logits, idx, seq=dev(np.array(seq, np.int32)))
    g = moe.sort_tokens(idx, E)
    y = dev(rng.standard_normal((T * k, D)).astype(np.float32))
    d_out = dev(rng.standard_normal((T, D)).astype(np.float32))
    moe.combine(g, y, w)
    _, dw = moe.combine_backward(g, d_out, y, w)
    db, dz = torch.full((2,), 0.5, device="cuda"), torch.full((2,), 0.1, device="cuda")
    d_logits = moe.logits_grad(logits, idx, l, db, dz, w, dw)
    dh, dwr, _ = moe.route_backward(h, wr, d_logits, dh_dtype=FP32)

    h64, wr64 = (torch.from_numpy(num(t).astype(np.float64)).requires_grad_() for t in (h, wr))
    idx64, pos = torch.from_numpy(host(idx).astype(np.int64)), torch.from_numpy(host(g.slot_pos).astype(np.int64))
    lo = h64 @ wr64.t()
    w64 = torch.softmax(torch.gather(lo, 1, idx64), 1)
    out = (w64[:, :, None] * torch.from_numpy(num(y).astype(np.float64))[pos]).sum(1)
    loss = (out * torch.from_numpy(num(d_out).astype(np.float64))).sum()
    for b in range(2):
        r = lo[seq[b]:seq[b + 1]]
        n = r.shape[0]
        counts = torch.bincount(idx64[seq[b]:seq[b + 1]].flatten(), minlength=E).double()
        balance = E / (k * n * n) * (counts * torch.softmax(r, 1).sum(0)).sum()
        z = (torch.logsumexp(r, 1) ** 2).mean()
        assert abs(float(l.balance[b]) - balance.item()) <= 1e-5 * balance.item() and abs(float(l.z[b]) - z.item()) <= 1e-5 * z.item()
        loss = loss + 0.5 * balance + 0.1 * z
    loss.backward()
    # each step is within some hundred roundings of its terms' size; the terms of a gradient here are about as large as the
    # largest gradient, 1000 U24 of it
    for got, want in ((dh, h64.grad), (dwr, wr64.grad)):
        want = want.numpy()
        assert np.abs(num(got) - want).max() <= 1000 * ref.U24 * np.abs(want).max()


def test_streams_and_graph_replays():
    """On a stream of its own, and captured: replays with new values in the captured buffers give what the eager calls give."""
    rng = np.random.default_rng(13)
    T, E, D, k = 600, 100, 128, 4
    seq = dev(np.array([0, 100, 600], np.int32))
    logits, g = torch.zeros((T, E), device="cuda"), torch.zeros((T, E), device="cuda")
    h, wr = bf16(rng, (T, D)), bf16(rng, (E, D))
    idx = dev(routing(rng, T, E, k))
    w, dw = (dev(a) for a in gate(rng, T, k))
    ones = torch.ones(2, device="cuda")

    def step():
        l = moe.router_losses(logits, idx, seq=seq)
        d = moe.logits_grad(logits, idx, l, ones, ones, w, dw)
        dh, dwr, dbias = moe.route_backward(h, wr, d, want_bias=True)
        return [l.balance, l.z, l.counts, l.tokens, l.prob_sums, l.lse, d, dh, dwr, dbias]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        logits.copy_(dev(rng.standard_normal((T, E)).astype(np.float32)))
        idx.copy_(dev(routing(rng, T, E, k, "wild")))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, step()))


def test_more_than_32_bits_of_logits():
    """Logits numbered past 2^31: 64 rows again and again, the last two repetitions sequences of their own."""
    rng = np.random.default_rng(14)
    E, k, T = 4096, 8, 2 ** 19 + 192
    base, idx = bf16(rng, (64, E)), routing(rng, 64, E, k)
    logits = base.repeat(T // 64, 1)
    many = dev(idx).repeat(T // 64, 1)
    l = moe.router_losses(logits, many, seq=dev(np.array([0, T - 128, T - 64, T], np.int32)))
    want, bound, _, _ = ref.losses(num(base), idx, None, None, k)
    for s in (1, 2):
        assert np.array_equal(num(l.counts)[s], want["counts"][0]) and num(l.tokens)[s] == 64
        for n in ("balance", "z", "prob_sums"):
            ref.close(num(getattr(l, n))[s:s + 1], want[n], bound[n], n)
    assert np.array_equal(num(l.counts)[0], want["counts"][0] * (T // 64 - 2))
    ref.close(num(l.lse)[-64:], want["lse"], bound["lse"], "lse")
    assert bool((l.lse.view(-1, 64) == l.lse[:64]).all())
    db, dz = np.array([0.5, -2.0, 3.0], np.float32), np.array([1.0, 0.5, -1.5], np.float32)
    w, dw = gate(rng, 64, k)
    d = moe.logits_grad(logits, many, l, dev(db), dev(dz), dev(w).repeat(T // 64, 1), dev(dw).repeat(T // 64, 1))
    for s, rows in ((1, slice(T - 128, T - 64)), (2, slice(T - 64, T))):
        got = {"counts": num(l.counts)[s:s + 1], "tokens": num(l.tokens)[s:s + 1], "lse": num(l.lse)[rows]}
        want_d, bound_d = ref.logits_grad(num(base), idx, got, db[s:s + 1], dz[s:s + 1], w, dw, None, k)
        ref.close(num(d[rows]), want_d, bound_d, f"d_logits of {s}")
    for i in range(0, T - 128, 1 << 16):
        rows = d[i:min(i + (1 << 16), T - 128)].view(-1, 64, E)
        assert bool((rows == d[:64]).all())


def test_more_than_32_bits_of_hidden_states():
    """h and dh numbered past 2^31, of small whole numbers: every sum is exact, in whatever order."""
    rng = np.random.default_rng(15)
    T, D, E = 2 ** 19 + 192, 4096, 9
    h, wr, g = (rng.integers(-a, a + 1, s).astype(np.float32) for a, s in ((2, (64, D)), (2, (E, D)), (1, (64, E))))
    n = T // 64
    dh, dwr, dbias = moe.route_backward(dev(h, BF16).repeat(n, 1), dev(wr, BF16), dev(g).repeat(n, 1), want_bias=True)
    assert np.array_equal(num(dwr), n * (g.T @ h)) and np.array_equal(num(dbias), n * g.sum(0))
    want = dev(g @ wr, BF16)
    for i in range(0, T, 1 << 16):
        assert bool((dh[i:i + (1 << 16)].view(-1, 64, D) == want).all()), f"rows from {i} on"
