"""The operators of include/moe_ops.h on the GPU against plain forms in 64 bits (ops_ref.py):
tokens grouped by expert and back, the FP8 quantisers with a scale per block of 128, the grouped
product and its gradients, at the sizes and routings where they can go wrong; a run of them
together; streams and graph replays."""
import numpy as np
import pytest
import torch

import block_scaled_moe_amd as moe
import ops_ref as ref
from gpu_util import host

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
INT_MIN = -2 ** 31


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def values(rng, shape, dtype="fp32"):
    x = rng.standard_normal(shape).astype(np.float32)
    return ref.bf16(x) if dtype == "bf16" else x


def num(t):
    return host(t.float() if t.dtype == torch.bfloat16 else t)


# ---------------------------------------------------------------- sort

def routing(kind, T, k, E, rng):
    if kind == "distinct":
        return np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    if kind == "one":      # every slot on one expert, the same one k times in a token
        return np.full((T, k), E // 2, np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    if kind == "wild":     # padding and values that are no expert, up to the ends of the type
        idx = rng.integers(0, E, (T, k)).astype(np.int32)
        bad = rng.choice(np.array([-1, -7, E, E + 5, INT_MIN, 2 ** 31 - 1], np.int64), (T, k)).astype(np.int32)
        return np.where(rng.random((T, k)) < 0.4, bad, idx).astype(np.int32)
    return rng.integers(0, E, (T, k)).astype(np.int32)  # "dup": repeats allowed


SORTS = [
    ("distinct", 1, 8, 384, 0, 384), ("distinct", 64, 8, 384, 96, 192), ("wild", 64, 8, 384, 96, 192),
    ("one", 50, 8, 16, 0, 16), ("none", 9, 4, 32, 0, 32), ("dup", 0, 8, 16, 0, 16), ("dup", 33, 3, 5, 4, 5),
    ("wild", 2000, 8, 60, 7, 50), ("dup", 1500, 7, 4096, 0, 4096), ("wild", 700, 1, 2000, 100, 2000),
    ("dup", 5000, 2, 1, 0, 1), ("dup", 0, 1, 2000, 0, 2000), ("one", 3000, 4, 3, 0, 3), ("dup", 1, 1, 1, 0, 1),
]


@pytest.mark.parametrize("kind,T,k,E,e0,e1", SORTS)
def test_sort(kind, T, k, E, e0, e1):
    rng = np.random.default_rng(T * 7 + E)
    idx = routing(kind, T, k, E, rng)
    g = moe.sort_tokens(dev(idx), E, e0, e1)
    off, ss, sp = ref.sort(idx, e0, e1)
    assert np.array_equal(host(g.offsets), off)
    assert np.array_equal(host(g.slot_pos), sp)
    assert np.array_equal(host(g.sorted_slot), ss)
    again = moe.sort_tokens(dev(np.roll(idx, 1, 0)), E, e0, e1, out=g)  # the same buffers for another batch
    off, ss, sp = ref.sort(np.roll(idx, 1, 0), e0, e1)
    assert again is g and np.array_equal(host(g.sorted_slot), ss) and np.array_equal(host(g.slot_pos), sp)


# ---------------------------------------------------------------- rows by expert and back

ROWS = [
    ("distinct", 1, 8, 64, 0, 64, 4096), ("wild", 37, 8, 16, 3, 11, 257), ("dup", 130, 3, 7, 0, 7, 1001),
    ("wild", 65, 5, 9, 0, 9, 8), ("none", 4, 2, 4, 0, 4, 72), ("one", 20, 8, 4, 0, 4, 640), ("dup", 9, 1, 3, 1, 3, 1),
    ("wild", 1300, 4, 12, 0, 6, 136), ("dup", 3, 6, 8, 0, 8, 2052), ("dup", 7, 2, 4, 0, 4, 516), ("dup", 300, 8, 8, 0, 4, 20),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind,T,k,E,e0,e1,D", ROWS)
def test_gather_and_its_gradient(kind, T, k, E, e0, e1, D, dtype):
    rng = np.random.default_rng(D + T)
    idx = routing(kind, T, k, E, rng)
    g = moe.sort_tokens(dev(idx), E, e0, e1)
    off, ss, sp = ref.sort(idx, e0, e1)
    S = off[-1]
    x = values(rng, (T, D), dtype)
    buf = torch.full((T * k + 3, D), 7.0, dtype=DT[dtype], device="cuda")
    rows = moe.gather(g, dev(x, DT[dtype]), out=buf[:T * k])
    assert np.array_equal(num(rows)[:S], x[ss[:S] // k])
    assert (num(buf)[S:] == 7.0).all()          # rows behind the last local one keep what they hold
    d = values(rng, (T * k, D), dtype)
    d[S:] = np.nan                              # and are not read
    dx = num(moe.gather_backward(g, dev(d, DT[dtype]))).astype(np.float64)
    terms = np.where(sp[:, :, None] >= 0, d[np.maximum(sp, 0)], 0).astype(np.float64)
    want, size = terms.sum(1), np.abs(terms).sum(1)
    bound = k * ref.U24 * size                  # k fp32 additions
    if dtype == "bf16":
        bound = bound + ref.U_BF16 * (np.abs(want) + bound)
    assert (np.abs(dx - want) <= bound).all()


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind,T,k,E,e0,e1,D", ROWS)
def test_combine_and_its_gradient(kind, T, k, E, e0, e1, D, dtype, out_dtype):
    rng = np.random.default_rng(D + T + 1)
    idx = routing(kind, T, k, E, rng)
    g = moe.sort_tokens(dev(idx), E, e0, e1)
    off, ss, sp = ref.sort(idx, e0, e1)
    S = off[-1]
    y, w, d = values(rng, (T * k, D), dtype), values(rng, (T, k)), values(rng, (T, D), out_dtype)
    y[S:] = np.nan
    local = (sp >= 0)[:, :, None]
    ys = np.where(local, y[np.maximum(sp, 0)], 0).astype(np.float64)
    terms = ys * w[:, :, None].astype(np.float64)
    want, size = terms.sum(1), np.abs(terms).sum(1)
    out = num(moe.combine(g, dev(y, DT[dtype]), dev(w), out_dtype=DT[out_dtype]))
    bound = k * ref.U24 * size                  # k fused multiply-adds
    if out_dtype == "bf16":
        bound = bound + ref.U_BF16 * (np.abs(want) + bound)
    assert (np.abs(out - want) <= bound).all()

    buf = torch.full((T * k + 2, D), 5.0, dtype=DT[dtype], device="cuda")
    dy, dw = moe.combine_backward(g, dev(d, DT[out_dtype]), dev(y, DT[dtype]), dev(w), dy=buf[:T * k])
    want_dy = (w.reshape(-1)[ss[:S]][:, None].astype(np.float64) * d[ss[:S] // k])
    step = ref.U24 * np.abs(want_dy)            # one product
    if dtype == "bf16":
        step = step + ref.U_BF16 * (np.abs(want_dy) + step)
    assert (np.abs(num(dy)[:S] - want_dy) <= step).all()
    assert (num(buf)[S:] == 5.0).all()
    prod = ys * d[:, None, :].astype(np.float64)
    # each thread's chain of multiply-adds (at most 8 per 256 of the row's pieces of one element), then a tree of at most 10
    depth = 8 * ((D + 255) // 256) + 10
    assert (np.abs(num(dw) - prod.sum(2)) <= depth * ref.U24 * np.abs(prod).sum(2)).all()
    assert (num(dw)[sp < 0] == 0).all()


def test_non_finite_rows_stay_in_their_sums():
    """A NaN or infinite row reaches its own token and no other; non-local slots contribute nothing."""
    idx = np.array([[0, 1], [1, 5], [-1, -1], [0, 0]], np.int32)  # expert 5 is remote
    g = moe.sort_tokens(dev(idx), 8, 0, 2)
    y = np.ones((8, 64), np.float32)
    y[4] = np.nan                                    # token 1's row at expert 1: slots sorted 0,6,7 | 1,2
    y[5:] = np.inf
    w = np.full((4, 2), 0.5, np.float32)
    w[1, 1] = np.inf                                 # weight of the remote slot
    out = num(moe.combine(g, dev(y), dev(w)))
    assert np.isnan(out[1]).all() and (out[0] == 1).all() and (out[2] == 0).all() and (out[3] == 1).all()


# ---------------------------------------------------------------- quantisers

def hard_values(rng, shape):
    """bf16 values whose blocks of 128 differ in size, with zeros, zero blocks, ends of the range, subnormals and ties."""
    x = rng.standard_normal(shape).astype(np.float32)
    x = x * np.exp2(rng.integers(-30, 30, size=shape[:-1] + (shape[-1] // 128,))).repeat(128, -1).astype(np.float32)
    flat = x.reshape(-1, 128)
    for i, f in enumerate((0.0, 2.0 ** -126, 2.0 ** -133, 2.0 ** 120, 2.0 ** -75, 2.0 ** 75)):
        if i < len(flat):
            flat[i] = 0.0 if f == 0 else rng.integers(-255, 256, 128) * np.float32(f)
    if len(flat) > 8:
        flat[7] = np.where(rng.random(128) < 0.5, 448.0, rng.integers(0, 64, 128) * 0.25)  # scale 1: exact ties
        flat[8, :] = 0.0
        flat[8, 5] = -3e38
    return ref.bf16(x)


def rows_codes(q):
    """Codes [C/128, R, 128] -> [R, C]."""
    c = host(q.codes)
    return c.transpose(1, 0, 2).reshape(c.shape[1], -1)


@pytest.mark.parametrize("R,C", [(1, 128), (3, 384), (129, 256), (300, 4096), (17, 1152)])
def test_quantise_rows(R, C):
    x = hard_values(np.random.default_rng(R), (R, C))
    q = moe.quantize_block(dev(x, torch.bfloat16))
    c, s = ref.rows(x)
    assert np.array_equal(host(q.scales)[:, :C // 128].copy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(rows_codes(q), c)


@pytest.mark.parametrize("E,N,K", [(1, 128, 128), (3, 256, 384), (2, 640, 128)])
def test_quantise_and_pack_weights(E, N, K):
    w = hard_values(np.random.default_rng(N), (E, N, K))
    q = moe.quantize_block_weights(dev(w, torch.bfloat16))
    c, s = ref.weights(w)
    assert np.array_equal(host(q.scales).view(np.uint32), s.view(np.uint32))
    assert np.array_equal(host(q.codes), ref.tile(c))
    p = moe.pack_block_weights(dev(c), dev(s))
    assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
    v = p.experts(E - 1, E)
    assert v.E == 1 and np.array_equal(host(v.codes)[0], ref.tile(c)[E - 1])


def exact_counts(counts, k=1):
    """Routing of k = 1 whose local expert e has counts[e] rows, tokens in a random order."""
    idx = np.repeat(np.arange(len(counts)), counts).astype(np.int32)
    return np.random.default_rng(3).permutation(idx)[:, None]


COUNTS = [[1], [0, 3, 0], [128, 129, 0, 127], [300, 0, 1, 260], [5] * 70, [0, 0], [16, 17, 15, 223, 224, 225, 449]]


@pytest.mark.parametrize("C", [128, 640])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_quantise_columns(counts, C):
    rng = np.random.default_rng(sum(counts))
    idx = exact_counts(counts)
    T = len(idx)
    g = moe.sort_tokens(dev(idx.reshape(T, 1)), len(counts))
    off, ss, _ = ref.sort(idx, 0, len(counts))
    x = hard_values(rng, (T, C)) if T else np.zeros((0, C), np.float32)
    sorted_x = x[ss]
    want = ref.columns(sorted_x, off)
    rows, cols = moe.quantize_block_both(dev(sorted_x, torch.bfloat16), g)
    only = moe.quantize_block_columns(dev(sorted_x, torch.bfloat16), g)
    tok = moe.quantize_block_columns(dev(x, torch.bfloat16), g, by_token=True)
    for q in (cols, only, tok):
        qc, qs = host(q.codes), host(q.scales)
        for b, (c, s) in want.items():
            assert np.array_equal(qs[b].view(np.uint32), s.view(np.uint32)), b
            assert np.array_equal(qc[b], c), b
    if T:
        c, s = ref.rows(sorted_x)
        assert np.array_equal(rows_codes(rows), c) and np.array_equal(host(rows.scales)[:, :C // 128], s)


def test_quantise_leaves_rows_behind_the_last_one():
    """Rows of remote experts are not quantised: their codes and scales keep what they hold."""
    idx = np.array([[0, 9], [9, 1], [9, 9]], np.int32)
    g = moe.sort_tokens(dev(idx), 16, 0, 2)
    x = torch.full((6, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:2] = 1.5
    codes = torch.full((2, 6, 128), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((6, 4), 9.0, device="cuda")
    import ctypes
    from block_scaled_moe_amd import ops
    a = ops.MoeBlockQuantizeArgs(rows=6, C=256, g=ctypes.pointer(g.struct), x=x.data_ptr(), codes=codes.data_ptr(),
                                 scales=scales.data_ptr())
    ops._call("moe_block_quantize", x.device, ctypes.byref(a))
    assert (host(codes)[:, :2] == 0x7E).all() and (host(codes)[:, 2:] == 9).all() and (host(scales)[2:] == 9).all()
    assert (host(scales)[:, 2:] == 9).all()     # nor the padding of a row's scales


# ---------------------------------------------------------------- products

def check(got, want, bound, what):
    bad = np.abs(got.astype(np.float64) - want) > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - want)[bad].max()}"


GEMMS = [(c, n, k) for c in COUNTS for n, k in ((128, 128), (384, 640))] + [
    ([257, 40, 600], 512, 256), ([1, 2, 0, 9], 256, 4352), ([70, 33], 128, 8448), ([513], 768, 384), ([20], 5120, 512)]


def setup_product(counts, N, K, seed, spread=True):
    rng = np.random.default_rng(seed)
    idx = exact_counts(counts)
    T = len(idx)
    g = moe.sort_tokens(dev(idx.reshape(T, 1)), len(counts))
    off, ss, _ = ref.sort(idx, 0, len(counts))
    w = ref.bf16(rng.standard_normal((len(counts), N, K)).astype(np.float32) *
                 np.exp2(rng.integers(-6, 6, (len(counts), N // 128, K // 128))).repeat(128, 1).repeat(128, 2))
    wq = moe.quantize_block_weights(dev(w, torch.bfloat16))
    expert = np.repeat(np.arange(len(counts)), counts)
    return rng, g, off, ss, wq, ref.weights(w), expert


@pytest.mark.parametrize("counts,N,K", GEMMS, ids=str)
def test_product(counts, N, K):
    rng, g, off, ss, wq, (wc, ws), expert = setup_product(counts, N, K, sum(counts) + N)
    T = g.T
    x = ref.bf16(rng.standard_normal((T, K)).astype(np.float32) * np.exp2(rng.integers(-4, 5, (T, 1))))
    xc, xs = ref.rows(x) if T else (np.zeros((0, K), np.uint8), np.zeros((0, K // 128), np.float32))
    y, bound = ref.product(xc[ss], xs[ss], wc, ws, expert)
    q = moe.quantize_block(dev(x, torch.bfloat16))
    check(num(moe.block_product(q, wq, g, by_token=True)), y, bound, "by token")
    qs = moe.quantize_block(dev(x[ss], torch.bfloat16), g)
    buf = torch.full((T + 1, N), 3.0, dtype=torch.bfloat16, device="cuda")
    check(num(moe.block_product(qs, wq, g, out=buf[:T])), y, bound, "sorted")
    assert (num(buf)[T:] == 3.0).all()


@pytest.mark.parametrize("K", [128, 256, 384])
def test_short_sums_over_many_items(K):
    """More work items than CUs with one to three blocks each, by token: an item's rows are looked up while the last
    one is computed."""
    test_product([40, 7, 33, 90] * 6, 5120, K)


FEW = [([0, 5, 16, 17] + [0] * 20, 256, 640), ([33, 64, 65] + [0] * 40, 128, 1152), ([300] + [0] * 59, 128, 256),
       ([1] * 7 + [100] + [2] * 40, 384, 128), ([224, 225] + [0] * 90, 128, 1664)]


@pytest.mark.parametrize("counts,N,K", FEW, ids=lambda v: str(v)[:20])
def test_product_few_rows_on_average(counts, N, K):
    """Groups of few rows on average (a decode batch), some with many rows, and blocks that the four waves share unevenly."""
    assert sum(counts) // len(counts) <= 5
    test_product(counts, N, K)


@pytest.mark.parametrize("counts,N,K", GEMMS, ids=str)
def test_product_gradients(counts, N, K):
    rng, g, off, ss, wq, (wc, ws), expert = setup_product(counts, N, K, sum(counts) + K)
    T = g.T
    dy = ref.bf16(rng.standard_normal((T, N)).astype(np.float32) * np.exp2(rng.integers(-4, 5, (T, 1))))
    x = ref.bf16(rng.standard_normal((T, K)).astype(np.float32))
    gq, gc = moe.quantize_block_both(dev(dy, torch.bfloat16), g)
    xq = moe.quantize_block_columns(dev(x, torch.bfloat16), g)
    if T:
        c, s = ref.rows(dy)
        want, bound = ref.product(c, s, wc, ws, expert, transposed=True)
        buf = torch.full((T + 1, K), 3.0, dtype=torch.bfloat16, device="cuda")
        check(num(moe.block_product_grad(gq, wq, g, out=buf[:T])), want, bound, "dx")
        assert (num(buf)[T:] == 3.0).all()
    dw = num(moe.block_weight_grad(gc, xq, g))
    cg, cx = ref.columns(dy, off), ref.columns(x, off)
    for e in range(len(counts) if T else 0):
        check(dw[e], *ref.weight_grad(cg, cx, off, e), f"dw[{e}]")
    assert (dw[np.array(counts) == 0] == 0).all()


@pytest.mark.parametrize("M", [1, 16, 17, 48, 65, 96, 97, 300, 513])
def test_one_group(M):
    """Without groups: a dense projection and its gradients."""
    rng = np.random.default_rng(M)
    N, K = 384, 512
    x, dy = values(rng, (M, K), "bf16"), values(rng, (M, N), "bf16")
    w = values(rng, (1, N, K), "bf16")
    wq = moe.quantize_block_weights(dev(w, torch.bfloat16))
    wc, ws = ref.weights(w)
    expert, off = np.zeros(M, int), np.array([0, M])
    check(num(moe.block_product(moe.quantize_block(dev(x, torch.bfloat16)), wq)), *ref.product(*ref.rows(x), wc, ws, expert), "y")
    gq, gc = moe.quantize_block_both(dev(dy, torch.bfloat16))
    check(num(moe.block_product_grad(gq, wq)), *ref.product(*ref.rows(dy), wc, ws, expert, transposed=True), "dx")
    xq = moe.quantize_block_columns(dev(x, torch.bfloat16))
    check(num(moe.block_weight_grad(gc, xq, rows=M))[0], *ref.weight_grad(ref.columns(dy, off), ref.columns(x, off), off, 0), "dw")


@pytest.mark.parametrize("k1,k2,k3", [(0, 1, 2), (0, 64, 1), (0, 127, 64), (5, 6, 100), (17, 90, 18)])
def test_small_products_beside_large_ones(k1, k2, k3):
    """A product counts in full beside one 2^13 times its size in the same block: 2^16 - 2^16 + 2^j keeps 2^j for
    j >= 3 at any places of the block (the tolerances of the products rest on it). Two unused values fix the scales at 1."""
    js = list(range(3, 17))
    x, w = np.zeros((len(js), 128), np.float32), np.zeros((1, 128, 128), np.float32)
    free = [k for k in range(128) if k not in (k1, k2, k3)][:2]
    x[:, free[0]], w[0, :, free[1]] = 448.0, 448.0
    x[:, k1], x[:, k2], w[0, :, k1], w[0, :, k2], w[0, :, k3] = 256.0, -256.0, 256.0, 256.0, 2.0 ** 8
    x[:, k3] = np.exp2(np.array(js) - 8)
    y = num(moe.block_product(moe.quantize_block(dev(x, torch.bfloat16)), moe.quantize_block_weights(dev(w, torch.bfloat16))))
    assert (y == np.exp2(np.array(js))[:, None]).all()


def test_gradients_against_differences():
    """The product's gradients against differences of the product itself. Where the values are E4M3 values
    with a scale that a change of one element does not move (each block holds a 448), quantising is exact, the
    product is bilinear, and a difference gives the derivative up to the roundings of y."""
    rng = np.random.default_rng(5)
    N, K, M = 128, 128, 6
    vals = ref.e4m3_value(np.arange(0x30, 0x60, dtype=np.uint8)).astype(np.float32)  # 1/4 .. 15
    x, w = rng.choice(vals, (M, K)), rng.choice(vals, (1, N, K))
    x[:, 0], w[0, 0, 0] = 448.0, 448.0
    dy = np.zeros((M, N), np.float32)
    dy[:, 3] = 448.0                       # the loss is 448 * sum of column 3 of y, scale 1
    wq = moe.quantize_block_weights(dev(w, torch.bfloat16))
    f = lambda xx, ww: num(moe.block_product(moe.quantize_block(dev(xx, torch.bfloat16)),
                                             moe.quantize_block_weights(dev(ww, torch.bfloat16)))).astype(np.float64)
    gq, gc = moe.quantize_block_both(dev(dy, torch.bfloat16))
    dx = num(moe.block_product_grad(gq, wq))
    dw = num(moe.block_weight_grad(gc, moe.quantize_block_columns(dev(x, torch.bfloat16)), rows=M))[0]
    base = f(x, w)
    for m, k in ((0, 5), (3, 77), (5, 127)):
        x2 = x.copy()
        x2[m, k] = 240.0 if x[m, k] < 16 else 1.0   # a value E4M3 holds
        diff = 448.0 * (f(x2, w)[m, 3] - base[m, 3]) / (x2[m, k] - x[m, k])
        slack = 448.0 * ref.U_BF16 * (abs(f(x2, w)[m, 3]) + abs(base[m, 3])) / abs(x2[m, k] - x[m, k])
        assert abs(diff - dx[m, k]) <= slack + ref.U_BF16 * abs(dx[m, k]) + 1e-3
    for k in (4, 90):
        w2 = w.copy()
        w2[0, 3, k] = 240.0
        diff = 448.0 * (f(x, w2)[:, 3] - base[:, 3]).sum() / (w2[0, 3, k] - w[0, 3, k])
        slack = 448.0 * ref.U_BF16 * (np.abs(f(x, w2)[:, 3]) + np.abs(base[:, 3])).sum() / abs(w2[0, 3, k] - w[0, 3, k])
        # x's columns are quantised anew for dw: half an E4M3 step of each element
        assert abs(diff - dw[3, k]) <= slack + (2.0 ** -4 + ref.U_BF16) * 448.0 * np.abs(x[:, k]).sum()


def test_experts_out_of_a_longer_array():
    """Weights whose scales do not start on 16 bytes: experts 1 .. 2 of four with one block each."""
    rng = np.random.default_rng(3)
    w, x = values(rng, (4, 128, 128), "bf16"), values(rng, (40, 128), "bf16")
    wq = moe.quantize_block_weights(dev(w, torch.bfloat16))
    out = moe.BlockWeights.empty(4, 128, 128)
    for t in (out.codes, out.scales):
        t.zero_()
    moe.quantize_block_weights(dev(w[1:3], torch.bfloat16), out=out.experts(1, 3))
    assert torch.equal(out.scales[1:3], wq.scales[1:3]) and torch.equal(out.codes[1:3], wq.codes[1:3])
    assert not out.scales[0].any() and not out.codes[3].any()
    wc, ws = ref.weights(w)
    idx = rng.integers(0, 4, 40).astype(np.int32)
    g = moe.sort_tokens(dev(idx.reshape(40, 1)), 4, 1, 3)
    off, ss, _ = ref.sort(idx, 1, 3)
    S = off[-1]
    expert = np.repeat(np.arange(1, 3), np.diff(off))
    y = num(moe.block_product(moe.quantize_block(dev(x, torch.bfloat16)), wq.experts(1, 3), g, by_token=True))
    check(y[:S], *ref.product(*ref.rows(x[ss[:S]]), wc, ws, expert), "y")
    d = moe.quantize_block(dev(np.concatenate([x[ss[:S]], x[S:]]), torch.bfloat16), g)
    check(num(moe.block_product_grad(d, wq.experts(1, 3), g))[:S],
          *ref.product(*ref.rows(x[ss[:S]]), wc, ws, expert, transposed=True), "dx")


@pytest.mark.parametrize("D", [8 * 256 * 65535 + 8, 256 * 65535 + 3])
def test_one_long_row(D):
    """One token's row in more pieces than a grid has workgroups in y."""
    g = moe.sort_tokens(dev(np.array([[1, 0]], np.int32)), 2)
    x = torch.arange(D, device="cuda", dtype=torch.int32).bitwise_and_(127).to(torch.bfloat16).reshape(1, D)
    rows = moe.gather(g, x)
    assert torch.equal(rows[0], x[0]) and torch.equal(rows[1], x[0])
    out = moe.combine(g, rows, torch.tensor([[1.0, 0.5]], device="cuda"), out_dtype=torch.bfloat16)
    assert torch.equal(out[0], x[0] * 1.5)   # both the rounded exact product


def test_places_past_32_bits():
    """Sorted rows of more than 2^31 values: the second expert's 300 rows, the last ones, give the bits that they
    give alone."""
    T, D, last = 530000, 4096, 300
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    idx = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    pick = torch.randperm(T, device="cuda", generator=gen)[:last].sort().values
    idx[pick] = 1
    x = torch.randn((T, D), dtype=torch.bfloat16, device="cuda", generator=gen)
    w = moe.quantize_block_weights(torch.randn((2, D, D), dtype=torch.bfloat16, device="cuda", generator=gen))
    g = moe.sort_tokens(idx, 2)
    one = moe.sort_tokens(torch.zeros((last, 1), dtype=torch.int32, device="cuda"), 1)
    rows = moe.gather(g, x)
    xs = x[pick]
    assert rows.numel() > 2 ** 31 and torch.equal(rows[-last:], xs)
    ones = torch.ones((T, 1), device="cuda")
    out = moe.combine(g, rows, ones, out_dtype=torch.bfloat16)
    assert torch.equal(out[pick], xs) and torch.equal(out[-1], x[-1])
    dy, dw = moe.combine_backward(g, out, rows, ones)
    assert torch.equal(dy[-last:], xs) and torch.equal(dw[pick], moe.combine_backward(one, xs, xs, ones[:last])[1])
    del out, dy
    q, c = moe.quantize_block_both(rows, g)
    q1, c1 = moe.quantize_block_both(xs, one)
    assert torch.equal(q.codes[:, -last:], q1.codes) and torch.equal(q.scales[-last:], q1.scales)
    w1 = w.experts(1, 2)
    y1 = moe.block_product(q1, w1, one)
    assert torch.equal(moe.block_product(q, w, g)[-last:], y1)
    assert torch.equal(moe.block_product(moe.quantize_block(x), w, g, by_token=True)[-last:], y1)
    assert torch.equal(moe.block_product_grad(q, w, g)[-last:], moe.block_product_grad(q1, w1, one))
    assert torch.equal(moe.block_weight_grad(c, c, g)[1], moe.block_weight_grad(c1, c1, one)[0])


# ---------------------------------------------------------------- together

def chain(h, wr, w1, w2, d_out, k, E, e0, e1):
    """A small expert layer and its gradients, as a training step runs them; every stage's tensors."""
    idx, w, _, _ = moe.route(h, wr, top_k=k)
    g = moe.sort_tokens(idx, E, e0, e1)
    y1 = moe.block_product(moe.quantize_block(h), w1, g, by_token=True)
    a = torch.relu(y1)                                  # the program's own activation between the products
    y2 = moe.block_product(moe.quantize_block(a, g), w2, g)
    out = moe.combine(g, y2, w)
    dy2, dw = moe.combine_backward(g, d_out, y2, w)
    q2, c2 = moe.quantize_block_both(dy2, g)
    da = moe.block_product_grad(q2, w2, g)
    dw2 = moe.block_weight_grad(c2, moe.quantize_block_columns(a, g), g)
    dy1 = torch.where(y1 > 0, da, torch.zeros_like(da))
    q1, c1 = moe.quantize_block_both(dy1, g)
    dh = moe.gather_backward(g, moe.block_product_grad(q1, w1, g))
    dw1 = moe.block_weight_grad(c1, moe.quantize_block_columns(h, g, by_token=True), g)
    return dict(idx=idx, w=w, y1=y1, a=a, y2=y2, out=out, dy2=dy2, dw=dw, da=da, dw2=dw2, dy1=dy1, dh=dh, dw1=dw1, g=g)


def chain_inputs(T, D, F, E, n, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(s, device="cuda", generator=gen).to(torch.bfloat16)
    return (r(T, D), r(E, D), moe.quantize_block_weights(r(n, F, D)), moe.quantize_block_weights(r(n, D, F)),
            torch.randn((T, D), device="cuda", generator=gen))


def dequant(w):
    c = host(w.codes).transpose(0, 1, 4, 2, 3, 5).reshape(w.E, w.N, w.K)
    return c, host(w.scales)


@pytest.mark.parametrize("T,E,e0,e1", [(1, 16, 0, 16), (90, 16, 0, 16), (200, 16, 4, 9)])
def test_layer_and_gradients_stage_by_stage(T, E, e0, e1):
    """route, sort, product, product, combine and all gradients: each stage against its definition in 64 bits on
    the tensors that the stage before it gave."""
    D, F, k = 256, 128, 4
    h, wr, w1, w2, d_out = chain_inputs(T, D, F, E, e1 - e0, T)
    r = chain(h, wr, w1, w2, d_out, k, E, e0, e1)
    off, ss, sp = ref.sort(host(r["idx"]), e0, e1)
    S = off[-1]
    expert = np.repeat(np.arange(e1 - e0), np.diff(off))
    tok = ss[:S] // k

    def prod(x, w, got, what, transposed=False):
        if S == 0:
            return
        check(num(got)[:S], *ref.product(*ref.rows(x), *dequant(w), expert, transposed), what)

    prod(num(h)[tok], w1, r["y1"], "y1")
    prod(num(r["a"])[:S], w2, r["y2"], "y2")
    prod(num(r["dy2"])[:S], w2, r["da"], "da", True)
    w = host(r["w"]).astype(np.float64)
    ys = np.where((sp >= 0)[:, :, None], num(r["y2"])[np.maximum(sp, 0)].astype(np.float64), 0)
    terms = ys * w[:, :, None]
    assert (np.abs(num(r["out"]) - terms.sum(1)) <= k * ref.U24 * np.abs(terms).sum(1)).all()
    p = ys * num(d_out)[:, None, :].astype(np.float64)
    assert (np.abs(num(r["dw"]) - p.sum(2)) <= 26 * ref.U24 * np.abs(p).sum(2)).all()
    for name, gy, x, wq in (("dw2", r["dy2"], num(r["a"])[:S], w2), ("dw1", r["dy1"], num(h)[tok], w1)):
        cg, cx = ref.columns(num(gy)[:S], off), ref.columns(x, off)
        for e in range(e1 - e0 if S else 0):
            check(num(r[name])[e], *ref.weight_grad(cg, cx, off, e), f"{name}[{e}]")


FINAL = ("out", "dw", "dw2", "dh", "dw1")


def test_graph_replays_and_streams():
    """The layer and its gradients captured into a graph, replayed with new inputs between eager runs, and run on two
    streams at once with separate groups: the same bits as alone."""
    T, D, F, E, k = 150, 256, 128, 16, 4
    sets = [chain_inputs(T, D, F, E, E, s) for s in (1, 2, 3)]
    want = []
    for s in sets:
        r = chain(*s, k, E, 0, E)
        want.append({n: r[n].clone() for n in FINAL})
    torch.cuda.synchronize()
    own_copy = lambda t: t.clone() if torch.is_tensor(t) else moe.BlockWeights(t.E, t.N, t.K, t.codes.clone(), t.scales.clone())
    static = tuple(own_copy(t) for t in sets[0])
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(*static, k, E, 0, E)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        r = chain(*static, k, E, 0, E)
    for i in (0, 1, 2, 0, 1):
        for a, b in ((static[0], sets[i][0]), (static[1], sets[i][1]), (static[4], sets[i][4])):
            a.copy_(b)
        for a, b in ((static[2], sets[i][2]), (static[3], sets[i][3])):
            a.codes.copy_(b.codes)
            a.scales.copy_(b.scales)
        graph.replay()
        torch.cuda.synchronize()
        for n in FINAL:
            assert torch.equal(r[n], want[i][n]), (i, n)
        chain(*sets[2], k, E, 0, E)  # eager work between the replays
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = chain(*sets[i + 1], k, E, 0, E)
        torch.cuda.synchronize()
        for i in (0, 1):
            for n in FINAL:
                assert torch.equal(got[i][n], want[i + 1][n]), n


def test_pack_into_experts_of_a_longer_array():
    """A checkpoint's experts packed into a view: the whole array has their codes and scales, and a product through a
    captured graph, which holds the array's addresses, sees both."""
    rng = np.random.default_rng(11)
    w, x = values(rng, (4, 128, 256), "bf16"), values(rng, (40, 256), "bf16")
    wc, ws = ref.weights(w)
    whole = moe.quantize_block_weights(dev(values(rng, (4, 128, 256), "bf16"), torch.bfloat16))
    idx = rng.integers(0, 4, 40).astype(np.int32)
    off, ss, _ = ref.sort(idx, 0, 4)
    g, q = moe.sort_tokens(dev(idx.reshape(40, 1)), 4), moe.quantize_block(dev(x, torch.bfloat16))
    moe.block_product(q, whole, g, by_token=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = moe.block_product(q, whole, g, by_token=True)
    for a, b in ((1, 3), (0, 1), (3, 4)):
        moe.pack_block_weights(dev(wc[a:b]), dev(ws[a:b]), out=whole.experts(a, b))
    assert np.array_equal(host(whole.codes), ref.tile(wc)) and np.array_equal(host(whole.scales), ws)
    want = ref.product(*ref.rows(x[ss]), wc, ws, idx[ss])
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(num(y), *want, "replay")
        check(num(moe.block_product(q, whole, g, by_token=True)), *want, "eager")


@pytest.mark.parametrize("D", [24, 4096, 1001])
def test_weights_gradient_in_the_weights_place(D):
    """dw over w itself: the same bits as beside it, for tokens that share a wave and for one over several."""
    rng = np.random.default_rng(D)
    idx = routing("dup", 77, 5, 9, rng)
    g = moe.sort_tokens(dev(idx), 9)
    d, y, w = dev(values(rng, (77, D))), dev(values(rng, (77 * 5, D))), dev(values(rng, (77, 5)))
    dy, dw = moe.combine_backward(g, d, y, w)
    w2 = w.clone()
    dy2, dw2 = moe.combine_backward(g, d, y, w2, dw=w2)
    assert dw2 is w2 and torch.equal(dw, dw2) and torch.equal(dy, dy2)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_values_reach_the_results(bad):
    """A NaN or an infinity makes its block's scale, and every result that the block enters, not finite; all other codes,
    scales and results keep their bits."""
    rng = np.random.default_rng(8)
    idx = exact_counts([200, 100])
    g = moe.sort_tokens(dev(idx.reshape(-1, 1)), 2)
    x, dy, w = values(rng, (300, 384), "bf16"), values(rng, (300, 256), "bf16"), values(rng, (2, 256, 384), "bf16")
    t = lambda a: dev(a, torch.bfloat16)
    put = lambda a, at: t(np.where(np.arange(a.size).reshape(a.shape) == np.ravel_multi_index(at, a.shape), np.float32(bad), a))
    zero = lambda a, at: t(np.where(np.arange(a.size).reshape(a.shape) == np.ravel_multi_index(at, a.shape), np.float32(0), a))

    def same_but(a, b, where, codes=False):
        a, b = num(a) if a.is_floating_point() else host(a), num(b) if b.is_floating_point() else host(b)
        hit = np.zeros(a.shape, bool)
        hit[where] = True
        assert np.array_equal(a[~hit], b[~hit])
        assert codes or not np.isfinite(a[hit]).any()

    wq = moe.quantize_block_weights(t(w))
    # a row's value: row 5 is in block 1 of its row, in the first expert's first run
    (q, c), (q0, c0) = moe.quantize_block_both(put(x, (5, 130)), g), moe.quantize_block_both(zero(x, (5, 130)), g)
    one, one0 = moe.quantize_block(put(x, (5, 130))), moe.quantize_block(zero(x, (5, 130)))
    only = moe.quantize_block_columns(put(x, (5, 130)), g)
    for a, b in ((q, q0), (one, one0)):
        same_but(a.scales[:, :3], b.scales[:, :3], (5, 1))
        same_but(a.codes, b.codes, (1, 5), True)
    runs = [0, 1, 2]  # offsets 0, 200: blocks 0, 1 of the first expert, 200 / 128 + 1 = 2 of the second
    for a in (c, only):
        same_but(a.scales[runs], c0.scales[runs], (0, 130))
        same_but(a.codes[runs], c0.codes[runs], (0, 4, slice(None), slice(None), 2), True)
    same_but(moe.block_product(q, wq, g), moe.block_product(q0, wq, g), 5)
    gq, gc = moe.quantize_block_both(t(dy), g)
    same_but(moe.block_weight_grad(gc, c, g), moe.block_weight_grad(gc, c0, g), (0, slice(None), 130))
    # an output gradient's, in the second expert's rows
    (q, c), (q0, c0) = moe.quantize_block_both(put(dy, (250, 7)), g), moe.quantize_block_both(zero(dy, (250, 7)), g)
    same_but(moe.block_product_grad(q, wq, g), moe.block_product_grad(q0, wq, g), 250)
    same_but(moe.block_weight_grad(c, only, g)[1:], moe.block_weight_grad(c0, only, g)[1:], (0, 7))
    # a token's, seen through its one sorted row
    row = int(np.nonzero(host(g.sorted_slot) == 17)[0][0])
    a, b = (moe.quantize_block_columns(f(x, (17, 200)), g, by_token=True) for f in (put, zero))
    run = row // 128 if row < 200 else 2
    same_but(a.scales[runs], b.scales[runs], (run, 200))
    # few rows: the kernel that streams the weights
    a, b = (moe.block_product(moe.quantize_block(f(x, (5, 130))[:20]), wq.experts(0, 1)) for f in (put, zero))
    same_but(a, b, 5)
    # a weight's
    a, b = (moe.quantize_block_weights(f(w, (1, 200, 300))) for f in (put, zero))
    same_but(a.scales, b.scales, (1, 1, 2))
    same_but(moe.block_product(one0, a, g), moe.block_product(one0, b, g), (slice(200, 300), slice(128, 256)))
    same_but(moe.block_product_grad(gq, a, g), moe.block_product_grad(gq, b, g), (slice(200, 300), slice(256, 384)))


def sorted_by_definition(idx, e0, e1):
    """ref.sort for many slots: a stable sort by expert, what is not local behind."""
    flat = idx.reshape(-1).astype(np.int64) - e0
    n = e1 - e0
    key = np.where((flat >= 0) & (flat < n), flat, n)
    order = np.argsort(key, kind="stable")
    off = np.searchsorted(key[order], np.arange(n + 1))
    S = off[-1]
    ss, sp = np.full(flat.size, -1), np.full(flat.size, -1)
    ss[:S] = order[:S]
    sp[order[:S]] = np.arange(S)
    return off, ss, sp.reshape(idx.shape)


@pytest.mark.parametrize("kind", ["dup", "wild", "hot", "one"])
@pytest.mark.parametrize("T,k,E,e0,e1", [
    (1024, 1, 384, 0, 384), (1025, 1, 384, 0, 384),    # one and two passes of the one workgroup
    (4095, 1, 384, 0, 384), (2048, 2, 384, 0, 384), (4097, 1, 384, 0, 384),  # one launch, two launches
    (2500, 8, 384, 0, 384), (2500, 8, 700, 0, 700), (2500, 8, 1024, 0, 1024), (2500, 8, 1025, 0, 1025),
    (2500, 8, 4096, 1000, 2024), (2500, 8, 65, 0, 65), (4096, 5, 513, 1, 513),
    (33000, 8, 384, 0, 384), (33000, 8, 384, 96, 192), (66001, 8, 1024, 0, 1024)])  # several passes a chunk
def test_sort_of_many_slots(kind, T, k, E, e0, e1):
    """Every branch of the sort by size: passes of a workgroup, one launch or two, threads or waves or all of the
    workgroup holding experts, chunks of more than one pass; against the definition, in full."""
    rng = np.random.default_rng(T + E + e0)
    if kind == "hot":  # most slots on a few experts, the rest anywhere
        idx = np.where(rng.random((T, k)) < 0.9, rng.integers(0, 3, (T, k)) * (E // 3), rng.integers(0, E, (T, k))).astype(np.int32)
    else:
        idx = routing(kind, T, k, E, rng)
    g = moe.sort_tokens(dev(idx), E, e0, e1)
    off, ss, sp = sorted_by_definition(idx, e0, e1)
    assert np.array_equal(host(g.offsets), off) and np.array_equal(host(g.slot_pos), sp) and np.array_equal(host(g.sorted_slot), ss)
    # the tiles of the products, through one: a row's product with its expert's number in the scale
    n = e1 - e0
    w = moe.BlockWeights(n, 128, 128, torch.full((n, 4, 2, 4, 32, 16), 0x38, dtype=torch.uint8, device="cuda"),
                         torch.arange(1, n + 1, device="cuda", dtype=torch.float32).reshape(n, 1, 1))
    x = torch.zeros((T, 128), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    out = torch.full((T * k, 128), -1.0, dtype=torch.bfloat16, device="cuda")
    moe.block_product(moe.quantize_block(x), w, g, by_token=True, out=out)
    S = int(off[-1])
    # 448 times fl32(1 / 448) times e + 1, rounded to bf16: within half a step of each of the three roundings
    want = np.repeat(np.arange(1, n + 1), np.diff(off)).astype(np.float64)
    got = num(out)
    assert (np.abs(got[:S] - want[:, None]) <= want[:, None] * (ref.U_BF16 + 4 * ref.U24)).all() and (got[S:] == -1.0).all()


def test_reference_sorts_agree():
    rng = np.random.default_rng(0)
    for kind in ("dup", "wild", "none"):
        idx = routing(kind, 50, 3, 20, rng)
        for a, b in zip(sorted_by_definition(idx, 4, 15), ref.sort(idx, 4, 15)):
            assert np.array_equal(a, b)


# Root mean square of the difference that a correct product may have; the largest single one (`check`) has room for a
# worst case that sums of ordinary values come nowhere near.
#  - rounding to bf16: for values not placed on purpose the error is spread evenly over half a step h to either side,
#    h^2 / 3 in the mean (10 % for the spread of the sample: over 10^4 values its deviation is under 1 %);
#  - the MFMA drops from each of a block's 128 products less than t = 2^-13 of the largest, the sign that of the product,
#    which is as often positive as negative: 128 t^2 / 3 in the mean at most;
#  - fp32: (blocks + 3) half steps of the sum of magnitudes, as in ops_ref.py, all in one direction.
def rms_check(got, want, size, top2, blocks, what):
    h = np.exp2(np.floor(np.log2(np.maximum(np.abs(want), 1e-30))) - 8)
    mean = 1.1 ** 2 * (h ** 2 / 3).mean() + (128 / 3 * 2.0 ** -26 * top2).mean() + (((blocks + 3) * ref.U24 * size) ** 2).mean()
    err = ((got - want) ** 2).mean()
    assert got.size >= 10000 and err <= mean, f"{what}: rms {np.sqrt(err)}, expected up to {np.sqrt(mean)}"
    assert np.sqrt(mean) <= 2.5e-3 * np.sqrt((want ** 2).mean())   # the bound itself is close to the rounding


@pytest.mark.parametrize("counts,N,K", [([300, 130], 384, 4352), ([300, 130], 256, 128), ([2] * 16, 384, 2176), ([1] * 90, 128, 256),
                                        ([90], 256, 2048), ([513], 512, 1152), ([128, 700], 256, 640)], ids=lambda v: str(v)[:20])
def test_products_in_the_mean(counts, N, K):
    """Product, its transposed form and the weight gradient on normal values, by the root mean square of their errors: a
    factor wrong by a per cent anywhere in a sum shows."""
    rng = np.random.default_rng(N + K + sum(counts))
    T = sum(counts)
    g = moe.sort_tokens(dev(np.repeat(np.arange(len(counts)), counts).astype(np.int32).reshape(T, 1)), len(counts))
    x, dy, w = values(rng, (T, K), "bf16"), values(rng, (T, N), "bf16"), values(rng, (len(counts), N, K), "bf16")
    wq, (wc, ws) = moe.quantize_block_weights(dev(w, torch.bfloat16)), ref.weights(w)
    (xr, xcol), (gr, gcol) = (moe.quantize_block_both(dev(a, torch.bfloat16), g) for a in (x, dy))
    off = np.concatenate([[0], np.cumsum(counts)])

    def product(rows, transposed):
        c, s = ref.rows(rows)
        v = ref.e4m3_value(c) * np.repeat(s.astype(np.float64), 128, 1)
        y, size, top2 = (np.zeros((T, K if transposed else N)) for _ in range(3))
        for e in range(len(counts)):
            at = slice(off[e], off[e + 1])
            we = ref.e4m3_value(wc[e]) * np.repeat(np.repeat(ws[e].astype(np.float64), 128, 0), 128, 1)
            we = we.T if transposed else we
            y[at], size[at] = v[at] @ we.T, np.abs(v[at]) @ np.abs(we).T
            top2[at] = ref.tops(v[at]) ** 2 @ (ref.tops(we) ** 2).T
        return y, size, top2, rows.shape[1] // 128

    rms_check(num(moe.block_product(xr, wq, g)), *product(x, False), "y")
    rms_check(num(moe.block_product_grad(gr, wq, g)), *product(dy, True), "dx")
    if len(counts) == 1:
        rms_check(num(moe.block_product(moe.quantize_block(dev(x, torch.bfloat16)), wq)), *product(x, False), "y without groups")
    got, cg, cx = num(moe.block_weight_grad(gcol, xcol, g)), ref.columns(dy, off), ref.columns(x, off)
    value = lambda q: ref.e4m3_value(q[0].transpose(1, 2, 4, 0, 3).reshape(128, -1)) * q[1].astype(np.float64)
    want, size, top2 = (np.zeros((len(counts), N, K)) for _ in range(3))
    runs = 0
    for b, r0, n in ref.column_blocks(off):
        e = np.searchsorted(off, r0, side="right") - 1
        u, v = value(cg[b]), value(cx[b])
        want[e] += u.T @ v
        size[e] += np.abs(u.T) @ np.abs(v)
        top2[e] += np.outer(np.abs(u).max(0), np.abs(v).max(0)) ** 2
        runs = max(runs, (counts[e] + 127) // 128)
    rms_check(got, want, size, top2, runs, "dw")


def test_rows_past_32_bit_bytes_of_a_plane():
    """2^24 + 1000 rows of one block: their codes lie past 2^31 bytes of the block's plane. The last 1000 rows give the
    bits that they give alone, by every form of the product, and so does a gradient that is zero before them."""
    R, last = 2 ** 24 + 1000, 1000
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x = torch.randn((R, 128), dtype=torch.bfloat16, device="cuda", generator=gen)
    w = moe.quantize_block_weights(torch.randn((1, 128, 128), dtype=torch.bfloat16, device="cuda", generator=gen))
    xs = x[-last:].clone()
    q, q1 = moe.quantize_block(x), moe.quantize_block(xs)
    assert torch.equal(q.codes[:, -last:], q1.codes) and torch.equal(q.scales[-last:, :1], q1.scales[:, :1])
    y = moe.block_product(q, w)
    assert torch.equal(y[-last:], moe.block_product(q1, w))
    g = moe.sort_tokens(torch.zeros((R, 1), dtype=torch.int32, device="cuda"), 1)
    assert torch.equal(moe.block_product(q, w, g, by_token=True), y) and torch.equal(moe.block_product(q, w, g), y)
    assert torch.equal(moe.block_product_grad(q, w)[-last:], moe.block_product_grad(q1, w))
    c, c1 = moe.quantize_block_columns(x), moe.quantize_block_columns(xs)
    assert torch.equal(c.codes[2 ** 24 // 128:], c1.codes) and torch.equal(c.scales[2 ** 24 // 128:], c1.scales)
    both, cb = moe.quantize_block_both(x, g)
    assert torch.equal(both.codes, q.codes) and torch.equal(cb.codes[2 ** 24 // 128:], c1.codes)
    x[:-last] = 0.0
    assert torch.equal(moe.block_weight_grad(moe.quantize_block_columns(x), c, rows=R), moe.block_weight_grad(c1, c1, rows=last))


def test_weight_gradient_of_no_rows():
    """Zeros without groups too; a buffer of no rows has no place that the output could overlap."""
    import ctypes
    from block_scaled_moe_amd import ops
    c = moe.quantize_block_columns(torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda"))
    dw = torch.full((1, 256, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    assert moe.block_weight_grad(c, c, rows=0, out=dw) is dw and not dw.any()
    dw.fill_(7.0)
    at = dw.data_ptr() + 256
    a = ops.MoeBlockWgradArgs(0, 256, 256, None, at, at, at, at, dw.data_ptr())
    ops._call("moe_block_wgrad", dw.device, ctypes.byref(a))
    assert not dw.any()
