"""The operators of include/moe_w4.h on the GPU against plain forms in 64 bits: packing, and the grouped product with 4-bit
weights at the sizes, groups and routings where it can go wrong; a decode step with sort and combine; graph replays."""
import numpy as np
import pytest
import torch

import block_scaled_moe_amd as moe
import ops_ref
from gpu_util import host

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
U24, U_BF16 = ops_ref.U24, ops_ref.U_BF16


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def num(t):
    return host(t.float() if t.dtype == BF16 else t)


def checkpoint(rng, E, N, K, G, scale=BF16, zeros=False):
    """Row-major codes, scales and zeros on the device, and the values that they stand for (weights, and 32 + code + zero
    times the scale: the size of what the product adds for a value of one) in 64 bits."""
    q = rng.integers(0, 16, (E, N, K)).astype(np.uint8)
    codes = q[:, :, 0::2] | q[:, :, 1::2] << 4
    s = dev((rng.random((E, N, K // G)) * 0.1 + 0.01).astype(np.float32), scale)
    z = rng.integers(0, 16, (E, N, K // G)).astype(np.uint8) if zeros else None
    zz = np.repeat(z, G, 2).astype(np.float64) if zeros else 8.0
    sv = np.repeat(host(s.float()).astype(np.float64), G, 2)
    return dev(codes), s, None if z is None else dev(z), (q - zz) * sv, (32.0 + q + zz) * np.abs(sv)


def expect(x, w, size, G, swiglu, out_bf16):
    """Product of rows with one expert's weights, and how far the operator may be from it: the MFMA's sums, one step (2 U24,
    should it cut off) of what is added for each of a group's values, twice; one product and sum per group and per part."""
    y = x @ w.T
    bound = (2 * G + 8) * 2 * U24 * (np.abs(x) @ size.T) + (x.shape[1] // G + 8) * 2 * U24 * (np.abs(x) @ np.abs(w).T)
    if swiglu:
        n = y.shape[1] // 2
        g, u, eg, eu = y[:, :n], y[:, n:], bound[:, :n], bound[:, n:]
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        y = silu * u
        # the derivative of silu is at most 1.1
        bound = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu) * eu + 16 * U24 * np.abs(y)
    return y, bound + (U_BF16 if out_bf16 else U24) * (np.abs(y) + bound) + 1e-37


def check(got, want, bound, what=""):
    err = np.abs(got - want)
    assert np.isfinite(got).all() and (err <= bound).all(), f"{what}: off by {err.max()}, {(err / bound).max()} of the bound"


@pytest.mark.parametrize("E,N,K,G,zeros", [(1, 1, 32, 32, False), (2, 17, 96, 32, True), (3, 33, 320, 64, False), (1, 48, 512, 128, True), (2, 5, 384, 128, False)])
def test_packing(E, N, K, G, zeros):
    """Against the order that the header gives, word by word."""
    rng = np.random.default_rng(N)
    codes, s, z, _, _ = checkpoint(rng, E, N, K, G, zeros=zeros)
    w = moe.pack_w4(codes, s, z)
    c = host(codes)
    q = np.zeros((E, (N + 15) // 16 * 16, (K + 255) // 256 * 256), np.uint32)
    q[:, :N, 0:K:2], q[:, :N, 1:K:2] = c & 15, c >> 4
    got = host(w.codes).view(np.uint32)
    i, g, j = np.meshgrid(np.arange(16), np.arange(4), np.arange(4), indexing="ij")
    for tile in range(got.shape[1]):
        for step in range(got.shape[2]):
            for half in range(2):
                word = np.zeros((E, 16, 4, 4), np.uint64)
                for m in range(8):
                    v = q[:, 16 * tile + i, 256 * step + 128 * half + 32 * j + 8 * g + m].astype(np.uint64)
                    word |= v << np.uint64(4 * (m // 2) + 16 * (m % 2))
                word = (word << np.uint64(3) | word >> np.uint64(29)) & np.uint64(0xFFFFFFFF)
                assert np.array_equal(got[:, tile, step, half].reshape(E, 4, 16, 4), word.transpose(0, 2, 1, 3).astype(np.uint32))
    per = 256 // G
    for packed, src in ((w.scales, s),) + (((w.zeros, z),) if zeros else ()):
        full = np.zeros((E, q.shape[1], q.shape[2] // G), np.float64)
        full[:, :N, :K // G] = num(src)
        if src is z:
            full = 0x80 + 8 * full
        want = full.reshape(E, -1, 16, q.shape[2] // 256, per).transpose(0, 1, 3, 2, 4)
        assert np.array_equal(num(packed), want)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 64, 65, 130, 300])
@pytest.mark.parametrize("N,K,G,scale,zeros,swiglu,out", [
    (64, 256, 128, BF16, False, False, BF16), (33, 96, 32, FP16, True, False, FP32), (130, 1088, 64, BF16, True, True, BF16),
    (2, 32, 32, BF16, False, True, FP32), (50, 640, 128, FP16, False, True, BF16), (96, 2592, 32, BF16, True, False, BF16),
    (1, 128, 64, BF16, False, False, FP32)])
def test_dense_rows(rows, N, K, G, scale, zeros, swiglu, out):
    rng = np.random.default_rng(rows * N + K)
    codes, s, z, w, size = checkpoint(rng, 1, N, K, G, scale, zeros)
    x = dev(rng.standard_normal((rows, K)).astype(np.float32), BF16)
    y = moe.w4_product(x, moe.pack_w4(codes, s, z), swiglu=swiglu, out_dtype=out)
    assert y.dtype == out and y.shape == (rows, N // 2 if swiglu else N)
    want, bound = expect(num(x).astype(np.float64), w[0], size[0], G, swiglu, out == BF16)
    check(num(y), want, bound)


def routed(rng, T, k, E, kind):
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "wild":
        idx = np.where(rng.random((T, k)) < 0.4, rng.choice(np.array([-1, E, 2 ** 31 - 1, -2 ** 31]), (T, k)), idx).astype(np.int32)
    if kind == "one":
        idx[:] = E // 2
    if kind == "hot":
        idx = np.where(rng.random((T, k)) < 0.8, E // 2, idx).astype(np.int32)
    if kind == "none":
        idx[:] = -1
    return idx


@pytest.mark.parametrize("T,k,E,e0,e1,kind", [(1, 8, 64, 0, 64, "dup"), (1, 1, 4, 1, 2, "dup"), (64, 8, 96, 24, 48, "wild"), (40, 2, 8, 0, 8, "one"), (200, 4, 10, 2, 9, "hot"),
                                              (30, 3, 12, 0, 12, "none"), (700, 2, 5, 0, 5, "dup"), (0, 2, 5, 0, 5, "dup")])
@pytest.mark.parametrize("N,K,G,scale,zeros,swiglu,out", [(96, 384, 128, BF16, False, False, BF16), (70, 160, 32, FP16, True, True, BF16), (34, 576, 64, BF16, True, False, FP32)])
@pytest.mark.parametrize("by_token", [False, True])
def test_grouped(T, k, E, e0, e1, kind, N, K, G, scale, zeros, swiglu, out, by_token):
    rng = np.random.default_rng(T * E + N)
    idx = routed(rng, T, k, E, kind)
    g = moe.sort_tokens(dev(idx), E, e0, e1)
    off, ss, _ = ops_ref.sort(idx, e0, e1)
    S, n = int(off[-1]), e1 - e0
    codes, s, z, w, size = checkpoint(rng, n, N, K, G, scale, zeros)
    x = dev(rng.standard_normal((T if by_token else T * k, K)).astype(np.float32), BF16)
    if not by_token:
        x[S:] = float("nan")  # not read
    C = N // 2 if swiglu else N
    y = torch.full((T * k, C), 77.0, dtype=out, device="cuda")
    assert moe.w4_product(x, moe.pack_w4(codes, s, z), g, by_token=by_token, swiglu=swiglu, out=y) is y
    rows = num(x).astype(np.float64)
    rows = rows[ss[:S] // k] if by_token else rows[:S]
    for e in range(n):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            want, bound = expect(rows[a:b], w[e], size[e], G, swiglu, out == BF16)
            check(num(y)[a:b], want, bound, f"expert {e}")
    assert (num(y)[S:] == 77.0).all()


@pytest.mark.parametrize("T,k,E,e0,e1,kind", [(13000, 3, 1300, 50, 1300, "dup"), (9000, 4, 700, 0, 700, "hot"), (2000, 8, 520, 3, 517, "wild")])
@pytest.mark.parametrize("by_token", [False, True])
def test_many_groups(T, k, E, e0, e1, kind, by_token):
    """More tiles than are brought into order at a time, even and uneven ones."""
    test_grouped(T, k, E, e0, e1, kind, 20, 64, 32, BF16, False, True, BF16, by_token)


@pytest.mark.parametrize("k", [1, 2, 3, 5, 6, 7, 8])
def test_token_of_a_slot(k):
    """Every token's row is its own, for every number of slots a token, in both kernels."""
    T, E = 400, 2
    for t, e in ((40, 40), (T, E)):
        idx = np.arange(t * k, dtype=np.int32).reshape(t, k) % e
        g = moe.sort_tokens(dev(idx), e)
        w = moe.pack_w4(torch.full((e, 16, 192), 0x99, dtype=torch.uint8, device="cuda"), torch.ones((e, 16, 3), dtype=BF16, device="cuda"))
        x = torch.zeros((t, 384), dtype=BF16, device="cuda")
        x[:, 0], x[:, 200] = torch.arange(t) % 16, 256 * torch.arange(t).div(16, rounding_mode="floor") / 16
        y = moe.w4_product(x, w, g, by_token=True, out_dtype=FP32)   # the sum of the row: weights of one
        want = host(g.sorted_slot) // k
        assert np.array_equal(host(y), np.repeat((want % 16 + want // 16 * 16).astype(np.float32)[:, None], 16, 1))


def test_products_in_the_mean():
    """By the root mean square: a scale, zero point or factor that is off by a per cent anywhere shows. The rounding to bf16 is
    spread evenly over half a step h to either side: h^2 / 3 in the mean, 10 % for the sample; the rest is far below it."""
    rng = np.random.default_rng(2)
    for G, zeros in ((32, True), (64, False), (128, True)):
        codes, s, z, w, _ = checkpoint(rng, 1, 512, 2048, G, zeros=zeros)
        for rows in (16, 200):
            x = dev(rng.standard_normal((rows, 2048)).astype(np.float32), BF16)
            y = num(x).astype(np.float64) @ w[0].T
            err = num(moe.w4_product(x, moe.pack_w4(codes, s, z))) - y
            half = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 1e-30))) - 8)
            assert (err ** 2).mean() <= 1.1 ** 2 * (half ** 2 / 3).mean()


def test_rows_do_not_mix():
    """A NaN or an infinity in a row or in a scale stays in the results that it enters."""
    rng = np.random.default_rng(3)
    codes, s, z, _, _ = checkpoint(rng, 2, 64, 256, 64, zeros=True)
    idx = dev(np.array([[0, 1]] * 20, np.int32))
    g = moe.sort_tokens(idx, 2)
    x = dev(rng.standard_normal((20, 256)).astype(np.float32), BF16)
    clean = num(moe.w4_product(x, moe.pack_w4(codes, s, z), g, by_token=True))
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[5, 200] = bad
        got = num(moe.w4_product(y, moe.pack_w4(codes, s, z), g, by_token=True))
        other = [r for r in range(40) if r % 20 != 5]
        assert np.array_equal(got[other], clean[other]) and not np.isfinite(got[[5, 25]]).any()
        t = s.clone()
        t[1, 9, 2] = bad
        got = num(moe.w4_product(x, moe.pack_w4(codes, t, z), g, by_token=True))
        assert not np.isfinite(got[20:, 9]).any()
        got[20:, 9] = clean[20:, 9]
        assert np.array_equal(got, clean)


def test_extreme_codes_and_values():
    """All codes 0 and all 15 with zero points 0 and 15, and rows far from one."""
    for q in (0, 15):
        for zp in (0, 15, None):
            codes = torch.full((1, 40, 64), q * 17, dtype=torch.uint8, device="cuda")
            s = torch.full((1, 40, 2), 0.5, dtype=BF16, device="cuda")
            z = None if zp is None else torch.full((1, 40, 2), zp, dtype=torch.uint8, device="cuda")
            for v in (1.0, 2.0 ** 100, 2.0 ** -90, -3.0):
                x = torch.full((3, 128), v, dtype=BF16, device="cuda")
                want = 128 * v * 0.5 * (q - (8 if zp is None else zp))  # every step of the sums is exact
                assert (num(moe.w4_product(x, moe.pack_w4(codes, s, z), out_dtype=FP32)) == want).all()


def test_views_of_experts_and_packing_again():
    rng = np.random.default_rng(5)
    codes, s, z, _, _ = checkpoint(rng, 6, 40, 320, 32, FP16, True)
    w = moe.pack_w4(codes, s, z)
    x = dev(rng.standard_normal((7, 320)).astype(np.float32), BF16)
    for e in (0, 3, 5):
        alone = moe.pack_w4(codes[e:e + 1].contiguous(), s[e:e + 1].contiguous(), z[e:e + 1].contiguous())
        assert torch.equal(moe.w4_product(x, w.experts(e, e + 1)), moe.w4_product(x, alone))
    kept = w.codes
    moe.pack_w4(codes.flip(0).contiguous(), s.flip(0).contiguous(), z.flip(0).contiguous(), out=w)
    assert w.codes is kept
    first = moe.w4_product(x, w.experts(0, 1))
    assert torch.equal(first, moe.w4_product(x, moe.pack_w4(codes[5:].contiguous(), s[5:].contiguous(), z[5:].contiguous())))


def test_decode_step():
    """route, sort, both products with the activation, combine, for one token and for some, in a graph too."""
    rng = np.random.default_rng(6)
    E, D, F, k, G = 16, 256, 192, 4, 64
    c1, s1, z1, w1, _ = checkpoint(rng, E, 2 * F, D, G, zeros=True)
    c2, s2, z2, w2, _ = checkpoint(rng, E, D, F, G)
    p1, p2 = moe.pack_w4(c1, s1, z1), moe.pack_w4(c2, s2)
    wr = dev(rng.standard_normal((E, D)).astype(np.float32) * 0.1, BF16)
    for T in (1, 20):
        h = dev(rng.standard_normal((T, D)).astype(np.float32), BF16)

        def step():
            idx, w, _, _ = moe.route(h, wr, top_k=k)
            g = moe.sort_tokens(idx, E)
            a = moe.w4_product(h, p1, g, by_token=True, swiglu=True)
            return idx, w, moe.combine(g, moe.w4_product(a, p2, g), w)

        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step()
        for _ in range(3):
            h.copy_(dev(rng.standard_normal((T, D)).astype(np.float32), BF16))
            graph.replay()
            torch.cuda.synchronize()
            kept = [t.clone() for t in captured]
            eager = step()
            assert all(torch.equal(a, b) for a, b in zip(kept, eager))
        idx, w, out = (num(t) for t in eager)
        x = num(h).astype(np.float64)
        want, size = np.zeros((T, D)), np.zeros((T, D))
        for t in range(T):
            for j in range(k):
                y = w1[idx[t, j]] @ x[t]
                a = y[:F] / (1 + np.exp(-y[:F])) * y[F:]
                want[t] += w[t, j] * (w2[idx[t, j]] @ a)
                size[t] += w[t, j] * (np.abs(w2[idx[t, j]]) @ np.abs(a))
        # a and the second product are rounded to bf16, everything else is fp32
        assert (np.abs(out - want) <= (2 * U_BF16 + 2000 * U24) * size).all()


def far(got, want, bound, period, chunk=1 << 17):
    """Rows repeat with a period, and so do their expected values; compared on the device, where they are too many for the host."""
    want, bound = dev(want), dev(bound)
    for i in range(0, len(got), chunk):
        g = got[i:i + chunk].view(-1, period, got.shape[1]).float()
        assert bool(((g - want.float()).abs() <= bound.float() + 2 * U24 * want.float().abs()).all()), f"rows from {i} on"


@pytest.mark.parametrize("rows,N,K", [(2 ** 19 + 320, 16, 4096), (2 ** 20 + 128, 2050, 32)], ids=["rows", "results"])
def test_more_than_32_bits_of_elements(rows, N, K):
    """Rows of x, or of the result, whose elements are numbered past 2^31."""
    rng = np.random.default_rng(8)
    codes, s, _, w, size = checkpoint(rng, 1, N, K, 32)
    x = dev(rng.standard_normal((64, K)).astype(np.float32), BF16)
    y, bound = expect(num(x).astype(np.float64), w[0], size[0], 32, False, True)
    out = torch.full((rows, N), float("nan"), dtype=BF16, device="cuda")
    moe.w4_product(x.repeat(rows // 64, 1), moe.pack_w4(codes, s), out=out)
    far(out, y, bound, 64)


def test_more_than_32_bits_of_codes():
    """Weights of 17 GB, and more column tiles than the grid of a workgroup each can have."""
    E, N, K, T, k = 128, 2 ** 20, 32, 16, 8
    gen = torch.Generator(device="cuda").manual_seed(9)
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = (torch.rand((E, N, 1), device="cuda", generator=gen) * 0.1 + 0.01).to(BF16)
    w = moe.pack_w4(codes, s)
    idx = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0).view(T, k).contiguous()
    x = torch.randn((T, K), device="cuda", generator=gen).to(BF16)
    g = moe.sort_tokens(idx, E)
    out = moe.w4_product(x, w, g, by_token=True)
    for e in (0, 1, 63, 64, 126, 127):
        q = torch.stack((codes[e] & 15, codes[e] >> 4), 2).view(N, K).double()
        v = x[(T * k - 1 - e) // k].double()
        sv = s[e].double()[:, 0]
        y, ay = ((q - 8) @ v) * sv, (((q - 8).abs() @ v.abs()) * sv)
        bound = (2 * K + 8) * 2 * U24 * ((40 + q) @ v.abs()) * sv + (K // 32 + 8) * 2 * U24 * ay  # as in expect
        err = (out[e].double() - y).abs()
        assert bool((err <= bound + U_BF16 * (y.abs() + bound) + 1e-37).all()), f"expert {e}"
