"""The product with 4-bit weights (include/moe_w4.h) on the GPU at the sizes that choose each of its kernels, each form of them and
each turn in them, against 64 bits. What a call takes is worked out beside it from the rules of launch_w4_gemm and launch_w4_tile, so
that a case that no longer reaches its kernel shows."""
import numpy as np
import pytest
import torch

import block_scaled_moe_amd as moe
import ops_ref
from gpu_util import host

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
U24, U_BF16 = ops_ref.U24, ops_ref.U_BF16


def form(T, k, E, n, N, G, swiglu):
    """(kernel, its waves a column tile or its columns of 64, workgroups that share the turns)"""
    C, S = N // 2 if swiglu else N, T * k
    tiles, mean = (min(S, n) + S // 224, S // E) if E else (-(-T // 224), T)
    nb = -(-C // (16 if swiglu else 32))
    if mean > (24 if E else 160) or tiles * nb >= 1 << 22:
        items = (tiles if E else -(-T // 128)) * -(-C // (128 if swiglu else 256))
        return "tile", 2 if G == 32 or (swiglu and C % 16) or items < 512 else 4, 1
    if not E and T > 16:
        return "wide", 8, 1
    return "stream", 1 if tiles * nb > 1024 else 4 if tiles * nb > 320 else 8, 4 if E and T > 64 else 1


def checkpoint(gen, E, N, K, G, scale, zeros):
    r = lambda *s: torch.rand(s, device="cuda", generator=gen)
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    z = torch.randint(0, 16, (E, N, K // G), dtype=torch.uint8, device="cuda", generator=gen) if zeros else None
    return codes, (r(E, N, K // G) * 0.1 + 0.01).to(scale), z


def expect(x, codes, s, z, G, swiglu, out_bf16):
    """Product of rows with one expert's weights in 64 bits, and how far the operator may be from it: the MFMA's sums, one step
    (2 U24, should it cut off) of what is added for each of a group's values, twice; one product and sum per group and per part."""
    q = torch.stack((codes & 15, codes >> 4), 2).flatten(1).double()
    sv = s.double().repeat_interleave(G, 1)
    zv = 8.0 if z is None else z.double().repeat_interleave(G, 1)
    w, size = (q - zv) * sv, (32.0 + q + zv) * sv
    x = x.double()
    y = x @ w.t().contiguous()
    bound = (2 * G + 8) * 2 * U24 * (x.abs() @ size.t().contiguous()) + (x.shape[1] // G + 8) * 2 * U24 * (x.abs() @ w.abs().t().contiguous())
    if swiglu:
        n = y.shape[1] // 2
        g, u, eg, eu = y[:, :n], y[:, n:], bound[:, :n], bound[:, n:]
        silu = g / (1 + torch.exp(-g))
        y = silu * u
        # the derivative of silu is at most 1.1
        bound = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + 16 * U24 * y.abs()
    return y, bound + (U_BF16 if out_bf16 else U24) * (y.abs() + bound) + 1e-37


def routed(rng, T, k, E, kind):
    idx = rng.integers(0, E, (T, k))
    if kind == "wild":
        idx = np.where(rng.random((T, k)) < 0.3, rng.choice(np.array([-1, E, 2 ** 31 - 1, -2 ** 31]), (T, k)), idx)
    if kind == "hot":    # one expert has most rows, some have none
        idx = np.where(rng.random((T, k)) < 0.6, E // 2, rng.integers(0, max(E // 2, 1), (T, k)))
    if kind == "steps":  # every number of rows from 1 on
        idx = np.sort(rng.choice(E, T * k, p=np.arange(1, E + 1) / (E * (E + 1) / 2))).reshape(T, k)
    return torch.from_numpy(idx.astype(np.int32)).cuda()


def run(T, k, E, e0, e1, kind, N, K, G, scale, zeros, swiglu, out, by_token=True):
    rng, gen, n = np.random.default_rng(T + N), torch.Generator(device="cuda").manual_seed(N + K), e1 - e0
    codes, s, z = checkpoint(gen, n, N, K, G, scale, zeros)
    w, C, S = moe.pack_w4(codes, s, z), N // 2 if swiglu else N, T * k
    x = torch.randn((T if by_token else S, K), device="cuda", generator=gen).to(BF16)
    y = torch.full((S, C), 77.0, dtype=out, device="cuda")
    if E:
        g = moe.sort_tokens(routed(rng, T, k, E, kind), E, e0, e1)
        off = host(g.offsets)
        rows = x[(g.sorted_slot[:off[-1]] // k).long()] if by_token else x[:off[-1]]
        moe.w4_product(x, w, g, by_token=by_token, swiglu=swiglu, out=y)
    else:
        off, rows = [0, T], x
        moe.w4_product(x, w, swiglu=swiglu, out=y)
    for e in range(n):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            want, bound = expect(rows[a:b], codes[e], s[e], z if z is None else z[e], G, swiglu, out == BF16)
            err = (y[a:b].double() - want).abs()
            assert bool((err <= bound).all()), f"expert {e}, rows {a} to {b}: {float((err / bound).max())} of the bound"
    assert bool((y[off[-1]:] == 77.0).all())


# ---------------------------------------------------------------- many rows

@pytest.mark.parametrize("T,k,E,kind", [(700, 2, 5, "even"), (500, 3, 3, "even"), (900, 1, 2, "steps"), (300, 8, 10, "hot"), (675, 2, 6, "even")])
@pytest.mark.parametrize("N,K,G,swiglu", [(70, 160, 32, False), (18432, 192, 64, False), (18432, 128, 128, True)])
def test_groups_longer_than_a_tile(T, k, E, kind, N, K, G, swiglu):
    """Groups of several tiles of 224 rows, cut into parts of 128 and 96."""
    assert form(T, k, E, E, N, G, swiglu)[0] == "tile"
    run(T, k, E, 0, E, kind, N, K, G, BF16, True, swiglu, BF16)


WIDE = [  # K of one, two, three and more stages of 128
    (1600, 64, 64, BF16, False, False, BF16), (1605, 192, 64, FP16, True, False, BF16), (1602, 320, 64, BF16, True, False, FP32),
    (1664, 1088, 64, FP16, False, True, BF16), (1600, 320, 64, BF16, True, True, FP32), (1601, 128, 128, FP16, False, False, BF16),
    (1600, 256, 128, BF16, True, False, BF16), (1664, 384, 128, BF16, False, True, BF16), (1632, 640, 128, FP16, True, True, BF16),
    (1700, 1152, 128, BF16, False, False, FP32), (1696, 128, 128, FP16, True, True, FP32), (1603, 1152, 128, FP16, True, False, BF16)]


@pytest.mark.parametrize("T,k,E,e0,e1,kind", [(400, 8, 64, 0, 64, "even"), (900, 8, 128, 40, 104, "wild"), (420, 8, 64, 0, 64, "hot"),
                                              (410, 8, 64, 0, 64, "steps")])
@pytest.mark.parametrize("N,K,G,scale,zeros,swiglu,out", WIDE)
def test_wide_tiles(T, k, E, e0, e1, kind, N, K, G, scale, zeros, swiglu, out):
    """A prompt's product: tiles of 256 columns, with the activation 128 of either half, parts of every number of pieces of 16 rows."""
    assert form(T, k, E, e1 - e0, N, G, swiglu) == ("tile", 4, 1)
    run(T, k, E, e0, e1, kind, N, K, G, scale, zeros, swiglu, out, by_token=K % 3 != 0)


@pytest.mark.parametrize("rows", [700, 3000])
@pytest.mark.parametrize("N,K,G,scale,zeros,swiglu,out", [(21888, 320, 64, BF16, True, False, BF16), (25600, 256, 128, FP16, False, True, BF16)])
def test_wide_tiles_of_one_weight(rows, N, K, G, scale, zeros, swiglu, out):
    assert form(rows, 1, 0, 1, N, G, swiglu) == ("tile", 4, 1)
    run(rows, 1, 0, 0, 1, "", N, K, G, scale, zeros, swiglu, out)


# ---------------------------------------------------------------- few rows

FORMS = [(G, scale, zeros, swiglu, out) for G, scale, zeros, swiglu, out in (
    (32, BF16, False, False, BF16), (32, FP16, True, True, BF16), (64, FP16, False, True, FP32), (64, BF16, True, False, BF16),
    (128, BF16, False, False, BF16), (128, BF16, False, True, BF16), (128, FP16, True, False, FP32))]


@pytest.mark.parametrize("waves,N,K", [(8, 126, 2688), (4, 442, 1152), (4, 446, 128), (1, 2050, 1152), (1, 2054, 2048), (1, 522, 384)])
@pytest.mark.parametrize("T,kind", [(64, "even"), (64, "hot"), (60, "steps"), (100, "even"), (110, "hot"), (180, "wild"), (190, "steps")])
@pytest.mark.parametrize("G,scale,zeros,swiglu,out", FORMS)
def test_few_rows_a_group(waves, N, K, T, kind, G, scale, zeros, swiglu, out):
    """Each number of waves that share a column tile; turns of up to 16 rows and (one wave, groups of 64 or 128 without zero points)
    of 32, several for the hot expert and several parts of the reduction in LDS; one or four workgroups that share the turns."""
    k, E = 8, 64
    if swiglu:
        N += N % 2
    assert form(T, k, E, E, N, G, swiglu) == ("stream", waves, 4 if T > 64 else 1)
    run(T, k, E, 0, E, kind, N, K, G, scale, zeros, swiglu, out, by_token=T % 20 == 0 or T == 64)


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("N,K,G,scale,zeros,swiglu", [(4096, 2560, 128, BF16, False, False), (1344, 1536, 32, FP16, True, True), (5101, 640, 64, BF16, True, False)])
def test_one_token(T, N, K, G, scale, zeros, swiglu):
    """Eight experts, some with the same row twice."""
    assert form(T, 8, 64, 64, N, G, swiglu) == ("stream", 4 if T * 8 * -(-N // 32) <= 1024 else 1, 1)
    run(T, 8, 64, 0, 64, "even", N, K, G, scale, zeros, swiglu, BF16)


@pytest.mark.parametrize("rows", [1, 5, 16])
@pytest.mark.parametrize("waves,N", [(8, 4100), (4, 16400), (1, 131110)])
@pytest.mark.parametrize("K,G,scale,zeros,swiglu,out", [(96, 32, BF16, True, False, BF16), (640, 128, FP16, False, True, BF16), (2112, 64, BF16, False, False, FP32)])
def test_few_rows_of_one_weight(rows, waves, N, K, G, scale, zeros, swiglu, out):
    assert form(rows, 1, 0, 1, N, G, swiglu) == ("stream", waves, 1)
    run(rows, 1, 0, 0, 1, "", N, K, G, scale, zeros, swiglu, out)


@pytest.mark.parametrize("rows", [17, 32, 33, 64, 65, 97, 128, 129, 160])
@pytest.mark.parametrize("N,K,G,scale,zeros,swiglu,out", [
    (67, 96, 32, FP16, True, False, BF16), (130, 2592, 32, BF16, False, True, BF16), (96, 1088, 64, BF16, True, True, FP32), (101, 640, 64, FP16, False, False, FP32),
    (64, 256, 128, BF16, True, False, BF16), (2, 128, 128, FP16, False, True, BF16)])
def test_some_rows_of_one_weight(rows, N, K, G, scale, zeros, swiglu, out):
    assert form(rows, 1, 0, 1, N, G, swiglu) == ("wide", 8, 1)
    run(rows, 1, 0, 0, 1, "", N, K, G, scale, zeros, swiglu, out)
