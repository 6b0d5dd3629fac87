"""Plain 64-bit forms of the operators of include/moe_ops.h, in numpy on the host, written from
their definitions: the tests' expected values."""
from __future__ import annotations

import numpy as np

U24 = 2.0 ** -24   # half a step of fp32, relative
U_BF16 = 2.0 ** -8  # half a step of bf16, relative (its largest)
# A block's sum of 128 E4M3 products in the FP8 MFMA: it brings the products it adds to the
# exponent of the largest of them and drops what lies more than 13 bits below that
# (test_gpu_ops.py measures it), so each of the 128 is off by less than 2^-13 of the largest.
MFMA = 128 * 2.0 ** -13


def bf16(x: np.ndarray) -> np.ndarray:
    """fp32 values rounded to bf16 (nearest, ties to even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return u.astype(np.uint32).view(np.float32).reshape(np.shape(x))


def e4m3_code(v: np.ndarray) -> np.ndarray:
    """Nearest E4M3 code of fp32 values, ties to even, saturating at 448."""
    a = np.abs(v.astype(np.float64))
    e = np.maximum(np.frexp(np.maximum(a, 2.0 ** -30))[1] - 1, -6)
    q = np.rint(np.ldexp(a, 3 - e))                      # in units of 2^(e - 3): np.rint ties to even
    e, q = np.where(q == 16, e + 1, e), np.where(q == 16, 8, q)
    code = np.where(q < 8, q, (e + 7) * 8 + q - 8)       # q < 8 only at e = -6: subnormal
    code = np.where(a >= 464, 0x7E, np.minimum(code, 0x7E)).astype(np.uint8)
    return code | (np.signbit(v).astype(np.uint8) << 7)


def e4m3_value(c: np.ndarray) -> np.ndarray:
    c = c.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, np.ldexp(1.0 + m / 8.0, e - 7))
    return np.where(c & 0x80, -v, v)


def scale_of(amax: np.ndarray) -> np.ndarray:
    amax = np.asarray(amax, np.float32)
    return np.where(amax > 0, amax / np.float32(448.0), np.float32(1.0)).astype(np.float32)


def quantise(x: np.ndarray, axes) -> tuple[np.ndarray, np.ndarray]:
    """(codes, scales) of x with one scale over `axes`; scales keep them as 1."""
    x = np.asarray(x, np.float32)
    s = scale_of(np.abs(x).max(axis=axes, keepdims=True))
    return e4m3_code(x / s), s


def rows(x: np.ndarray):
    R, C = x.shape
    c, s = quantise(x.reshape(R, C // 128, 128), (2,))
    return c.reshape(R, C), s.reshape(R, C // 128)


def weights(w: np.ndarray):
    E, N, K = w.shape
    c, s = quantise(w.reshape(E, N // 128, 128, K // 128, 128), (2, 4))
    return c.reshape(E, N, K), s.reshape(E, N // 128, K // 128)


def tile(codes: np.ndarray) -> np.ndarray:
    """Row-major codes [E, N, K] -> [E, N/32, K/64, 4, 32, 16]."""
    E, N, K = codes.shape
    return np.ascontiguousarray(codes.reshape(E, N // 32, 32, K // 64, 4, 16).transpose(0, 1, 3, 4, 2, 5))


def column_blocks(offsets: np.ndarray):
    """(block, first row, rows) of every run of 128 rows of every expert."""
    for e in range(len(offsets) - 1):
        o, cnt = int(offsets[e]), int(offsets[e + 1] - offsets[e])
        for i in range((cnt + 127) // 128):
            yield o // 128 + e + i, o + 128 * i, min(128, cnt - 128 * i)


def columns(x: np.ndarray, offsets: np.ndarray):
    """{block: (codes [C/32, 2, 4, 32, 16], scales [C])} of sorted rows x."""
    got = {}
    C = x.shape[1]
    for b, r0, n in column_blocks(offsets):
        run = np.zeros((128, C), np.float32)
        run[:n] = x[r0:r0 + n]
        c, s = quantise(run, (0,))
        got[b] = (c.reshape(2, 4, 16, C // 32, 32).transpose(3, 0, 1, 4, 2), s.reshape(C))
    return got


def sort(idx: np.ndarray, e0: int, e1: int):
    """offsets, sorted_slot (-1 behind), slot_pos by the definition: slots in order of (expert, slot)."""
    flat = idx.reshape(-1).astype(np.int64)
    n = e1 - e0
    order = sorted((int(e) - e0, s) for s, e in enumerate(flat) if e0 <= e < e1)
    counts = np.zeros(n, np.int64)
    slot_pos = np.full(flat.size, -1, np.int64)
    sorted_slot = np.full(flat.size, -1, np.int64)
    for p, (e, s) in enumerate(order):
        counts[e] += 1
        slot_pos[s] = p
        sorted_slot[p] = s
    return np.concatenate([[0], np.cumsum(counts)]), sorted_slot, slot_pos.reshape(idx.shape)


def tops(v: np.ndarray) -> np.ndarray:
    """Largest |value| of each block of 128 of the rows of v."""
    return np.abs(v).reshape(v.shape[0], -1, 128).max(2)


def product(xc, xs, wc, ws, expert_of_row, transposed=False):
    """y in fp64 and how far the operator's bf16 result may be from it, for sorted rows of codes xc and row-major
    weight codes."""
    x = e4m3_value(xc) * np.repeat(xs.astype(np.float64), 128, axis=1)
    C = wc.shape[2] if transposed else wc.shape[1]
    y, bound = np.zeros((x.shape[0], C)), np.zeros((x.shape[0], C))
    for e in range(wc.shape[0]):
        at = np.nonzero(expert_of_row == e)[0]
        if len(at):
            w = e4m3_value(wc[e]) * np.repeat(np.repeat(ws[e].astype(np.float64), 128, 0), 128, 1)
            w = w.T if transposed else w
            y[at] = x[at] @ w.T
            bound[at] = product_bound(y[at], np.abs(x[at]) @ np.abs(w).T, tops(x[at]) @ tops(w).T, x.shape[1] // 128)
    return y, bound


def weight_grad(cg, cx, off, e):
    """(dw[e], bound) from the column forms {block: (codes, scales)} of the output gradient and of the input."""
    N, K = next(iter(cg.values()))[1].size, next(iter(cx.values()))[1].size
    want, size, top, runs = np.zeros((N, K)), np.zeros((N, K)), np.zeros((N, K)), 0
    for b, r0, n in column_blocks(off):
        if off[e] <= r0 < off[e + 1]:
            value = lambda q: e4m3_value(q[0].transpose(1, 2, 4, 0, 3).reshape(128, -1)) * q[1].astype(np.float64)
            u, v = value(cg[b]), value(cx[b])
            want += u.T @ v
            size += np.abs(u.T) @ np.abs(v)
            top += np.outer(np.abs(u).max(0), np.abs(v).max(0))
            runs += 1
    return want, product_bound(want, size, top, runs)


def product_bound(y, size, top, blocks):
    """How far the operator's bf16 result may be from y, a sum of terms of total size `size`, `top` the sum over
    the blocks of a bound of the block's largest term: the block sums in the MFMA, a product of scales and a
    multiply-add per block in fp32 (each at most half a step of a sum that is at most `size`), and the rounding."""
    fp32 = MFMA * top + (blocks + 3) * U24 * size
    return fp32 + U_BF16 * (np.abs(y) + fp32) + 1e-38
