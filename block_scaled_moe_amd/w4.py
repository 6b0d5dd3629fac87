"""Grouped products with 4-bit integer weights (include/moe_w4.h): codes 0 .. 15 with a scale, and perhaps a zero point,
for each group of 32, 64 or 128 values along the reduction, as such checkpoints hold them, and bf16 rows.

The functions marshal arguments like ops.py's, and stand between its sort_tokens and combine:

    w1, w2 = pack_w4(codes1, scales1, zeros1), pack_w4(codes2, scales2, zeros2)    # once
    g = sort_tokens(topk_idx, E)
    a = w4_product(h, w1, g, by_token=True, swiglu=True)     # gate and up matrix with the activation
    out = combine(g, w4_product(a, w2, g), topk_w)
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from .ops import DTYPES, Groups, MoeGroups, _ask, _call, _filled, _int32, _out

SCALE_TYPES = {torch.bfloat16: 1, torch.float16: 2}


class MoeW4Weights(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("group", ctypes.c_int32),
                ("scale_type", ctypes.c_int32), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p)]


class MoeW4GemmArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("by_token", ctypes.c_int32), ("swiglu", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("g", ctypes.POINTER(MoeGroups)), ("x", ctypes.c_void_p), ("w", MoeW4Weights),
                ("out", ctypes.c_void_p)]


_P, _I, _Z, _W = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.POINTER(MoeW4Weights)

# every symbol include/moe_w4.h declares, with its ctypes signature
SIGNATURES = {
    "moe_w4_abi_version": ([], _I),
    "moe_w4_code_bytes": ([_W], _Z),
    "moe_w4_scale_bytes": ([_W], _Z),
    "moe_w4_zero_bytes": ([_W], _Z),
    "moe_w4_pack": ([_P, _P, _P, _W, _P], _I),
    "moe_w4_gemm": ([ctypes.POINTER(MoeW4GemmArgs), _P], _I),
}


@dataclasses.dataclass
class W4Weights:
    """Packed weights [E, N, K] = scale * (code - zero): codes int32 [E, N/16, K/256, 2, 64, 4], scales bf16 or fp16
    [E, N/16, K/256, 16, 256/group], zeros uint8 of the scales' shape or None (8 everywhere); divisions rounded up, in the
    order and with the values that include/moe_w4.h gives."""
    E: int
    N: int
    K: int
    group: int
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: torch.Tensor | None

    @staticmethod
    def _shapes(E: int, N: int, K: int, group: int):
        tiles, steps = (N + 15) // 16, (K + 255) // 256
        return (E, tiles, steps, 2, 64, 4), (E, tiles, steps, 16, 256 // group)

    @staticmethod
    def empty(E: int, N: int, K: int, group: int, scale_dtype: torch.dtype = torch.bfloat16, zeros: bool = False,
              device="cuda") -> "W4Weights":
        if group not in (32, 64, 128) or K < 1 or K % group:
            raise ValueError(f"groups of {group} along K = {K}: need 32, 64 or 128, and a multiple of it")
        if scale_dtype not in SCALE_TYPES:
            raise ValueError(f"scales: dtype {scale_dtype}")
        c, s = W4Weights._shapes(E, N, K, group)
        return W4Weights(E, N, K, group, torch.empty(c, dtype=torch.int32, device=device),
                         torch.empty(s, dtype=scale_dtype, device=device),
                         torch.empty(s, dtype=torch.uint8, device=device) if zeros else None)

    def experts(self, e0: int, e1: int) -> "W4Weights":
        """View of experts e0..e1-1."""
        return W4Weights(e1 - e0, self.N, self.K, self.group, self.codes[e0:e1], self.scales[e0:e1],
                         None if self.zeros is None else self.zeros[e0:e1])

    def struct(self, device: torch.device) -> MoeW4Weights:
        for v in (self.E, self.N, self.K):
            _int32("weights", v)
        if self.group not in (32, 64, 128):
            raise ValueError(f"groups of {self.group}: need 32, 64 or 128")
        c, s = self._shapes(self.E, self.N, self.K, self.group)
        _ask("weight codes", self.codes, c, torch.int32, device)
        _ask("weight scales", self.scales, s, SCALE_TYPES, device)
        if self.zeros is not None:
            _ask("weight zeros", self.zeros, s, torch.uint8, device)
        return MoeW4Weights(self.E, self.N, self.K, self.group, SCALE_TYPES[self.scales.dtype], self.codes.data_ptr(),
                            self.scales.data_ptr(), None if self.zeros is None else self.zeros.data_ptr())


def pack_w4(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None,
            out: W4Weights | None = None) -> W4Weights:
    """A checkpoint's row-major arrays -> W4Weights (moe_w4_pack): codes uint8 [E, N, K/2], the even value's code in a
    byte's low half, scales bf16 or fp16 [E, N, K/group], zeros uint8 [E, N, K/group] or None (8 everywhere). The
    group follows from the shapes."""
    if codes.dim() != 3 or scales.dim() != 3:
        raise ValueError(f"codes, scales: shapes {tuple(codes.shape)}, {tuple(scales.shape)}, expected three dimensions")
    E, N, K = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
    groups = scales.shape[2]
    if groups < 1 or K % groups:
        raise ValueError(f"scales: {groups} groups along K = {K}")
    dev = codes.device
    _ask("codes", codes, (E, N, K // 2), torch.uint8, dev)
    _ask("scales", scales, (E, N, groups), SCALE_TYPES, dev)
    if zeros is not None:
        _ask("zeros", zeros, (E, N, groups), torch.uint8, dev)
    if out is None:
        out = W4Weights.empty(E, N, K, K // groups, scales.dtype, zeros is not None, dev)
    if (out.E, out.N, out.K, out.group, out.scales.dtype, out.zeros is None) != (E, N, K, K // groups, scales.dtype, zeros is None):
        raise ValueError("out: weights of another shape or form")
    st = out.struct(dev)
    _call("moe_w4_pack", dev, codes.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(), ctypes.byref(st))
    return out


def w4_product(x: torch.Tensor, w: W4Weights, g: Groups | None = None, by_token: bool = False, swiglu: bool = False,
               out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Each sorted row times its expert's weight, bf16 x [rows, K] -> [T * k, N] in `out`'s dtype or out_dtype (bf16 or fp32);
    with swiglu [T * k, N / 2], silu(first half) * second half (moe_w4_gemm). by_token: x has one row per token. Without
    groups, every row of x times the one expert of w. Rows behind the last local one keep what they hold."""
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected [rows, K]")
    dev = x.device if g is None else g.device
    rows = x.shape[0] if g is None else g.T if by_token else g.rows
    _int32("x", rows)
    _ask("x", x, (rows, w.K), torch.bfloat16, dev)
    if w.E != (1 if g is None else g.n):
        raise ValueError(f"w: {w.E} experts, expected {1 if g is None else g.n}")
    if g is None and by_token:
        raise ValueError("by_token needs groups")
    if swiglu and w.N % 2:
        raise ValueError(f"swiglu: {w.N} columns are not two halves")
    if out is None and out_dtype not in DTYPES:
        raise ValueError(f"out_dtype: {out_dtype}")
    out = _out("out", out, (rows if g is None else g.rows, w.N // 2 if swiglu else w.N), out_dtype if out is None else DTYPES, dev)
    _filled(g)
    a = MoeW4GemmArgs(rows, by_token, swiglu, DTYPES[out.dtype], None if g is None else g.pointer, x.data_ptr(), w.struct(dev),
                      out.data_ptr())
    _call("moe_w4_gemm", dev, ctypes.byref(a))
    return out
