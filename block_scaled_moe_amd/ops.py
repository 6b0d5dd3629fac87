"""Operators around the routed-expert layer (include/moe_ops.h): tokens grouped by expert and
back, and the expert product in FP8 with a scale for each block of 128, each with its gradient.

The functions marshal arguments like the package's other calls: torch provides device memory
and the current stream of the tensors' device, every step runs in the library's kernels, and an
argument the library refuses raises MoeError. Wrong dtypes, shapes, devices or strides raise
ValueError before the call; tensors are contiguous. Autograd does not see these calls: each gradient is a
call of its own, and a tensor with requires_grad is refused unless gradients are off (torch.no_grad).

    g = sort_tokens(topk_idx, E)                       # after route()
    y = block_product(quantize_block(x), w, g, by_token=True)      # rows [T * k, N], sorted
    out = combine(g, y, topk_w)

Arrays of sorted rows have T * top_k rows; rows behind the last local one keep what they hold.
As with torch's own operators, a tensor (or Groups.buffer) that is used on another stream than its
own needs record_stream before it is freed.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools

import torch

DTYPES = {torch.bfloat16: 1, torch.float32: 2}


class MoeGroups(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("top_k", ctypes.c_int32), ("E", ctypes.c_int32), ("e_begin", ctypes.c_int32),
                ("e_end", ctypes.c_int32), ("offsets", ctypes.c_void_p), ("sorted_slot", ctypes.c_void_p),
                ("slot_pos", ctypes.c_void_p), ("plan", ctypes.c_void_p), ("plan_bytes", ctypes.c_size_t)]


class MoeBlockWeights(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


class MoeBlockQuantizeArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("C", ctypes.c_int32), ("by_token", ctypes.c_int32),
                ("g", ctypes.POINTER(MoeGroups)), ("x", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("col_codes", ctypes.c_void_p), ("col_scales", ctypes.c_void_p)]


class MoeBlockGemmArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("by_token", ctypes.c_int32), ("transposed", ctypes.c_int32),
                ("g", ctypes.POINTER(MoeGroups)), ("x_codes", ctypes.c_void_p), ("x_scales", ctypes.c_void_p),
                ("w", MoeBlockWeights), ("out", ctypes.c_void_p)]


class MoeBlockWgradArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("g", ctypes.POINTER(MoeGroups)), ("g_codes", ctypes.c_void_p), ("g_scales", ctypes.c_void_p),
                ("x_codes", ctypes.c_void_p), ("x_scales", ctypes.c_void_p), ("dw", ctypes.c_void_p)]


_G, _P, _I = ctypes.POINTER(MoeGroups), ctypes.c_void_p, ctypes.c_int32

# every symbol include/moe_ops.h declares, with its ctypes signature
SIGNATURES = {
    "moe_ops_abi_version": ([], _I),
    "moe_groups_plan_bytes": ([_G], ctypes.c_size_t),
    "moe_sort": ([_G, _P, _P], _I),
    "moe_gather": ([_G, _I, _I, _P, _P, _P], _I),
    "moe_gather_backward": ([_G, _I, _I, _P, _P, _P], _I),
    "moe_combine": ([_G, _I, _I, _I, _P, _P, _P, _P], _I),
    "moe_combine_backward": ([_G, _I, _I, _I, _P, _P, _P, _P, _P, _P], _I),
    "moe_block_column_blocks": ([_I, _I], ctypes.c_int64),
    "moe_block_quantize": ([ctypes.POINTER(MoeBlockQuantizeArgs), _P], _I),
    "moe_block_quantize_weights": ([_P, _I, _I, _I, _P, _P, _P], _I),
    "moe_block_pack_weights": ([_P, _I, _I, _I, _P, _P], _I),
    "moe_block_gemm": ([ctypes.POINTER(MoeBlockGemmArgs), _P], _I),
    "moe_block_wgrad": ([ctypes.POINTER(MoeBlockWgradArgs), _P], _I),
}


_FN: dict = {}  # the library's functions by name, once loaded


def _function(name: str):
    fn = _FN.get(name)
    if fn is None:
        from . import lib
        fn = _FN[name] = getattr(lib(), name)
    return fn


def _call(name: str, device: torch.device, *args):
    """The library's entry point `name` on the current stream of `device`, made current for the call."""
    fn = _FN.get(name) or _function(name)
    i = device.index
    if i is None:
        raise ValueError(f"{name}: tensors on {device}, expected a GPU")
    if i == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(i):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if rc:
        from . import MoeError
        raise MoeError(name, rc)


def _int32(what: str, v: int):
    """ctypes passes the low 32 bits of a larger number on."""
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{what}: {v} does not fit 32 bits")


def _ask(what: str, t: torch.Tensor, shape: tuple, dtype, device: torch.device):
    """t has this shape, dtype (one or a collection of them) and device, is contiguous, and autograd does not follow it."""
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype and (isinstance(dtype, torch.dtype) or t.dtype not in dtype):
        raise ValueError(f"{what}: dtype {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: not contiguous")
    if t.requires_grad and torch.is_grad_enabled():  # the result would have no history, and the gradient be lost
        raise ValueError(f"{what}: asks autograd for a gradient; detach it, and use the operators' own gradients")
    return t


def _out(what: str, out: torch.Tensor | None, shape: tuple, dtype, device: torch.device):
    return torch.empty(shape, dtype=dtype, device=device) if out is None else _ask(what, out, shape, dtype, device)


# ------------------------------------------------------------------ tokens by expert

class _once:
    """A property computed at its first use and kept as the object's attribute (functools' takes a lock)."""

    def __init__(self, f):
        self.f, self.__doc__ = f, f.__doc__

    def __set_name__(self, owner, name):
        self.name = name

    def __get__(self, obj, owner=None):
        if obj is None:
            return self
        v = obj.__dict__[self.name] = self.f(obj)
        return v


class Groups:
    """The token-slots of a batch sorted by expert (moe_groups; filled by sort_tokens). Its arrays share one
    allocation; offsets, sorted_slot and slot_pos are views of it."""

    def __init__(self, T: int, top_k: int, E: int, e_begin: int = 0, e_end: int | None = None, device="cuda"):
        e_end = E if e_end is None else e_end
        self.T, self.top_k, self.E, self.e_begin, self.e_end = T, top_k, E, e_begin, e_end
        self.n, self.rows = e_end - e_begin, T * top_k
        self._at = _groups_layout(T, top_k, E, e_begin, e_end)
        slots, pos, plan, end = self._at
        self.buffer = torch.empty(end // 4, dtype=torch.int32, device=device)
        self.device = self.buffer.device
        self.filled = False  # by sort_tokens
        base = self.buffer.data_ptr()
        self.struct = MoeGroups(T, top_k, E, e_begin, e_end, base, base + slots, base + pos, base + plan, end - plan)
        self.ref = ctypes.byref(self.struct)

    @_once
    def pointer(self):
        return ctypes.pointer(self.struct)

    @staticmethod
    def empty(T: int, top_k: int, E: int, e_begin: int = 0, e_end: int | None = None, device="cuda") -> "Groups":
        return Groups(T, top_k, E, e_begin, e_end, device)

    @_once
    def offsets(self) -> torch.Tensor:
        """int32 [n + 1]: first sorted row of each local expert; [n] = local slots."""
        return self.buffer.as_strided((self.n + 1,), (1,), 0)

    @_once
    def sorted_slot(self) -> torch.Tensor:
        """int32 [T * top_k]: slot of each sorted row, -1 behind the local ones."""
        return self.buffer.as_strided((self.rows,), (1,), self._at[0] // 4)

    @_once
    def slot_pos(self) -> torch.Tensor:
        """int32 [T, top_k]: sorted row of each slot, -1 if not local."""
        return self.buffer.as_strided((self.T, self.top_k), (self.top_k, 1), self._at[1] // 4)


@functools.lru_cache(maxsize=256)
def _groups_layout(T: int, top_k: int, E: int, e_begin: int, e_end: int) -> tuple[int, int, int, int]:
    """Byte offsets of sorted_slot, slot_pos and the plan behind offsets, and the total, each a multiple of 256."""
    from . import MoeError
    for v in (T, top_k, E, e_begin, e_end):
        _int32("groups", v)
    st = MoeGroups(T, top_k, E, e_begin, e_end)
    n_plan = int(_function("moe_groups_plan_bytes")(ctypes.byref(st)))
    if n_plan == 0:
        raise MoeError("moe_groups_plan_bytes", -1)
    up = lambda b: (b + 255) // 256 * 256
    slots = up(4 * (e_end - e_begin + 1))
    pos = slots + up(4 * T * top_k)
    plan = pos + up(4 * T * top_k)
    return slots, pos, plan, plan + n_plan


def sort_tokens(topk_idx: torch.Tensor, E: int, e_begin: int = 0, e_end: int | None = None,
                out: Groups | None = None) -> Groups:
    """topk_idx int32 [T, k] -> Groups (moe_sort). Experts outside [e_begin, e_end), such as -1
    for padding, have no row. `out`: groups of the same sizes to fill again."""
    if topk_idx.dim() != 2:
        raise ValueError(f"topk_idx: shape {tuple(topk_idx.shape)}, expected [T, k]")
    T, k = topk_idx.shape
    _ask("topk_idx", topk_idx, (T, k), torch.int32, topk_idx.device)
    e_end = E if e_end is None else e_end
    if out is None:
        out = Groups.empty(T, k, E, e_begin, e_end, device=topk_idx.device)
    elif (out.T, out.top_k, out.E, out.e_begin, out.e_end, out.device) != (T, k, E, e_begin, e_end, topk_idx.device):
        raise ValueError("out: groups of other sizes or on another device")
    _call("moe_sort", out.device, out.ref, topk_idx.data_ptr())
    out.filled = True
    return out


def _filled(g: Groups | None):
    if g is not None and not g.filled:
        raise ValueError("groups that sort_tokens has not filled")


def _row_width(what: str, t: torch.Tensor) -> int:
    if t.dim() != 2:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected [rows, D]")
    rows, D = t.shape
    if rows >= 2 ** 31 or D >= 2 ** 31:
        _int32(what, max(rows, D))
    return D


def gather(g: Groups, x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Token rows x [T, D] (bf16 or fp32) -> sorted rows [T * k, D] (moe_gather)."""
    D = _row_width("x", x)
    _ask("x", x, (g.T, D), DTYPES, g.device)
    out = _out("out", out, (g.rows, D), x.dtype, g.device)
    _filled(g)
    _call("moe_gather", g.device, g.ref, DTYPES[x.dtype], D, x.data_ptr(), out.data_ptr())
    return out


def gather_backward(g: Groups, d_rows: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of gather: d_rows [T * k, D] -> dx [T, D], the sum over each token's local rows."""
    D = _row_width("d_rows", d_rows)
    _ask("d_rows", d_rows, (g.rows, D), DTYPES, g.device)
    out = _out("out", out, (g.T, D), d_rows.dtype, g.device)
    _filled(g)
    _call("moe_gather_backward", g.device, g.ref, DTYPES[d_rows.dtype], D, d_rows.data_ptr(),
          out.data_ptr())
    return out


def combine(g: Groups, y: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None,
            out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Sorted rows y [T * k, D] and weights w fp32 [T, k] -> out [T, D], each token's weighted sum over its
    local slots (moe_combine). `out`'s dtype, or out_dtype, is bf16 or fp32."""
    D = _row_width("y", y)
    _ask("y", y, (g.rows, D), DTYPES, g.device)
    _ask("w", w, (g.T, g.top_k), torch.float32, g.device)
    if out is None and out_dtype not in DTYPES:
        raise ValueError(f"out_dtype: {out_dtype}")
    out = _out("out", out, (g.T, D), out_dtype if out is None else DTYPES, g.device)
    _filled(g)
    _call("moe_combine", g.device, g.ref, DTYPES[y.dtype], DTYPES[out.dtype], D, y.data_ptr(),
          w.data_ptr(), out.data_ptr())
    return out


def combine_backward(g: Groups, d_out: torch.Tensor, y: torch.Tensor, w: torch.Tensor, dy: torch.Tensor | None = None,
                     dw: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of combine: d_out [T, D] -> (dy [T * k, D] in y's dtype, dw fp32 [T, k])."""
    D = _row_width("y", y)
    _ask("y", y, (g.rows, D), DTYPES, g.device)
    _ask("w", w, (g.T, g.top_k), torch.float32, g.device)
    _ask("d_out", d_out, (g.T, D), DTYPES, g.device)
    dy = _out("dy", dy, (g.rows, D), y.dtype, g.device)
    dw = _out("dw", dw, (g.T, g.top_k), torch.float32, g.device)
    _filled(g)
    _call("moe_combine_backward", g.device, g.ref, DTYPES[y.dtype], DTYPES[d_out.dtype], D,
          d_out.data_ptr(), y.data_ptr(), w.data_ptr(), dy.data_ptr(), dw.data_ptr())
    return dy, dw


# ------------------------------------------------------------------ FP8 with a scale per block of 128

class _Quantised:
    """Codes and scales: either two tensors given, or one allocation of which they are views, made when asked for."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        self.codes, self.scales, self.buffer = codes, scales, None

    @classmethod
    def empty(cls, rows: int, C: int, device: torch.device):
        """Room for `rows` rows (of the column form: blocks) of C columns on `device`."""
        q = cls.__new__(cls)
        q.rows, q.C, q.device = rows, C, device
        n, m = cls.sizes(rows, C)
        q.split = (n + 255) // 256 * 256
        q.buffer = torch.empty(q.split + 4 * m, dtype=torch.uint8, device=device)
        return q

    @_once
    def codes(self) -> torch.Tensor:
        n, _ = self.sizes(self.rows, self.C)
        return self.buffer[:n].view(self.shapes(self.rows, self.C)[0])

    @_once
    def scales(self) -> torch.Tensor:
        return self.buffer[self.split:].view(torch.float32).view(self.shapes(self.rows, self.C)[1])

    def place(self) -> torch.device:
        """Device of the codes."""
        return self.codes.device if "codes" in self.__dict__ else self.device

    def pointers(self, what: str, rows: int, C: int, device: torch.device) -> tuple[int, int]:
        """Addresses of codes and scales, which hold `rows` rows of C columns on `device`."""
        own = self.__dict__
        if "codes" not in own and "scales" not in own:  # nobody has set them: as allocated
            if (self.rows, self.C, self.device) != (rows, C, device):
                raise ValueError(f"{what}: {self.rows} x {self.C} on {self.device}, expected {rows} x {C} on {device}")
            base = self.buffer.data_ptr()
            return base, base + self.split
        codes, scales = self.shapes(rows, C)
        return (_ask(what + " codes", self.codes, codes, torch.uint8, device).data_ptr(),
                _ask(what + " scales", self.scales, scales, torch.float32, device).data_ptr())


class BlockRows(_Quantised):
    """Rows in E4M3 with an fp32 scale per 1 x 128 block: codes uint8 [C / 128, rows, 128], scales
    [rows, S], S being C / 128 rounded up to a multiple of 4 (the rest is unused)."""

    @property
    def height(self) -> int:
        if "codes" not in self.__dict__:
            return self.rows
        if self.codes.dim() != 3:
            raise ValueError(f"x codes: shape {tuple(self.codes.shape)}, expected [blocks, rows, 128]")
        return self.codes.shape[1]

    @staticmethod
    def sizes(rows: int, C: int):
        return rows * C, rows * ((C // 128 + 3) // 4 * 4)

    @staticmethod
    def shapes(rows: int, C: int):
        return (C // 128, rows, 128), (rows, (C // 128 + 3) // 4 * 4)


class BlockColumns(_Quantised):
    """Sorted rows in E4M3 with an fp32 scale per column of each run of 128 rows of an expert (the column
    form of include/moe_ops.h): codes uint8 [blocks, C / 32, 2, 4, 32, 16], scales [blocks, C]."""
    height = None  # rows of the one group that it was made from, where known on the host

    @property
    def width(self) -> int:
        return self.scales.shape[-1] if "scales" in self.__dict__ else self.C

    @staticmethod
    def sizes(blocks: int, C: int):
        return blocks * C * 128, blocks * C

    @staticmethod
    def shapes(blocks: int, C: int):
        return (blocks, C // 32, 2, 4, 32, 16), (blocks, C)


def _ask_form(what: str, q, form):
    """One form's allocation is too small for the other's reads."""
    if not isinstance(q, form):
        raise ValueError(f"{what}: {type(q).__name__}, expected {form.__name__}")


@dataclasses.dataclass
class BlockWeights:
    """Expert weights [E, N, K] in E4M3 with an fp32 scale per 128 x 128 block: codes uint8
    [E, N/32, K/64, 4, 32, 16] (the tiled layout of moe.h's FP8 weights), scales [E, N/128, K/128]."""
    E: int
    N: int
    K: int
    codes: torch.Tensor
    scales: torch.Tensor

    @staticmethod
    def empty(E: int, N: int, K: int, device="cuda") -> "BlockWeights":
        if N % 128 or K % 128:
            raise ValueError(f"block weights need N and K in multiples of 128 (got N={N}, K={K})")
        return BlockWeights(E, N, K, torch.empty((E, N // 32, K // 64, 4, 32, 16), dtype=torch.uint8, device=device),
                            torch.empty((E, N // 128, K // 128), dtype=torch.float32, device=device))

    def experts(self, e0: int, e1: int) -> "BlockWeights":
        """View of experts e0..e1-1."""
        return BlockWeights(e1 - e0, self.N, self.K, self.codes[e0:e1], self.scales[e0:e1])

    def struct(self, device: torch.device) -> MoeBlockWeights:
        E, N, K = self.E, self.N, self.K
        _ask("weight codes", self.codes, (E, N // 32, K // 64, 4, 32, 16), torch.uint8, device)
        _ask("weight scales", self.scales, (E, N // 128, K // 128), torch.float32, device)
        return MoeBlockWeights(E, N, K, self.codes.data_ptr(), self.scales.data_ptr())


def quantize_block_weights(w: torch.Tensor, out: BlockWeights | None = None) -> BlockWeights:
    """bf16 weights [E, N, K] -> BlockWeights (moe_block_quantize_weights)."""
    if w.dim() != 3:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected [E, N, K]")
    E, N, K = w.shape
    _ask("w", w, (E, N, K), torch.bfloat16, w.device)
    out = BlockWeights.empty(E, N, K, device=w.device) if out is None else out
    if (out.E, out.N, out.K) != (E, N, K):
        raise ValueError("out: weights of another shape")
    st = out.struct(w.device)
    _call("moe_block_quantize_weights", w.device, w.data_ptr(), E, N, K, st.codes, st.scales)
    return out


def pack_block_weights(codes: torch.Tensor, scales: torch.Tensor, out: BlockWeights | None = None) -> BlockWeights:
    """A checkpoint's E4M3 codes (uint8 or float8_e4m3fn [E, N, K], row-major) and fp32 scales
    [E, N/128, K/128] -> BlockWeights (moe_block_pack_weights). Without `out` the weights hold `scales` itself;
    with it, the scales are copied into its buffer like the codes."""
    if codes.dim() != 3:
        raise ValueError(f"codes: shape {tuple(codes.shape)}, expected [E, N, K]")
    E, N, K = codes.shape
    _ask("codes", codes, (E, N, K), (torch.uint8, torch.float8_e4m3fn), codes.device)
    _ask("scales", scales, (E, N // 128, K // 128), torch.float32, codes.device)
    if out is None:
        out = BlockWeights.empty(E, N, K, device=codes.device)
        out.scales = scales
    if (out.E, out.N, out.K) != (E, N, K):
        raise ValueError("out: weights of another shape")
    st = out.struct(codes.device)
    _call("moe_block_pack_weights", codes.device, codes.data_ptr(), E, N, K, st.codes)
    if out.scales is not scales:
        out.scales.copy_(scales)
    return out


def _blocks_of_128(what: str, C: int):
    if C % 128 or C < 128:
        raise ValueError(f"{what}: {C} columns are not a multiple of 128")


def _quantize(x: torch.Tensor, g: Groups | None, by_token: bool, rows: bool, columns: bool):
    C = _row_width("x", x)
    _blocks_of_128("x", C)
    dev = x.device if g is None else g.device
    R = x.shape[0] if g is None else g.T if by_token else g.rows
    _ask("x", x, (R, C), torch.bfloat16, dev)
    r = c = None
    rc = rs = cc = cs = None
    if rows:
        r = BlockRows.empty(R, C, dev)
        rc = r.buffer.data_ptr()
        rs = rc + r.split
    if columns:
        n = (R if g is None else g.rows) // 128 + (1 if g is None else g.n)  # moe_block_column_blocks
        c = BlockColumns.empty(n, C, dev)
        if g is None:
            c.height = R
        cc = c.buffer.data_ptr()
        cs = cc + c.split
    _filled(g)
    if R > 0:
        a = MoeBlockQuantizeArgs(R, C, by_token, None if g is None else g.pointer, x.data_ptr(), rc, rs, cc, cs)
        _call("moe_block_quantize", dev, ctypes.byref(a))
    return r, c


def quantize_block(x: torch.Tensor, g: Groups | None = None) -> BlockRows:
    """bf16 x [rows, C] by rows; with g, x holds sorted rows, of which the local ones are quantised."""
    return _quantize(x, g, False, True, False)[0]


def quantize_block_columns(x: torch.Tensor, g: Groups | None = None, by_token: bool = False) -> BlockColumns:
    """bf16 sorted rows x [T * k, C] by columns; by_token: x is [T, C] and a sorted row is its token's row.
    Without g, all rows of x are one group."""
    return _quantize(x, g, by_token, False, True)[1]


def quantize_block_both(x: torch.Tensor, g: Groups | None = None) -> tuple[BlockRows, BlockColumns]:
    """bf16 sorted rows x by rows and by columns, from one read."""
    return _quantize(x, g, False, True, True)


def _product(x: BlockRows, w: BlockWeights, g: Groups | None, by_token: bool, transposed: bool, out):
    _ask_form("x", x, BlockRows)
    R, C = (w.N, w.K) if transposed else (w.K, w.N)
    if g is not None:
        dev, n_x = g.device, g.T if by_token else g.rows
    else:
        dev, n_x = x.place(), x.height
    codes, scales = x.pointers("x", n_x, R, dev)
    if w.E != (1 if g is None else g.n):
        raise ValueError(f"w: {w.E} experts, expected {1 if g is None else g.n}")
    if g is None and by_token:
        raise ValueError("by_token needs groups")
    out = _out("out", out, (n_x if g is None else g.rows, C), torch.bfloat16, dev)
    _filled(g)
    a = MoeBlockGemmArgs(n_x, by_token, transposed, None if g is None else g.pointer, codes, scales,
                         w.struct(dev), out.data_ptr())
    if n_x > 0:
        _call("moe_block_gemm", dev, ctypes.byref(a))
    return out


def block_product(x: BlockRows, w: BlockWeights, g: Groups | None = None, by_token: bool = False,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Each sorted row times its expert's weight, x [rows, K] -> bf16 [T * k, N] (moe_block_gemm). by_token: x
    has one row per token. Without groups, every row of x times the one expert of w."""
    return _product(x, w, g, by_token, False, out)


def block_product_grad(dy: BlockRows, w: BlockWeights, g: Groups | None = None,
                       out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of block_product's (sorted) input rows: dy [T * k, N] -> bf16 [T * k, K]."""
    return _product(dy, w, g, False, True, out)


def block_weight_grad(dy: BlockColumns, x: BlockColumns, g: Groups | None = None, rows: int | None = None,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of every expert's weight, bf16 [n, N, K], from the column forms of the output gradient and of
    the input (moe_block_wgrad). Without groups, `rows` says how many rows they hold."""
    if g is None and rows is None:
        raise ValueError("rows: needed without groups")
    _ask_form("dy", dy, BlockColumns)
    _ask_form("x", x, BlockColumns)
    dev = dy.place() if g is None else g.device
    R = rows if g is None else g.rows
    for q in (dy, x) if g is None else ():
        if R < 0 or q.height not in (None, R):
            raise ValueError(f"rows: {R}, but a column form holds {q.height}")
    N, K, n = dy.width, x.width, 1 if g is None else g.n
    _blocks_of_128("dy", N)
    _blocks_of_128("x", K)
    blocks = R // 128 + n
    g_codes, g_scales = dy.pointers("dy", blocks, N, dev)
    x_codes, x_scales = x.pointers("x", blocks, K, dev)
    out = _out("out", out, (n, N, K), torch.bfloat16, dev)
    _filled(g)
    a = MoeBlockWgradArgs(R, N, K, None if g is None else g.pointer, g_codes, g_scales, x_codes, x_scales,
                          out.data_ptr())
    _call("moe_block_wgrad", dev, ctypes.byref(a))
    return out
