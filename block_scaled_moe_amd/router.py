"""What trains the router (include/moe_router.h): the balance loss and the z-loss of every sequence of a batch with the
slots per expert, and the gradients of the logits, of the hidden states and of the router's weight.

The functions marshal arguments like ops.py's: wrong dtypes, shapes, devices or strides raise ValueError before the call, an
argument that the library refuses raises MoeError, and autograd does not see the calls (a tensor that asks for a gradient is
refused while gradients are on).

    idx, w, logits, _ = route(h, wr, want_logits=True)
    l = router_losses(logits, idx, seq=starts)                       # l.balance, l.z: fp32 [B]
    ...                                                              # experts, combine; combine_backward gives d_w
    d_logits = logits_grad(logits, idx, l, d_balance=a, d_z=b, topk_w=w, d_topk_w=d_w)
    dh, dwr, _ = route_backward(h, wr, d_logits)
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .ops import DTYPES, _ask, _call, _function, _int32, _once, _out


class MoeLosses(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("top_k", ctypes.c_int32), ("B", ctypes.c_int32),
                ("seq", ctypes.c_void_p), ("balance", ctypes.c_void_p), ("z", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("tokens", ctypes.c_void_p), ("prob_sums", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class MoeLogitsGradArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("top_k", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("l", ctypes.POINTER(MoeLosses)), ("logits", ctypes.c_void_p), ("d_balance", ctypes.c_void_p),
                ("d_z", ctypes.c_void_p), ("topk_idx", ctypes.c_void_p), ("topk_w", ctypes.c_void_p),
                ("d_topk_w", ctypes.c_void_p), ("d_logits", ctypes.c_void_p)]


class MoeRouteBackwardArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("D", ctypes.c_int32), ("E", ctypes.c_int32), ("dh_dtype", ctypes.c_int32),
                ("dwr_dtype", ctypes.c_int32), ("h", ctypes.c_void_p), ("wr", ctypes.c_void_p), ("d_logits", ctypes.c_void_p),
                ("dh", ctypes.c_void_p), ("dwr", ctypes.c_void_p), ("dbias", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


_P, _I, _Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_L, _B = ctypes.POINTER(MoeLosses), ctypes.POINTER(MoeRouteBackwardArgs)

# every symbol include/moe_router.h declares, with its ctypes signature
SIGNATURES = {
    "moe_router_abi_version": ([], _I),
    "moe_router_losses_workspace_bytes": ([_L], _Z),
    "moe_router_losses": ([_L, _I, _P, _P, _P, _P, _Z, _P], _I),
    "moe_logits_grad": ([ctypes.POINTER(MoeLogitsGradArgs), _P], _I),
    "moe_logits_grad_all": ([ctypes.POINTER(MoeLogitsGradArgs), _P], _I),
    "moe_route_backward_workspace_bytes": ([_B], _Z),
    "moe_route_backward": ([_B, _P], _I),
}


def _matrix(what: str, t: torch.Tensor) -> tuple[int, int]:
    if t.dim() != 2:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected two dimensions")
    rows, columns = t.shape
    if rows >= 2 ** 31 or columns >= 2 ** 31:
        _int32(what, max(rows, columns))
    return rows, columns


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _refuse(name: str, status: int = -1):
    from . import MoeError
    raise MoeError(name, status)


@functools.lru_cache(maxsize=256)
def _losses_layout(T: int, E: int, top_k: int, B: int, seq: bool) -> tuple[int, ...]:
    """Places of prob_sums, lse, counts, tokens, balance, z and the workspace in RouterLosses.buffer, in 4-byte words, each a
    multiple of 64, and its words in all; the workspace's bytes."""
    for v in (T, E, top_k, B):
        _int32("losses", v)
    st = MoeLosses(T, E, top_k, B, 256 if seq else None)
    n = int(_function("moe_router_losses_workspace_bytes")(ctypes.byref(st)))
    if n == 0:
        _refuse("moe_router_losses_workspace_bytes")
    up = lambda words: (words + 63) // 64 * 64
    at = [0]
    for words in (B * E, T, B * E, B, B, B, (n + 3) // 4):
        at.append(at[-1] + up(words))
    return (*at, n)


class RouterLosses:
    """Losses of the B sequences of a batch, with what their gradient reads (moe_losses; filled by router_losses). The
    arrays share one allocation, of which they are views. counts and tokens may be added to (sums over several batches or
    ranks) before the gradient is asked for; they are changed in place, not replaced."""

    def __init__(self, T: int, E: int, top_k: int, seq: torch.Tensor | None = None, device="cuda"):
        if seq is not None and (seq.dim() != 1 or seq.shape[0] < 2):
            raise ValueError(f"seq: shape {tuple(seq.shape)}, expected [B + 1], B > 0")
        self.T, self.E, self.top_k = T, E, top_k
        self.B = 1 if seq is None else seq.shape[0] - 1
        self._at = at = _losses_layout(T, E, top_k, self.B, seq is not None)
        self.buffer = torch.empty(at[7], dtype=torch.float32, device=device)
        self.device = self.buffer.device
        if seq is not None:
            _ask("seq", seq, (self.B + 1,), torch.int32, self.device)
        self.seq = seq  # int32 [B + 1], or None: one sequence of all tokens
        self.filled = False  # by router_losses
        base = self.buffer.data_ptr()
        self.struct = MoeLosses(T, E, top_k, self.B, _ptr(seq), base + 4 * at[4], base + 4 * at[5], base + 4 * at[2], base + 4 * at[3],
                                base, base + 4 * at[1])
        self.workspace = base + 4 * at[6]
        self.ref = ctypes.byref(self.struct)

    @staticmethod
    def empty(T: int, E: int, top_k: int, seq: torch.Tensor | None = None, device="cuda") -> "RouterLosses":
        return RouterLosses(T, E, top_k, seq, device)

    @_once
    def pointer(self):
        return ctypes.pointer(self.struct)

    @_once
    def _words(self) -> torch.Tensor:
        return self.buffer.view(torch.int32)

    @_once
    def balance(self) -> torch.Tensor:
        """fp32 [B]"""
        return self.buffer.as_strided((self.B,), (1,), self._at[4])

    @_once
    def z(self) -> torch.Tensor:
        """fp32 [B]"""
        return self.buffer.as_strided((self.B,), (1,), self._at[5])

    @_once
    def counts(self) -> torch.Tensor:
        """int32 [B, E]: slots of every expert."""
        return self._words.as_strided((self.B, self.E), (self.E, 1), self._at[2])

    @_once
    def tokens(self) -> torch.Tensor:
        """int32 [B]: tokens that count."""
        return self._words.as_strided((self.B,), (1,), self._at[3])

    @_once
    def prob_sums(self) -> torch.Tensor:
        """fp32 [B, E]"""
        return self.buffer.as_strided((self.B, self.E), (self.E, 1), 0)

    @_once
    def lse(self) -> torch.Tensor:
        """fp32 [T]; -inf: the token does not count, or lies in no sequence."""
        return self.buffer.as_strided((self.T,), (1,), self._at[1])

    def check(self):
        """Somebody put another tensor in an array's place: the library would not see it."""
        own = self.__dict__
        for name, at in (("counts", 2), ("tokens", 3), ("lse", 1)):
            if name in own and own[name].data_ptr() != self.buffer.data_ptr() + 4 * self._at[at] and own[name].numel():
                raise ValueError(f"losses: {name} was replaced; it is changed in place")


def router_losses(logits: torch.Tensor, topk_idx: torch.Tensor, valid: torch.Tensor | None = None,
                  seq: torch.Tensor | None = None, out: RouterLosses | None = None) -> RouterLosses:
    """logits [T, E] (fp32 or bf16) and topk_idx int32 [T, k] -> RouterLosses (moe_router_losses). valid: bool or uint8 [T],
    the tokens that count (default: all). seq: int32 [B + 1] starts of packed sequences, each with losses of its own
    (default: one sequence); tokens before the first one or from the last start on count nowhere. `out`: losses of the same
    sizes to fill again, which hold their own seq."""
    T, E = _matrix("logits", logits)
    k = _matrix("topk_idx", topk_idx)[1]
    dev = logits.device
    _ask("logits", logits, (T, E), DTYPES, dev)
    _ask("topk_idx", topk_idx, (T, k), torch.int32, dev)
    if valid is not None:
        _ask("valid", valid, (T,), (torch.bool, torch.uint8), dev)
    if out is None:
        out = RouterLosses(T, E, k, seq, dev)
    elif (out.T, out.E, out.top_k, out.device) != (T, E, k, dev) or (seq is not None and seq is not out.seq):
        raise ValueError("out: losses of other sizes, sequences or on another device")
    out.check()
    _call("moe_router_losses", dev, out.ref, DTYPES[logits.dtype], logits.data_ptr(), topk_idx.data_ptr(), _ptr(valid),
          out.workspace, out._at[8])
    out.filled = True
    return out


def logits_grad(logits: torch.Tensor, topk_idx: torch.Tensor, losses: RouterLosses | None = None,
                d_balance: torch.Tensor | None = None, d_z: torch.Tensor | None = None, topk_w: torch.Tensor | None = None,
                d_topk_w: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of the logits, fp32 [T, E] (moe_logits_grad): of the losses (d_balance and d_z fp32 [B], None: no
    gradient), of the gate's weights (topk_w and d_topk_w fp32 [T, k]; without `losses` of them alone), or of both. Tokens
    that do not count or lie in no sequence have the gate's gradient alone, or zeros. In a given `out` the rows of tokens in no
    sequence keep what they hold."""
    T, E = _matrix("logits", logits)
    k = _matrix("topk_idx", topk_idx)[1]
    dev = logits.device
    _ask("logits", logits, (T, E), DTYPES, dev)
    _ask("topk_idx", topk_idx, (T, k), torch.int32, dev)
    if (topk_w is None) != (d_topk_w is None):
        raise ValueError("topk_w and d_topk_w belong together")
    if losses is None and topk_w is None:
        raise ValueError("neither losses nor the gate's weights are given")
    if losses is None and (d_balance is not None or d_z is not None):
        raise ValueError("d_balance, d_z: without losses")
    for what, t in (("topk_w", topk_w), ("d_topk_w", d_topk_w)):
        if t is not None:
            _ask(what, t, (T, k), torch.float32, dev)
    l = None
    if losses is not None:
        if (losses.T, losses.E, losses.top_k, losses.device) != (T, E, k, dev):
            raise ValueError("losses: of other sizes or on another device")
        if not losses.filled:
            raise ValueError("losses that router_losses has not filled")
        losses.check()
        l = losses.pointer
        for what, t in (("d_balance", d_balance), ("d_z", d_z)):
            if t is not None:
                _ask(what, t, (losses.B,), torch.float32, dev)
    name = "moe_logits_grad_all" if out is None else "moe_logits_grad"
    out = _out("out", out, (T, E), torch.float32, dev)
    a = MoeLogitsGradArgs(T, E, k, DTYPES[logits.dtype], l, logits.data_ptr(), _ptr(d_balance), _ptr(d_z), topk_idx.data_ptr(),
                          _ptr(topk_w), _ptr(d_topk_w), out.data_ptr())
    _call(name, dev, ctypes.byref(a))
    return out


def _backward_args(T, D, E, dh_dtype, dwr_dtype, want_dh, want_dwr, want_bias) -> MoeRouteBackwardArgs:
    mark = lambda want: 16 if want else None  # which outputs there are; no address yet
    return MoeRouteBackwardArgs(T, D, E, DTYPES.get(dh_dtype, 0), DTYPES.get(dwr_dtype, 0), None, None, None, mark(want_dh),
                                mark(want_dwr), mark(want_bias), None, 0)


@functools.lru_cache(maxsize=256)
def _backward_bytes(T: int, D: int, E: int, dh_dtype, dwr_dtype, want_dh: bool, want_dwr: bool, want_bias: bool) -> int:
    for v in (T, D, E):
        _int32("sizes", v)
    a = _backward_args(T, D, E, dh_dtype, dwr_dtype, want_dh, want_dwr, want_bias)
    n = int(_function("moe_route_backward_workspace_bytes")(ctypes.byref(a)))
    if n == 0:
        _refuse("moe_route_backward_workspace_bytes")
    return n


def route_backward_workspace(T: int, D: int, E: int, dh_dtype: torch.dtype = torch.bfloat16,
                             dwr_dtype: torch.dtype = torch.float32, want_dh: bool = True, want_dwr: bool = True,
                             want_bias: bool = False, device="cuda") -> torch.Tensor:
    """Device scratch for route_backward with these arguments (reusable across calls that do not overlap)."""
    n = _backward_bytes(T, D, E, dh_dtype, dwr_dtype, want_dh, want_dwr, want_bias)
    return torch.empty(n, dtype=torch.uint8, device=device)


def route_backward(h: torch.Tensor, wr: torch.Tensor, d_logits: torch.Tensor, dh: torch.Tensor | None = None,
                   dwr: torch.Tensor | None = None, dh_dtype: torch.dtype = torch.bfloat16,
                   dwr_dtype: torch.dtype = torch.float32, want_dh: bool = True, want_dwr: bool = True, want_bias: bool = False,
                   workspace: torch.Tensor | None = None):
    """Gradients of the router's product from d_logits fp32 [T, E] -> (dh [T, D], dwr [E, D], dbias fp32 [E]), None
    for what is not wanted (moe_route_backward). h [T, D] and wr [E, D] are bf16. dh and dwr: buffers to fill, which
    set their types; otherwise dh_dtype and dwr_dtype, bf16 or fp32."""
    T, D = _matrix("h", h)
    E = _matrix("wr", wr)[0]
    dev = h.device
    _ask("h", h, (T, D), torch.bfloat16, dev)
    _ask("wr", wr, (E, D), torch.bfloat16, dev)
    _ask("d_logits", d_logits, (T, E), torch.float32, dev)
    if dh_dtype not in DTYPES or dwr_dtype not in DTYPES:
        raise ValueError(f"dh_dtype, dwr_dtype: {dh_dtype}, {dwr_dtype}")
    if (dh is not None and not want_dh) or (dwr is not None and not want_dwr) or (want_bias and not want_dwr):
        raise ValueError("dh, dwr: a buffer for what is not wanted, or the bias's gradient without the weight's")
    if want_dh:
        dh = _out("dh", dh, (T, D), dh_dtype if dh is None else DTYPES, dev)
        dh_dtype = dh.dtype
    if want_dwr:
        dwr = _out("dwr", dwr, (E, D), dwr_dtype if dwr is None else DTYPES, dev)
        dwr_dtype = dwr.dtype
    dbias = torch.empty(E, dtype=torch.float32, device=dev) if want_bias else None
    a = _backward_args(T, D, E, dh_dtype, dwr_dtype, want_dh, want_dwr, want_bias)
    if workspace is None:
        workspace = torch.empty(_backward_bytes(T, D, E, dh_dtype, dwr_dtype, want_dh, want_dwr, want_bias), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace: on another device, or not contiguous")
    a.h, a.wr, a.d_logits = h.data_ptr(), wr.data_ptr(), d_logits.data_ptr()
    a.dh, a.dwr, a.dbias = _ptr(dh), _ptr(dwr), _ptr(dbias)
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call("moe_route_backward", dev, ctypes.byref(a))
    return dh, dwr, dbias
