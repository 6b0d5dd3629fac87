"""The C ABIs of include/moe_router.h and include/moe_w4.h on the host (no GPU needed): exported symbols, the documented refusals
before anything is enqueued, and the bindings' own checks."""
import ctypes
import os
import re

import pytest
import torch

import block_scaled_moe_amd as moe
from block_scaled_moe_amd import ops, router, w4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EUNSUP, EALIGN, EWS = 0, -1, -2, -3, -4
A = 1 << 40  # a fake, aligned "device" address: never dereferenced on these paths


@pytest.mark.parametrize("header,module,version", [("moe_router.h", router, "moe_router_abi_version"), ("moe_w4.h", w4, "moe_w4_abi_version")])
def test_header_functions_are_exported_and_bound(header, module, version):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))
    assert sorted(module.SIGNATURES) == names
    lib = moe.lib()
    for n in names:
        assert hasattr(lib, n)
    assert getattr(lib, version)() == 1


FAR = 1 << 36  # between fake buffers


def losses(**over):
    l = router.MoeLosses(100, 64, 4, 3, *(A + i * FAR for i in range(7)))
    for k, v in over.items():
        setattr(l, k, v)
    return l


def run_losses(dtype=2, logits=A + 10 * FAR, idx=A + 11 * FAR, valid=A + 12 * FAR + 1, ws=A + 13 * FAR, n=1 << 30, **over):
    return moe.lib().moe_router_losses(ctypes.byref(losses(**over)), dtype, logits, idx, valid, ws, n, None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), EINVAL), (dict(T=1 << 30), EUNSUP), (dict(E=0), EINVAL), (dict(E=4097), EINVAL), (dict(top_k=0), EINVAL), (dict(top_k=9), EINVAL),
    (dict(B=0), EINVAL), (dict(B=1 << 14), EUNSUP), (dict(seq=0), EINVAL), (dict(balance=0), EINVAL), (dict(z=0), EINVAL), (dict(counts=0), EINVAL),
    (dict(tokens=0), EINVAL), (dict(prob_sums=0), EINVAL), (dict(lse=0), EINVAL), (dict(logits=0), EINVAL), (dict(idx=0), EINVAL), (dict(dtype=3), EINVAL),
    (dict(ws=0), EWS), (dict(n=64), EWS), (dict(ws=A + 13 * FAR + 8), EALIGN), (dict(logits=A + 4), EALIGN), (dict(lse=A + 4), EALIGN),
    (dict(counts=A + 8), EALIGN), (dict(seq=A + 4), EALIGN), (dict(z=A + FAR + 32, balance=A + FAR + 32), EINVAL), (dict(lse=A + 10 * FAR + 64), EINVAL),
    (dict(prob_sums=A + 13 * FAR + 16), EINVAL), (dict(counts=A + 11 * FAR), EINVAL), (dict(tokens=A), EINVAL)])
def test_losses_refuse(over, status):
    assert run_losses(**over) == status
    bytes_of = lambda: moe.lib().moe_router_losses_workspace_bytes(ctypes.byref(losses(**{k: v for k, v in over.items() if k in ("T", "E", "top_k", "B", "seq")})))
    sizes = set(over) & {"T", "E", "top_k", "B"} or over.get("seq") == 0
    assert (bytes_of() == 0) == bool(sizes)


def test_losses_refuse_nothing_at_all():
    assert moe.lib().moe_router_losses(None, 2, A, A, None, A, 1 << 20, None) == EINVAL
    assert moe.lib().moe_logits_grad(None, None) == EINVAL and moe.lib().moe_route_backward(None, None) == EINVAL
    assert moe.lib().moe_route_backward_workspace_bytes(None) == 0 and moe.lib().moe_router_losses_workspace_bytes(None) == 0


def run_grad(over_l=(), **over):
    l = losses(**dict(over_l))
    a = router.MoeLogitsGradArgs(100, 64, 4, 2, ctypes.pointer(l), *(A + i * FAR for i in range(10, 17)))
    for k, v in over.items():
        setattr(a, k, v)
    return moe.lib().moe_logits_grad(ctypes.byref(a), None)


NO_L = ctypes.POINTER(router.MoeLosses)()


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), EINVAL), (dict(T=99), EINVAL), (dict(E=65), EINVAL), (dict(top_k=5), EINVAL), (dict(dtype=0), EINVAL), (dict(logits=0), EINVAL),
    (dict(topk_w=0), EINVAL), (dict(d_topk_w=0), EINVAL), (dict(topk_idx=0), EINVAL), (dict(d_logits=0), EINVAL), (dict(l=NO_L), EINVAL),
    (dict(l=NO_L, d_balance=0, d_z=0, topk_w=0, d_topk_w=0), EINVAL), (dict(logits=A + 2), EALIGN), (dict(d_logits=A + 8), EALIGN), (dict(topk_w=A + 4), EALIGN),
    (dict(d_z=A + 2), EALIGN), (dict(d_logits=A + 10 * FAR), EINVAL), (dict(d_logits=A + 6 * FAR), EINVAL), (dict(d_logits=A + 3 * FAR), EINVAL), (dict(d_logits=A + 13 * FAR), EINVAL),
    (dict(over_l=dict(lse=0)), EINVAL), (dict(over_l=dict(counts=A + 4)), EALIGN), (dict(over_l=dict(B=0)), EINVAL)])
def test_logits_grad_refuses(over, status):
    assert run_grad(**over) == status


def test_logits_grad_of_no_tokens():
    assert run_grad(dict(T=0), T=0, d_logits=0, logits=0) == OK


def backward(**over):
    a = router.MoeRouteBackwardArgs(20000, 1024, 128, 1, 2, *(A + i * FAR for i in range(7)), 1 << 30)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), EINVAL), (dict(D=0), EINVAL), (dict(E=0), EINVAL), (dict(E=4097), EINVAL), (dict(D=96), EUNSUP), (dict(D=1 << 24), EUNSUP), (dict(T=1 << 24), EUNSUP),
    (dict(T=(1 << 24) - 1, D=1 << 20), EUNSUP), (dict(E=4096, D=1 << 20), EUNSUP), (dict(dh_dtype=3), EINVAL), (dict(dwr_dtype=0), EINVAL), (dict(dh=0, dwr=0, dbias=0), EINVAL),
    (dict(dwr=0), EINVAL), (dict(h=0), EINVAL), (dict(wr=0), EINVAL), (dict(d_logits=0), EINVAL), (dict(workspace=0), EWS), (dict(workspace_bytes=256), EWS), (dict(h=A + 8), EALIGN),
    (dict(dbias=A + 4), EALIGN), (dict(workspace=A + 8), EALIGN), (dict(dh=A), EINVAL), (dict(dwr=A + FAR), EINVAL), (dict(dh=A + 2 * FAR + 16), EINVAL),
    (dict(dbias=A + 4 * FAR), EINVAL), (dict(dh=A + 6 * FAR), EINVAL)])
def test_route_backward_refuses(over, status):
    assert moe.lib().moe_route_backward(ctypes.byref(backward(**over)), None) == status


def test_route_backward_workspace():
    f = lambda **o: moe.lib().moe_route_backward_workspace_bytes(ctypes.byref(backward(**o)))
    assert f() > 0 and f(T=0) > 0 and f(T=40000) > f() and f(dwr=0, dbias=0) < f() and f(dh=0) < f() and f(dwr=0) == 0 and f(D=100) == 0
    assert moe.lib().moe_route_backward(ctypes.byref(backward(T=0, dwr=0, dbias=0, d_logits=0, h=0, wr=0)), None) == OK


def weights(**over):
    w = w4.MoeW4Weights(8, 100, 256, 64, 1, A, A + FAR, A + 2 * FAR)
    for k, v in over.items():
        setattr(w, k, v)
    return w


WEIGHT_FAULTS = [
    (dict(E=0), EINVAL), (dict(E=4097), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(scale_type=0), EINVAL), (dict(scale_type=3), EINVAL), (dict(group=16), EUNSUP),
    (dict(group=96), EUNSUP), (dict(K=250), EUNSUP), (dict(N=(1 << 20) + 1), EUNSUP), (dict(K=1 << 21), EUNSUP), (dict(N=1 << 20, K=1 << 17), EUNSUP), (dict(codes=0), EINVAL),
    (dict(scales=0), EINVAL), (dict(codes=A + 8), EALIGN), (dict(scales=A + FAR + 2), EALIGN), (dict(zeros=A + 2 * FAR + 1), EALIGN)]


@pytest.mark.parametrize("over,status", WEIGHT_FAULTS)
def test_w4_calls_check_their_weights(over, status):
    lib, w = moe.lib(), weights(**over)
    assert lib.moe_w4_pack(A + 3 * FAR, A + 4 * FAR, A + 5 * FAR, ctypes.byref(w), None) == status
    g = ctypes.pointer(ops.MoeGroups(32, 4, 8, 0, 8, A, A, A, A, 1 << 30))
    a = w4.MoeW4GemmArgs(128, 0, 0, 1, g, A + 3 * FAR, w, A + 4 * FAR)
    assert lib.moe_w4_gemm(ctypes.byref(a), None) == status
    if not set(over) & {"codes", "scales", "zeros"}:
        assert lib.moe_w4_code_bytes(ctypes.byref(w)) == lib.moe_w4_scale_bytes(ctypes.byref(w)) == lib.moe_w4_zero_bytes(ctypes.byref(w)) == 0


def test_w4_sizes():
    lib = moe.lib()
    w = ctypes.byref(weights(N=17, K=320))
    assert lib.moe_w4_code_bytes(w) == 8 * 2 * 2 * 2048 and lib.moe_w4_scale_bytes(w) == 8 * 2 * 2 * 16 * 4 * 2 and lib.moe_w4_zero_bytes(w) == 8 * 2 * 2 * 16 * 4
    t = moe.W4Weights.empty(8, 17, 320, 64, zeros=True, device="cpu")
    assert t.codes.numel() * 4 == lib.moe_w4_code_bytes(w) and t.scales.numel() * 2 == lib.moe_w4_scale_bytes(w) and t.zeros.numel() == lib.moe_w4_zero_bytes(w)


def test_w4_calls_refuse():
    lib = moe.lib()
    pack = lambda c=A + 3 * FAR, s=A + 4 * FAR, z=A + 5 * FAR, **o: lib.moe_w4_pack(c, s, z, ctypes.byref(weights(**o)), None)
    assert pack(c=0) == EINVAL and pack(s=0) == EINVAL and pack(z=0) == EINVAL and pack(zeros=0) == EINVAL
    assert pack(c=A + 3 * FAR + 4) == EALIGN and pack(c=A) == EINVAL and pack(s=A + FAR + 16) == EINVAL and pack(zeros=A + 64) == EINVAL
    assert lib.moe_w4_pack(A, A, A, None, None) == EINVAL and lib.moe_w4_gemm(None, None) == EINVAL

    def gemm(rows=128, by_token=0, swiglu=0, dtype=1, groups=True, x=A + 3 * FAR, out=A + 4 * FAR, over=(), **go):
        g = ops.MoeGroups(32, 4, 8, 0, 8, A, A, A, A, 1 << 30)
        for k, v in go.items():
            setattr(g, k, v)
        a = w4.MoeW4GemmArgs(rows, by_token, swiglu, dtype, ctypes.pointer(g) if groups else None, x, weights(**dict(over)), out)
        return lib.moe_w4_gemm(ctypes.byref(a), None)

    assert gemm(rows=-1) == EINVAL and gemm(dtype=3) == EINVAL and gemm(rows=32) == EINVAL and gemm(by_token=1) == EINVAL
    assert gemm(groups=False) == EINVAL and gemm(groups=False, by_token=1, over=dict(E=1)) == EINVAL      # eight experts, by token
    assert gemm(over=dict(E=7)) == EINVAL and gemm(swiglu=1, over=dict(N=101)) == EINVAL
    assert gemm(x=0) == EINVAL and gemm(out=0) == EINVAL and gemm(x=A + 3 * FAR + 2) == EALIGN and gemm(out=A + 4 * FAR + 8) == EALIGN
    assert gemm(out=A + 3 * FAR) == EINVAL and gemm(out=A) == EINVAL and gemm(out=A + FAR) == EINVAL and gemm(out=A + 2 * FAR) == EINVAL
    assert gemm(plan=0) == EWS and gemm(offsets=0) == EINVAL and gemm(T=-1) == EINVAL
    assert gemm(rows=1 << 25, groups=False, over=dict(E=1)) == EUNSUP
    assert gemm(rows=0, groups=False, over=dict(E=1), x=0, out=0) == OK


def test_bindings_check_their_tensors():
    f, i = lambda *s: torch.zeros(s), lambda *s: torch.zeros(s, dtype=torch.int32)
    for bad in (lambda: moe.router_losses(f(4), i(4, 2)), lambda: moe.router_losses(f(4, 8).half(), i(4, 2)), lambda: moe.router_losses(f(4, 8), i(3, 2)),
                lambda: moe.router_losses(f(4, 8), i(4, 2).long()), lambda: moe.router_losses(f(8, 4).t(), i(4, 2)),
                lambda: moe.router_losses(f(4, 8), i(4, 2), valid=f(4)), lambda: moe.router_losses(f(4, 8), i(4, 2), seq=i(1)),
                lambda: moe.router_losses(f(4, 8), i(4, 2), seq=i(3).long()), lambda: moe.router_losses(f(4, 8).requires_grad_(), i(4, 2)),
                lambda: moe.router_losses(f(4, 8), i(4, 2)),  # not on a GPU
                lambda: moe.router_losses(f(4, 8), i(4, 2), out=moe.RouterLosses.empty(4, 8, 3, device="cpu")),
                lambda: moe.router_losses(f(4, 8), i(4, 2), out=moe.RouterLosses.empty(5, 8, 2, device="cpu")),
                lambda: moe.logits_grad(f(4, 8), i(4, 2)), lambda: moe.logits_grad(f(4, 8), i(4, 2), topk_w=f(4, 2)),
                lambda: moe.logits_grad(f(4, 8), i(4, 2), topk_w=f(4, 2), d_topk_w=f(4, 3)), lambda: moe.logits_grad(f(4, 8), i(4, 2), d_z=f(1), topk_w=f(4, 2), d_topk_w=f(4, 2)),
                lambda: moe.logits_grad(f(4, 8), i(4, 2), moe.RouterLosses.empty(4, 8, 2, device="cpu"), d_balance=f(2)),
                lambda: moe.logits_grad(f(4, 8), i(4, 2), topk_w=f(4, 2), d_topk_w=f(4, 2), out=f(4, 9)),
                lambda: moe.route_backward(f(4, 64), f(8, 64).bfloat16(), f(4, 8)), lambda: moe.route_backward(f(4, 64).bfloat16(), f(8, 64).bfloat16(), f(4, 9)),
                lambda: moe.route_backward(f(4, 64).bfloat16(), f(8, 64).bfloat16(), f(4, 8), dh_dtype=torch.float16),
                lambda: moe.route_backward(f(4, 64).bfloat16(), f(8, 64).bfloat16(), f(4, 8), want_bias=True, want_dwr=False),
                lambda: moe.route_backward(f(4, 64).bfloat16(), f(8, 64).bfloat16(), f(4, 8), dh=f(4, 64), want_dh=False)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoeError):
        moe.route_backward_workspace(4, 100, 8, device="cpu")
    with pytest.raises(ValueError):
        moe.route_backward_workspace(2 ** 32 + 4, 64, 8, device="cpu")
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    for bad in (lambda: moe.pack_w4(u(2, 4), b(2, 4, 1)), lambda: moe.pack_w4(u(1, 4, 48), b(1, 4, 2)), lambda: moe.pack_w4(u(1, 4, 32), b(1, 4, 0)),
                lambda: moe.pack_w4(u(1, 4, 32), f(1, 4, 2)), lambda: moe.pack_w4(u(1, 4, 32), b(1, 4, 2), b(1, 4, 2)), lambda: moe.pack_w4(u(1, 4, 32).int(), b(1, 4, 2)),
                lambda: moe.pack_w4(u(1, 4, 32), b(1, 4, 2)), lambda: moe.pack_w4(u(1, 4, 32), b(1, 4, 2), out=moe.W4Weights.empty(1, 4, 64, 64, device="cpu")),
                lambda: moe.W4Weights.empty(1, 4, 100, 32, device="cpu"), lambda: moe.W4Weights.empty(1, 4, 64, 16, device="cpu"),
                lambda: moe.W4Weights.empty(1, 4, 64, 32, torch.float32, device="cpu")):
        with pytest.raises(ValueError):
            bad()
    w, x = moe.W4Weights.empty(1, 5, 64, 32, device="cpu"), b(3, 64)
    for bad in (lambda: moe.w4_product(x, w), lambda: moe.w4_product(x[0], w), lambda: moe.w4_product(x.float(), w), lambda: moe.w4_product(b(3, 96), w),
                lambda: moe.w4_product(x, w, swiglu=True), lambda: moe.w4_product(x, w, by_token=True), lambda: moe.w4_product(x, w, out_dtype=torch.float16),
                lambda: moe.w4_product(x, w, out=b(3, 6)), lambda: moe.w4_product(x, w, moe.Groups.empty(3, 1, 2, device="cpu"))):
        with pytest.raises(ValueError):
            bad()
