"""The operators of include/moe_router.h on the GPU where sizes choose another path or values ask for every bit: the router's
product with its operand cut beforehand, and results that only the gradient's last bits make; against plain forms in 64 bits."""
import numpy as np
import pytest
import torch

import block_scaled_moe_amd as moe
import router_ref as ref
from gpu_util import host

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
KINDS = [(BF16, FP32, False), (BF16, BF16, False), (FP32, FP32, True), (BF16, BF16, True), (FP32, BF16, False)]


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def num(t):
    return host(t.float() if t.dtype == BF16 else t)


# ---------------------------------------------------------------- the router's product

def cut_beforehand(T, E, D):
    """The rule of route_backward_plan: values of d_logits times column tiles of 256 from 2^23 on."""
    return T * E * ((D + 255) // 256) >= 1 << 23


# T, E, D on both sides of the rule; a step is 32 of the reduction, a tile 128 (64) rows
SMALL, LARGE = [(300, 60, 320), (129, 128, 256), (31, 384, 64)], [(2100, 100, 10304), (8300, 129, 2112), (5003, 384, 1344), (33000, 257, 192)]


@pytest.mark.parametrize("T,E,D", LARGE)
@pytest.mark.parametrize("kinds", KINDS, ids=str)
def test_product_cut_beforehand(T, E, D, kinds):
    """Every number of steps and tiles of experts, of every type of results, with values that have all their bits."""
    assert cut_beforehand(T, E, D)
    dh_t, dwr_t, bias = kinds
    rng = np.random.default_rng(T + E)
    g = rng.standard_normal((T, E)).astype(np.float32) * 1e-4
    g = np.where(rng.random((T, E)) < 0.05, g * 1000, g).astype(np.float32)
    h, wr = (dev(rng.standard_normal(s).astype(np.float32), BF16) for s in ((T, D), (E, D)))
    dh, dwr, dbias = moe.route_backward(h, wr, dev(g), dh_dtype=dh_t, dwr_dtype=dwr_t, want_bias=bias)
    g = g.astype(np.float64)
    for name, got, a, b, t in (("dh", dh, g, num(wr), dh_t), ("dwr", dwr, np.ascontiguousarray(g.T), num(h), dwr_t)):
        assert got.dtype == t
        y, bound, mean = ref.product(a, b.astype(np.float64), t == BF16, 3, 256)
        ref.close(num(got), y, bound, name)
        err = np.sqrt(((num(got) - y) ** 2).mean())
        assert err <= mean, f"{name}: rms {err}, expected up to {mean}"
    if bias:
        y, bound, _ = ref.product(np.ascontiguousarray(g.T), np.ones((T, 1)), False, 3, 256)
        ref.close(num(dbias), y[:, 0], bound[:, 0], "dbias")
    else:
        assert dbias is None


def pairs(rng, n, m):
    """[n, 2 m] values of 19 bits whose neighbours cancel but for their last six bits, and [n, m] what is left of each pair. Sums of
    up to 64 of either have 24 bits at most."""
    a, s = rng.integers(1 << 18, 1 << 19, (n, m)), rng.integers(-32, 33, (n, m))
    v = np.empty((n, 2 * m), np.float32)
    v[:, 0::2], v[:, 1::2] = (a + s) * 2.0 ** -18, -a * 2.0 ** -18
    return v, s * 2.0 ** -18


@pytest.mark.parametrize("kinds", KINDS, ids=str)
def test_hidden_gradient_of_parts_that_cancel(kinds):
    """What all experts' weights share cancels in dh, as a token's gradients sum to nearly nothing, and the rest is in the last bits
    of d_logits: every sum here is exact in fp32, so the result is rounded once if at all."""
    dh_t, dwr_t, bias = kinds
    for T, E, D in ((200, 64, 320), (5100, 64, 6656)):
        rng = np.random.default_rng(T)
        g, left = pairs(rng, T, E // 2)
        w = rng.choice(np.array([-1.0, 1.0], np.float32), (E // 2, D))
        dh, _, _ = moe.route_backward(torch.zeros((T, D), dtype=BF16, device="cuda"), dev(np.repeat(w, 2, 0), BF16), dev(g),
                                      dh_dtype=dh_t, dwr_dtype=dwr_t, want_bias=bias)
        assert torch.equal(dh.cpu(), torch.from_numpy(left @ w.astype(np.float64)).to(dh_t)), (T, E, D)


@pytest.mark.parametrize("kinds", KINDS, ids=str)
def test_weight_gradient_of_parts_that_cancel(kinds):
    dh_t, dwr_t, bias = kinds
    for T, E, D in ((64, 300, 320), (64, 4096, 8192)):
        rng = np.random.default_rng(E)
        g, left = pairs(rng, E, T // 2)
        h = rng.choice(np.array([-1.0, 1.0], np.float32), (T // 2, D))
        _, dwr, dbias = moe.route_backward(dev(np.repeat(h, 2, 0), BF16), torch.zeros((E, D), dtype=BF16, device="cuda"),
                                           dev(np.ascontiguousarray(g.T)), dh_dtype=dh_t, dwr_dtype=dwr_t, want_bias=bias)
        assert torch.equal(dwr.cpu(), torch.from_numpy(left @ h.astype(np.float64)).to(dwr_t)), (T, E, D)
        if bias:
            assert torch.equal(dbias.cpu(), torch.from_numpy(left.sum(1)).float())


@pytest.mark.parametrize("T,E,D", SMALL + LARGE)
def test_product_repeats_itself(T, E, D):
    """The same bits every time, whatever the workspace held."""
    assert cut_beforehand(T, E, D) == ((T, E, D) in LARGE)
    gen = torch.Generator(device="cuda").manual_seed(T)
    h, wr = (torch.randn(s, device="cuda", generator=gen).to(BF16) for s in ((T, D), (E, D)))
    g = torch.randn((T, E), device="cuda", generator=gen)
    ws = moe.route_backward_workspace(T, D, E, want_bias=True).zero_()
    first = moe.route_backward(h, wr, g, want_bias=True, workspace=ws)
    for fill in (255, 127, 1):
        again = moe.route_backward(h, wr, g, want_bias=True, workspace=ws.fill_(fill))
        assert all(torch.equal(a, b) for a, b in zip(first, again))
