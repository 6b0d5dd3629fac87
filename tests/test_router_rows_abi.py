"""moe_logits_grad_all of include/moe_router.h on the host (no GPU needed): the refusals of moe_logits_grad, before anything is
enqueued."""
import ctypes

import pytest

import block_scaled_moe_amd as moe
from block_scaled_moe_amd import router

OK, EINVAL, EUNSUP, EALIGN = 0, -1, -2, -3
A, FAR = 1 << 40, 1 << 36  # fake, aligned "device" addresses, never dereferenced on these paths
NO_L = ctypes.POINTER(router.MoeLosses)()


def run(name, over_l=(), **over):
    l = router.MoeLosses(100, 64, 4, 3, *(A + i * FAR for i in range(7)))
    for k, v in dict(over_l).items():
        setattr(l, k, v)
    a = router.MoeLogitsGradArgs(100, 64, 4, 2, ctypes.pointer(l), *(A + i * FAR for i in range(10, 17)))
    for k, v in over.items():
        setattr(a, k, v)
    return getattr(moe.lib(), name)(ctypes.byref(a), None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), EINVAL), (dict(T=1 << 30), EUNSUP), (dict(T=99), EINVAL), (dict(E=65), EINVAL), (dict(dtype=0), EINVAL), (dict(logits=0), EINVAL),
    (dict(topk_w=0), EINVAL), (dict(topk_idx=0), EINVAL), (dict(d_logits=0), EINVAL), (dict(l=NO_L), EINVAL), (dict(logits=A + 2), EALIGN),
    (dict(d_logits=A + 8), EALIGN), (dict(d_logits=A + 10 * FAR), EINVAL), (dict(d_logits=A + 6 * FAR), EINVAL), (dict(over_l=dict(lse=0)), EINVAL),
    (dict(over_l=dict(T=0), T=0, d_logits=0, logits=0), OK)])
def test_both_forms_refuse_alike(over, status):
    assert run("moe_logits_grad_all", **over) == run("moe_logits_grad", **over) == status
    assert moe.lib().moe_logits_grad_all(None, None) == EINVAL


@pytest.mark.parametrize("T", [0, 1, 64, 65, 100, 40000, 1 << 20])
def test_workspace_is_the_same_with_and_without_sequences(T):
    """It follows from the sizes: a program may ask for it before it has the starts."""
    size = lambda seq: moe.lib().moe_router_losses_workspace_bytes(ctypes.byref(router.MoeLosses(T, 64, 4, 1, seq)))
    assert size(A) == size(0) > 0


@pytest.mark.parametrize("T,top_k,fits", [((1 << 28) - 1, 8, True), (1 << 28, 8, False), ((1 << 30) - 1, 2, True), ((1 << 30) - 1, 3, False), ((1 << 30) - 1, 1, True)])
def test_counts_of_slots_fit_their_type(T, top_k, fits):
    """All slots may be of one expert, whose count is a 32-bit number."""
    l = router.MoeLosses(T, 64, top_k, 3, *(A + i * 16 * FAR for i in range(7)))
    assert (moe.lib().moe_router_losses_workspace_bytes(ctypes.byref(l)) > 0) == fits
    if not fits:
        call = moe.lib().moe_router_losses(ctypes.byref(l), 2, A + 200 * FAR, A + 220 * FAR, None, A + 240 * FAR, 1 << 34, None)
        assert call == EUNSUP and run("moe_logits_grad", dict(T=T, top_k=top_k), T=T, top_k=top_k) == EUNSUP
