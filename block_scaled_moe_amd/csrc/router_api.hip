// router_api.hip - host side of the C ABI declared in include/moe_router.h: argument validation (pure host
// code, no HIP call), workspaces and the launches on the caller's stream.
#include "router_internal.h"

#include "api_common.h"

using namespace moe;

namespace {

int32_t check_sizes(int32_t T, int32_t E, int32_t top_k) {
    if (T < 0 || E < 1 || E > 4096 || top_k < 1 || top_k > 8) return MOE_ERR_INVALID_ARG;
    return T < (1 << 30) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

int32_t check_losses_sizes(const moe_losses *l) {
    if (!l) return MOE_ERR_INVALID_ARG;
    const int32_t rc = check_sizes(l->T, l->E, l->top_k);
    if (rc != MOE_OK) return rc;
    if (l->B < 1 || (!l->seq && l->B != 1)) return MOE_ERR_INVALID_ARG;
    if ((int64_t)l->T * l->top_k > INT32_MAX) return MOE_ERR_UNSUPPORTED;  // one expert may have every slot
    return l->B < (1 << 14) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

// The buffers of l that a gradient reads, and those that the losses fill.
int32_t check_losses_read(const moe_losses *l) {
    if (!l->counts || !l->tokens || (l->T > 0 && !l->lse)) return MOE_ERR_INVALID_ARG;
    return aligned(l->counts, 16) && aligned(l->tokens, 16) && aligned(l->lse, 16) && aligned(l->seq, 16) ? MOE_OK
                                                                                                          : MOE_ERR_ALIGNMENT;
}

int32_t check_route_backward_sizes(const moe_route_backward_args *a) {
    if (!a || a->T < 0 || a->D < 1 || a->E < 1 || a->E > 4096) return MOE_ERR_INVALID_ARG;
    if ((!a->dh && !a->dwr) || (a->dbias && !a->dwr)) return MOE_ERR_INVALID_ARG;
    if ((a->dh && !type_ok(a->dh_dtype)) || (a->dwr && !type_ok(a->dwr_dtype))) return MOE_ERR_INVALID_ARG;
    if (a->D % 64 || a->D >= (1 << 24) || a->T >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
    return (int64_t)a->T * a->D < (1ll << 38) && (int64_t)a->E * a->D < (1ll << 32) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

int32_t logits_grad(const moe_logits_grad_args *a, bool all, void *stream) {
    if (!a) return MOE_ERR_INVALID_ARG;
    int32_t rc = check_sizes(a->T, a->E, a->top_k);
    if (rc != MOE_OK) return rc;
    if ((!a->l && !a->topk_w) || !a->topk_w != !a->d_topk_w || (!a->l && (a->d_balance || a->d_z))) return MOE_ERR_INVALID_ARG;
    if (a->l) {
        rc = check_losses_sizes(a->l);
        if (rc != MOE_OK) return rc;
        if (a->l->T != a->T || a->l->E != a->E || a->l->top_k != a->top_k || !type_ok(a->dtype)) return MOE_ERR_INVALID_ARG;
        rc = check_losses_read(a->l);
        if (rc != MOE_OK) return rc;
    }
    if (a->T == 0) return MOE_OK;
    if (!a->d_logits || (a->l && !a->logits) || (a->topk_w && !a->topk_idx)) return MOE_ERR_INVALID_ARG;
    if (!aligned(a->d_logits, 16) || !aligned(a->topk_idx, 16) || !aligned(a->topk_w, 16) || !aligned(a->d_topk_w, 16) ||
        !aligned(a->d_balance, 4) || !aligned(a->d_z, 4) || (a->l && !aligned(a->logits, 16)))
        return MOE_ERR_ALIGNMENT;
    const int64_t row = (int64_t)a->E, slots = 4 * (int64_t)a->top_k;
    const Extent out = {a->d_logits, a->T, 4 * row};
    if (a->topk_w && outputs_meet({out}, {{a->topk_idx, a->T, slots}, {a->topk_w, a->T, slots}, {a->d_topk_w, a->T, slots}}))
        return MOE_ERR_INVALID_ARG;
    if (a->l) {
        const moe_losses &l = *a->l;
        if (outputs_meet({out}, {{a->logits, a->T, type_bytes(a->dtype) * row}, {a->d_balance, l.B, 4}, {a->d_z, l.B, 4},
                                 {l.seq, (int64_t)l.B + 1, 4}, {l.counts, l.B, 4 * row}, {l.tokens, l.B, 4}, {l.lse, a->T, 4}}))
            return MOE_ERR_INVALID_ARG;
    }
    return status_of(launch_logits_grad(*a, all, (hipStream_t)stream));
}

}  // namespace

extern "C" {

int32_t moe_router_abi_version(void) { return MOE_ROUTER_ABI_VERSION; }

size_t moe_router_losses_workspace_bytes(const moe_losses *l) {
    return check_losses_sizes(l) == MOE_OK ? loss_plan(l->T, l->E, l->B, l->seq).total : 0;
}

int32_t moe_router_losses(const moe_losses *l, int32_t dtype, const void *logits, const int32_t *topk_idx,
                          const uint8_t *valid, void *workspace, size_t workspace_bytes, void *stream) {
    int32_t rc = check_losses_sizes(l);
    if (rc != MOE_OK) return rc;
    if (!type_ok(dtype) || !l->balance || !l->z || !l->prob_sums) return MOE_ERR_INVALID_ARG;
    rc = check_losses_read(l);
    if (rc != MOE_OK) return rc;
    if (l->T > 0 && (!logits || !topk_idx)) return MOE_ERR_INVALID_ARG;
    if (!aligned(l->balance, 16) || !aligned(l->z, 16) || !aligned(l->prob_sums, 16) || !aligned(logits, 16) ||
        !aligned(topk_idx, 16))
        return MOE_ERR_ALIGNMENT;
    const size_t need = loss_plan(l->T, l->E, l->B, l->seq).total;
    if (!workspace || workspace_bytes < need) return MOE_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return MOE_ERR_ALIGNMENT;
    const int64_t be = (int64_t)l->B * l->E;
    if (outputs_meet({{l->balance, l->B, 4}, {l->z, l->B, 4}, {l->counts, be, 4}, {l->tokens, l->B, 4}, {l->prob_sums, be, 4},
                      {l->lse, l->T, 4}, {workspace, 1, (int64_t)need}},
                     {{logits, l->T, type_bytes(dtype) * l->E}, {topk_idx, l->T, 4 * (int64_t)l->top_k}, {valid, l->T, 1},
                      {l->seq, (int64_t)l->B + 1, 4}}))
        return MOE_ERR_INVALID_ARG;
    return status_of(launch_router_losses(*l, dtype, logits, topk_idx, valid, static_cast<uint8_t *>(workspace),
                                          (hipStream_t)stream));
}

int32_t moe_logits_grad(const moe_logits_grad_args *a, void *stream) { return logits_grad(a, false, stream); }
int32_t moe_logits_grad_all(const moe_logits_grad_args *a, void *stream) { return logits_grad(a, true, stream); }

size_t moe_route_backward_workspace_bytes(const moe_route_backward_args *a) {
    return check_route_backward_sizes(a) == MOE_OK ? route_backward_plan(*a).total : 0;
}

int32_t moe_route_backward(const moe_route_backward_args *a, void *stream) {
    const int32_t rc = check_route_backward_sizes(a);
    if (rc != MOE_OK) return rc;
    if (a->T > 0 && (!a->d_logits || (a->dh && !a->wr) || (a->dwr && !a->h))) return MOE_ERR_INVALID_ARG;
    if (!aligned(a->d_logits, 16) || !aligned(a->dh, 16) || !aligned(a->dwr, 16) || !aligned(a->dbias, 16) ||
        (a->dh && !aligned(a->wr, 16)) || (a->dwr && !aligned(a->h, 16)))
        return MOE_ERR_ALIGNMENT;
    const RouteBackwardPlan p = route_backward_plan(*a);
    if (!a->workspace || a->workspace_bytes < p.total) return MOE_ERR_WORKSPACE;
    if (!aligned(a->workspace, 16)) return MOE_ERR_ALIGNMENT;
    const int64_t D = a->D;
    if (outputs_meet({{a->dh, a->T, D * type_bytes(a->dh_dtype)}, {a->dwr, a->E, D * type_bytes(a->dwr_dtype)}, {a->dbias, a->E, 4},
                      {a->workspace, 1, (int64_t)p.total}},
                     {{a->d_logits, a->T, 4 * (int64_t)a->E}, {a->dh ? a->wr : nullptr, a->E, D * 2},
                      {a->dwr ? a->h : nullptr, a->T, D * 2}}))
        return MOE_ERR_INVALID_ARG;
    if (a->T == 0 && !a->dwr) return MOE_OK;
    return status_of(launch_route_backward(*a, p, (hipStream_t)stream));
}

}  // extern "C"
