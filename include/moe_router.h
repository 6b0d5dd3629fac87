/*
 * moe_router.h - C ABI of what trains the router of moe.h (AMD MI355X, gfx950; the same library):
 * the losses that keep it balanced with the slots per expert, and the gradients that moe_route and
 * moe_combine leave open: of the logits, of the hidden states and of the router's weight.
 *
 * Conventions: those of moe_ops.h (device pointers owned by the caller and 16-byte aligned unless
 * stated, a hipStream_t as void* that belongs to the current device, arguments checked on the host
 * before anything is enqueued, nothing synchronises, no allocation, no global state; an output that
 * overlaps another buffer of its call is refused). Results do not depend on the order in which
 * workgroups run. Calls that share a workspace must not overlap.
 */
#ifndef BLOCK_SCALED_MOE_ROUTER_H
#define BLOCK_SCALED_MOE_ROUTER_H

#include "moe_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ROUTER_ABI_VERSION 1
int32_t moe_router_abi_version(void);

/* Losses of the B sequences of a batch of T tokens. Sequence s holds tokens seq[s] .. seq[s + 1] - 1
 * (0 <= seq[0] <= .. <= seq[B] <= T, on the device; values outside 0 .. T are taken as the nearer end, and other
 * orders give wrong sums, never a wrong access). A sequence may be empty, and tokens before seq[0] or from seq[B] on
 * are in none: they count nowhere, and their lse is -inf.
 * A token counts if valid[t] != 0 (valid NULL: every token) and any of its logits is above -inf or a
 * NaN; the rows of others may hold anything. Over the tokens of s that count, with n their number:
 *   p[t][e]      = exp(l[t][e] - lse[t]),  lse[t] = log sum over e of exp(l[t][e])   (-inf: does not count)
 *   counts[s][e] = slots (t, j) with topk_idx[t][j] = e; any index outside 0 .. E - 1 counts for none
 *   prob_sums[s][e] = sum of p[t][e],  tokens[s] = n
 *   balance[s]   = E / (top_k n^2) * sum over e of counts * prob_sums     (1 if both are even)
 *   z[s]         = 1 / n * sum of lse[t]^2
 * and both losses are 0 for n = 0. Probabilities, a row's sum and sums over some tokens are fp32, the logarithm added to the maximum,
 * squares and the sums over those and over experts 64-bit, rounded once. NaN and infinite logits of a token that counts reach the losses and
 * prob_sums of its own sequence only. */
typedef struct moe_losses {
    int32_t T, E;             /* tokens, 0 <= T < 2^30; experts, 1 <= E <= 4096   */
    int32_t top_k, B;         /* 1 <= top_k <= 8, T * top_k < 2^31; sequences, 1 <= B < 2^14 */
    const int32_t *seq;       /* [B + 1], or NULL: one sequence of all tokens (B = 1) */
    float *balance, *z;       /* [B] */
    int32_t *counts;          /* [B][E] */
    int32_t *tokens;          /* [B] */
    float *prob_sums;         /* [B][E] */
    float *lse;               /* [T] */
} moe_losses;

/* Device scratch of moe_router_losses, from the size fields; 0 if those are invalid. Host only. */
size_t moe_router_losses_workspace_bytes(const moe_losses *l);

/* Fills every output of l. logits [T][E] of `dtype` (MOE_DT_*), topk_idx [T][top_k], valid [T] bytes
 * (any alignment) or NULL. */
int32_t moe_router_losses(const moe_losses *l, int32_t dtype, const void *logits, const int32_t *topk_idx,
                          const uint8_t *valid, void *workspace, size_t workspace_bytes, void *stream);

/* Gradient of the logits, fp32 [T][E]: the sum of
 *   losses (l given): for each token that counts (lse[t] > -inf or a NaN), with p the softmax of its logits (from the row itself, by
 *     its maximum and sum: not from lse, which is rounded), the counts, tokens and lse of l (a program that
 *     balances over several batches or ranks puts their sums into counts and tokens) and a[e] =
 *     d_balance[s] E / (top_k tokens[s]^2) counts[s][e], which no gradient passes through:
 *       p[t][e] (a[e] - sum over i of p[t][i] a[i])  +  2 d_z[s] / tokens[s] * lse[t] p[t][e]
 *   gate (topk_w given): at e = topk_idx[t][j], for w the softmax over the token's chosen logits that moe_route
 *     returns, g[j] = topk_w[t][j] (d_topk_w[t][j] - sum over i of topk_w[t][i] d_topk_w[t][i]); slots whose index
 *     is outside 0 .. E - 1 take part in nothing, several slots of one expert add up.
 * d_balance, d_z: fp32 [B] gradients of the losses, 4-byte aligned; NULL: that loss has none. With l, moe_logits_grad leaves the rows of
 * tokens in no sequence as they are, and moe_logits_grad_all writes every row: theirs are the gate's gradient alone, zeros
 * without it. Without l, logits is not read (may be NULL) and either writes every row. */
typedef struct moe_logits_grad_args {
    int32_t T, E, top_k;      /* as in moe_losses */
    int32_t dtype;            /* of logits */
    const moe_losses *l;      /* host pointer or NULL; of the same T, E and top_k */
    const void *logits;       /* [T][E] */
    const float *d_balance, *d_z;
    const int32_t *topk_idx;  /* [T][top_k] */
    const float *topk_w, *d_topk_w; /* [T][top_k], both or neither */
    float *d_logits;          /* [T][E] */
} moe_logits_grad_args;
int32_t moe_logits_grad(const moe_logits_grad_args *a, void *stream);
int32_t moe_logits_grad_all(const moe_logits_grad_args *a, void *stream);

/* Gradients of the router's product logits = h wr^T + bias:
 *   dh [T][D] = d_logits wr,  dwr [E][D] = d_logits^T h,  dbias[e] = sum over t of d_logits[t][e]
 * dh or dwr may be NULL (not computed), dbias is computed beside dwr only. h [T][D] and wr [E][D] are bf16, d_logits fp32; dh and dwr are of the
 * given types. d_logits enters the bf16 MFMA in three pieces of 8 bits, which hold it exactly: what all experts share cancels in dh,
 * so that a result may be made of the last bits. Sums are fp32, those over
 * long T in parts that are then added in order. D % 64 == 0, D < 2^24, T < 2^24, E <= 4096 (moe_route: 1024); T * D
 * below 2^38, E * D below 2^32.
 * A NaN or an infinity makes every result that it enters not finite. */
typedef struct moe_route_backward_args {
    int32_t T, D, E;
    int32_t dh_dtype, dwr_dtype; /* MOE_DT_* */
    const uint16_t *h;        /* read for dwr only */
    const uint16_t *wr;       /* read for dh only */
    const float *d_logits;
    void *dh, *dwr;
    float *dbias;
    void *workspace;
    size_t workspace_bytes;   /* moe_route_backward_workspace_bytes */
} moe_route_backward_args;
/* From the size and type fields and which outputs are NULL; 0 if those are invalid. Host only. */
size_t moe_route_backward_workspace_bytes(const moe_route_backward_args *a);
int32_t moe_route_backward(const moe_route_backward_args *a, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* BLOCK_SCALED_MOE_ROUTER_H */
