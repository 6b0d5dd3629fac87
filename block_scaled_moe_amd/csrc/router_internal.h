// router_internal.h - launchers of the operators declared in include/moe_router.h, shared between their
// kernel files and the host API (router_api.hip). Every launcher enqueues on `stream` and returns
// hipGetLastError().
#pragma once
#include "../../include/moe_router.h"
#include "internal.h"

namespace moe {

// Runs of up to 2^log_rows tokens of one sequence. Without `seq` they are numbered in a row. Else the tokens before seq[0] and those
// from seq[B] on count as sequences -1 and B, and run i of sequence s has number (its first token >> log_rows) + s + 1 + i: no
// two runs share one, and they are fewer than (T >> log_rows) + B + 2.
struct RunSplit {
    int32_t log_rows;
    int64_t n;
};
RunSplit run_split(int32_t T, int32_t B, bool seq, int32_t rows_at_least, int32_t runs_at_most);

// Byte offsets inside the workspace of moe_router_losses.
struct LossPlan {
    RunSplit runs;
    size_t sums, counts, squares, tokens, parts, arrived, total;
};
LossPlan loss_plan(int32_t T, int32_t E, int32_t B, bool seq);
hipError_t launch_router_losses(const moe_losses &l, int32_t dtype, const void *logits, const int32_t *topk_idx,
                                const uint8_t *valid, uint8_t *workspace, hipStream_t s);
hipError_t launch_logits_grad(const moe_logits_grad_args &a, bool all, hipStream_t s);  // all: rows of tokens in no sequence too

// Workspace and work of moe_route_backward.
struct RouteBackwardPlan {
    bool cut;                           // d_logits into pieces beforehand
    int32_t t_tiles, e_tiles;           // of 128 rows, 64 if not cut beforehand
    int32_t t_steps, e_steps;           // of 32 along the reduction
    int32_t splits, steps_per_split;    // of dwr's reduction
    size_t a_h, a_w, parts, bias_parts, total;
};
RouteBackwardPlan route_backward_plan(const moe_route_backward_args &a);
hipError_t launch_route_backward(const moe_route_backward_args &a, const RouteBackwardPlan &p, hipStream_t s);

}  // namespace moe
