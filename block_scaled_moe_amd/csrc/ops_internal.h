// ops_internal.h - launchers of the operators declared in include/moe_ops.h, shared between
// their kernel files and the host API (ops_api.hip). Every launcher enqueues on `stream`
// and returns hipGetLastError().
#pragma once
#include "../../include/moe_ops.h"
#include "internal.h"

namespace moe {

// Rows per work-list tile of the grouped products; the lists are written by moe_sort.
constexpr int32_t kGroupTile = 224;
// Largest dimension that blocks of 128 run along (32-bit byte offsets of 128 of its columns).
constexpr int32_t kMaxBlockDim = 1 << 24;

// Byte offsets inside moe_groups::plan.
struct GroupsPlan {
    int32_t n, max_tiles, chunk_tokens, n_chunks;
    size_t ctrl, counts, tile_expert, tile_row0, chunk_counts, total;
};
GroupsPlan groups_plan(int32_t T, int32_t top_k, int32_t n);

// Scales of a row of a rows form, padded so that four blocks' are one aligned 16-byte load.
__host__ __device__ inline int32_t scale_stride(int32_t C) { return (C / 128 + 3) / 4 * 4; }
// A row's place in its block's plane of codes, and in the scales, is a 32-bit byte offset.
inline bool rows_form_fits(int32_t rows, int32_t C) {
    return rows < (1 << 25) && (int64_t)rows * scale_stride(C) < (1 << 30);
}

// What a grouped product's workgroups read to find their rows. offsets == NULL: one group of
// `rows` rows, tiles computed from it.
struct GroupView {
    const Ctrl *ctrl;
    const int32_t *tile_expert, *tile_row0, *offsets, *sorted_slot;
    int32_t rows, top_k, n, max_tiles;
    int32_t mean_rows;  // average rows of a group for an even routing (host's rule for the kernel)
};
// Status of g's fields (as moe_sort filled them), and the view of a batch of g's slots or, without g, of `rows` rows
// (ops_api.hip).
int32_t check_filled_groups(const moe_groups *g);
GroupView group_view(const moe_groups *g, int32_t rows);

// ---- sort (sort.hip), for up to kSortMaxLocal local experts: fills what launch_permute does
constexpr int32_t kSortMaxLocal = 1024;
int32_t sort_chunk_slots(int64_t n_slots);  // slots of one row of chunk_counts
hipError_t launch_sort(const PermuteArgs &a, int32_t n_slots, hipStream_t s);

// ---- rows by expert and back (tokens.hip)
hipError_t launch_gather(const moe_groups &g, int32_t dtype, int32_t D, const void *x, void *rows, hipStream_t s);
// w NULL: weights of 1
hipError_t launch_combine_rows(const moe_groups &g, int32_t y_dtype, int32_t out_dtype, int32_t D, const void *y,
                               const float *w, void *out, hipStream_t s);
hipError_t launch_combine_backward(const moe_groups &g, int32_t y_dtype, int32_t out_dtype, int32_t D,
                                   const void *d_out, const void *y, const float *w, void *d_y, float *d_w,
                                   hipStream_t s);

// ---- quantisers (block_quant.hip)
struct BlockQuantArgs {
    const int32_t *offsets;      // NULL: one group of `rows` rows
    const int32_t *sorted_slot;  // by token: row p is x[sorted_slot[p] / top_k]
    int32_t rows, n, top_k, C;
    int32_t tiles;  // of 128 columns per workgroup (set by the launcher)
    const uint16_t *x;
    uint8_t *codes;
    float *scales;
    uint8_t *col_codes;
    float *col_scales;
};
hipError_t launch_block_quant_rows(const BlockQuantArgs &a, hipStream_t s);
hipError_t launch_block_quant_columns(BlockQuantArgs a, hipStream_t s);  // with rows if codes is set
hipError_t launch_block_quant_weights(const uint16_t *w, int32_t E, int32_t N, int32_t K, uint8_t *codes, float *scales,
                                      hipStream_t s);

// ---- products (block_gemm.hip, block_wgrad.hip)
struct BlockGemmArgs {
    GroupView v;
    int32_t by_token;
    int32_t x_rows;  // rows of the rows form x
    int32_t R, C;  // reduction length and output columns: K, N (transposed: N, K)
    const uint8_t *x_codes;
    const float *x_scales;
    const uint8_t *w_codes;
    const float *w_scales;
    int64_t w_expert_bytes;    // N * K
    int32_t w_expert_scales;   // (N / 128) * (K / 128)
    int32_t w_kb;              // K / 128 (row length of the weight scales)
    uint16_t *out;
};
hipError_t launch_block_gemm(const BlockGemmArgs &a, bool transposed, hipStream_t s);

struct BlockWgradArgs {
    const int32_t *offsets;  // NULL: one group of `rows` rows
    int32_t rows, n, N, K;
    const uint8_t *g_codes, *x_codes;
    const float *g_scales, *x_scales;
    uint16_t *dw;
};
hipError_t launch_block_wgrad(const BlockWgradArgs &a, hipStream_t s);

}  // namespace moe
