/*
 * moe_ops.h - C ABI of the operators around the routed-expert layer of moe.h (AMD MI355X,
 * gfx950; the same library): the grouping of tokens by expert and the way back, each with
 * its gradient, and the expert product in FP8 with a scale for each block of 128, with both
 * of its gradients. For programs that run their own expert MLP between the router
 * (moe_route) and the combine, train the experts, or hold FP8 checkpoints with 128 x 128
 * block scales.
 *
 * Conventions: those of moe.h (device pointers owned by the caller and 16-byte aligned, a
 * hipStream_t as void*, arguments checked on the host before anything is enqueued, nothing
 * synchronises, no allocation, no global state). `stream` must belong to the current
 * device. An output that overlaps an input of its call or another output is refused
 * (MOE_ERR_INVALID_ARG) unless the call allows it; the groups' own arrays, which nothing
 * else may write, are not compared. The row operators pass NaN and infinite values through
 * to the rows and sums they belong to and to no others; what they do to a quantised block
 * stands at the format below.
 */
#ifndef BLOCK_SCALED_MOE_OPS_H
#define BLOCK_SCALED_MOE_OPS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OPS_ABI_VERSION 1
int32_t moe_ops_abi_version(void);

/* Element types of rows. */
#define MOE_DT_BF16 1
#define MOE_DT_FP32 2

/* ------------------------------------------------------------------ tokens by expert
 * Slot s = t * top_k + j is token t's j-th routed expert topk_idx[t][j]; it is local when
 * that lies in [e_begin, e_end). Any other value (a remote expert, -1 for padding) has no
 * row here. The S local slots sorted by expert, stable in s, are the sorted rows; arrays of
 * sorted rows have room for T * top_k rows, of which calls read and write the first S and
 * leave the others as they are. The same expert may occur twice in a token's list.
 * n = e_end - e_begin local experts. S is known on the device only (offsets[n]). */
typedef struct moe_groups {
    int32_t T, top_k;         /* tokens, 1 <= top_k <= 8                                  */
    int32_t E;                /* routed experts, 1 <= E <= 4096                           */
    int32_t e_begin, e_end;   /* local experts, 0 <= e_begin < e_end <= E                 */
    int32_t *offsets;         /* [n + 1] first sorted row of each local expert; [n] = S   */
    int32_t *sorted_slot;     /* [T * top_k] slot of each sorted row; -1 behind row S     */
    int32_t *slot_pos;        /* [T * top_k] sorted row of each slot, -1 if not local     */
    void *plan;               /* work lists of the grouped products, moe_groups_plan_bytes */
    size_t plan_bytes;
} moe_groups;

/* Bytes of `plan`: from the size fields, 0 if those are invalid. Host only. */
size_t moe_groups_plan_bytes(const moe_groups *g);

/* Fills offsets, sorted_slot, slot_pos and the plan from topk_idx [T][top_k]. The calls
 * below read them and may run at the same time on different streams after it. T = 0 is
 * allowed (all groups empty). */
int32_t moe_sort(const moe_groups *g, const int32_t *topk_idx, void *stream);

/* rows[p] = x[sorted_slot[p] / top_k] for p < S. x [T][D], rows [T * top_k][D], both of
 * type dtype (MOE_DT_*). This call and the next three: T < 2^24, 1 <= D <= 2^30. */
int32_t moe_gather(const moe_groups *g, int32_t dtype, int32_t D, const void *x, void *rows, void *stream);

/* Gradient of moe_gather: dx[t] = sum over the token's local slots, j ascending, of
 * d_rows[slot_pos], in fp32, rounded once; a token without one gets zeros. */
int32_t moe_gather_backward(const moe_groups *g, int32_t dtype, int32_t D, const void *d_rows, void *dx, void *stream);

/* out[t] = sum over the token's local slots, j ascending, of w[t][j] * y[slot_pos], fp32
 * fused multiply-adds, rounded once to out_dtype; a token without a local slot gets zeros.
 * y [T * top_k][D] of y_dtype, w fp32 [T][top_k], out [T][D]. */
int32_t moe_combine(const moe_groups *g, int32_t y_dtype, int32_t out_dtype, int32_t D, const void *y, const float *w,
                    void *out, void *stream);

/* Gradient of moe_combine for d_out [T][D] of out_dtype:
 *   d_y[slot_pos] = w[t][j] * d_out[t]  (rounded once to y_dtype; rows behind S untouched)
 *   d_w[t][j]     = sum over D of d_out[t] * y[slot_pos], fp32; 0 for a slot not local.
 * d_w may be w. */
int32_t moe_combine_backward(const moe_groups *g, int32_t y_dtype, int32_t out_dtype, int32_t D, const void *d_out,
                             const void *y, const float *w, void *d_y, float *d_w, void *stream);

/* ------------------------------------------------------------------ FP8, blocks of 128
 * E4M3 (OCP "FN") codes with one fp32 scale per block of 128: s = fl32(max |block| / 448),
 * 1 for an all-zero block; code = E4M3(fl32(x / s)), nearest, ties to even. The value is
 * code * s. A NaN or an infinity makes its block's scale a NaN or an infinity (the codes are
 * then not specified), and with it every result that the block enters. All dimensions that blocks run along are multiples of 128 up to 2^24.
 *   rows     codes [C/128][R][128] (the rows' first blocks, then their second ones, ..),
 *            scales [R][S], S = C/128 rounded up to a multiple of 4 (the rest of a row is
 *            neither written nor used): blocks of 1 x 128; R < 2^25 and R * S < 2^30
 *   columns  of sorted rows, blocks of 128 x 1: expert e's rows in runs of 128 from its first
 *            row (the last one padded with zeros), run i at block b = offsets[e] / 128 + e + i
 *            (integer division; blocks that belong to no run are never read):
 *            codes [blocks][C/32][2][4][32][16]: 32 columns, then the run's 64-row halves,
 *            16-row quarters of a half, column, row; scales [blocks][C];
 *            blocks = moe_block_column_blocks(rows, n)
 *   weights  W [E][N][K], codes in moe.h's tiled layout of MOE_FMT_FP8
 *            ([E][N/32][K/64][4][32][16]), scales [E][N/128][K/128]: blocks of 128 x 128 */

/* Expert weights [E][N][K]; device buffers set by the caller. */
typedef struct moe_block_weights {
    int32_t E, N, K;   /* N % 128 == 0, K % 128 == 0 */
    const uint8_t *codes;
    const float *scales;   /* 4-byte aligned: experts of a longer array may be given */
} moe_block_weights;

/* Runs of 128 rows (blocks) that the column form of `rows` sorted rows in `n` groups has
 * room for: rows / 128 + n. 0 if rows < 0 or n < 1. Host only. */
int64_t moe_block_column_blocks(int32_t rows, int32_t n);

/* Quantise bf16 x [rows][C] by rows (codes, scales), by columns (col_codes, col_scales), or
 * both from one read. g = NULL: every row (fewer than 2^30), one group. g given: rows =
 * T * top_k sorted rows, of which the S local ones are quantised; or, with by_token, x is
 * [T][C] and sorted row p is x[sorted_slot[p] / top_k] (columns only; rows = T). */
typedef struct moe_block_quantize_args {
    int32_t rows, C;          /* C % 128 == 0 */
    int32_t by_token;
    const moe_groups *g;      /* host pointer or NULL */
    const uint16_t *x;
    uint8_t *codes;           /* by rows, or NULL */
    float *scales;
    uint8_t *col_codes;       /* by columns, or NULL */
    float *col_scales;
} moe_block_quantize_args;
int32_t moe_block_quantize(const moe_block_quantize_args *a, void *stream);

/* Quantise bf16 weights w [E][N][K] into w's buffers `codes` and `scales` (tiled layout). */
int32_t moe_block_quantize_weights(const uint16_t *w, int32_t E, int32_t N, int32_t K, uint8_t *codes, float *scales,
                                   void *stream);
/* Codes of a checkpoint, row-major [E][N][K], into the tiled layout (scales stay as they
 * are). */
int32_t moe_block_pack_weights(const uint8_t *rowmajor, int32_t E, int32_t N, int32_t K, uint8_t *codes, void *stream);

/* Grouped product with W: for sorted row p of expert e (g = NULL: every row, W's one expert)
 *   transposed = 0: out[p][n] = sum over K-blocks of fl32(sx * sw) * sum over the block of cx * cw
 *   transposed = 1: out[p][k] = the same over N-blocks with W transposed (the gradient of the
 *                   former's input from the gradient of its output)
 * x holds the rows form of length K (N if transposed), out is bf16 [rows][N] ([rows][K]).
 * A block's sum is formed by the gfx950 FP8 MFMA, which drops what lies more than 13 bits below
 * the largest of the products it adds (about 2^-16 of the sum's size on normally distributed
 * values, far below the E4M3 rounding of the operands and the bf16 rounding of the result);
 * the sum over blocks is in fp32 in a fixed order, with one rounding to bf16.
 * by_token (not with transposed): x has T rows and sorted row p reads row sorted_slot[p] / top_k;
 * otherwise rows = T * top_k, already sorted. W has n experts (the local ones). */
typedef struct moe_block_gemm_args {
    int32_t rows;             /* rows of x */
    int32_t by_token, transposed;
    const moe_groups *g;      /* host pointer or NULL */
    const uint8_t *x_codes;
    const float *x_scales;
    moe_block_weights w;
    uint16_t *out;
} moe_block_gemm_args;
int32_t moe_block_gemm(const moe_block_gemm_args *a, void *stream);

/* Gradient of every expert's weight from column forms of the output gradient (N columns) and
 * of the input (K columns) of the same sorted rows:
 *   dw[e][n][k] = sum over e's runs of 128 rows of sum over the run of cg * cx, times sg * sx
 * bf16 [E][N][K], accumulated in fp32 in ascending order; zeros for an expert without rows.
 * g = NULL: one group of `rows` < 2^30 rows (E = 1). N % 128 == 0, K % 128 == 0. */
typedef struct moe_block_wgrad_args {
    int32_t rows;             /* T * top_k, or the rows of the one group */
    int32_t N, K;
    const moe_groups *g;      /* host pointer or NULL */
    const uint8_t *g_codes;   /* columns of the output gradient */
    const float *g_scales;
    const uint8_t *x_codes;   /* columns of the input */
    const float *x_scales;
    uint16_t *dw;
} moe_block_wgrad_args;
int32_t moe_block_wgrad(const moe_block_wgrad_args *a, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* BLOCK_SCALED_MOE_OPS_H */
