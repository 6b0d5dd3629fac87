/*
 * moe_w4.h - C ABI of the grouped product with 4-bit integer weights, a scale and perhaps a zero
 * point for each group of values along the reduction, and bf16 rows (AMD MI355X, gfx950; the same
 * library): what programs that hold such checkpoints run between moe_sort and moe_combine, one
 * token at a time or many.
 *
 * Conventions: those of moe_ops.h (device pointers owned by the caller and 16-byte aligned, a
 * hipStream_t as void* that belongs to the current device, arguments checked on the host before
 * anything is enqueued, nothing synchronises, no allocation, no global state; an output that
 * overlaps another buffer of its call is refused).
 */
#ifndef BLOCK_SCALED_MOE_W4_H
#define BLOCK_SCALED_MOE_W4_H

#include "moe_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_W4_ABI_VERSION 1
int32_t moe_w4_abi_version(void);

/* Types of the scales. */
#define MOE_W4_SCALE_BF16 1
#define MOE_W4_SCALE_FP16 2

/*
 * Weights W [E][N][K] = scale * (code - zero): codes 0 .. 15, for each row one scale and one zero
 * point (0 .. 15; without zero points 8) per `group` of 32, 64 or 128 values along K. K is a multiple of the
 * group, N of any size. A checkpoint's form is row-major: codes [E][N][K/2] with the even value's code in a
 * byte's low half, scales [E][N][K/group] (bf16 or fp16), zeros [E][N][K/group] bytes.
 * Packed, the matrix is cut into tiles of 16 rows (n) and steps of 256 columns, both filled up at the end:
 *   codes  [E][N/16][K/256][2][64][4] 32-bit words: the step's halves of 128 columns; in half c lane 16 g + i
 *          has, in word j, row i's columns 128 c + 32 j + 8 g .. + 7: with r the word rotated right by 3 bits, value 2 m
 *          in bits 4 m .. 4 m + 3 of r, value 2 m + 1 in bits 16 + 4 m .. (m < 4)
 *   scales [E][N/16][K/256][16][256/group]; zeros in the same order, a byte 0x80 + 8 * zero point each
 * (divisions rounded up). What fills up are zero codes, scales and zero points.
 */
typedef struct moe_w4_weights {
    int32_t E, N, K;
    int32_t group;            /* 32, 64 or 128 */
    int32_t scale_type;       /* MOE_W4_SCALE_* */
    const uint32_t *codes;
    const uint16_t *scales;
    const uint8_t *zeros;     /* or NULL: 8 everywhere */
} moe_w4_weights;

/* Bytes of the packed arrays, from the size fields; 0 if those are invalid. Host only. */
size_t moe_w4_code_bytes(const moe_w4_weights *w);
size_t moe_w4_scale_bytes(const moe_w4_weights *w);
size_t moe_w4_zero_bytes(const moe_w4_weights *w);

/* Packs a checkpoint's arrays into w's buffers (w->zeros and zeros both or neither). A zero point's low four bits count. */
int32_t moe_w4_pack(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, const moe_w4_weights *w,
                    void *stream);

/* For sorted row p of expert e (g = NULL: every row, W's one expert)
 *   y[p][n] = sum over groups of scale[n] * (sum over the group of x * code - zero * sum of x)
 *   out[p]  = y[p], or with swiglu (N even): out[p][i] = y[p][i] / (1 + exp(-y[p][i])) * y[p][N/2 + i], i < N/2
 * x bf16 of rows of K; out [rows][N or N/2] of out_dtype (MOE_DT_*). Sums are fp32, rounded once.
 * by_token: x has T rows and sorted row p reads row sorted_slot[p] / top_k; otherwise rows = T * top_k, already
 * sorted. W has n experts (the local ones); rows behind the last local one are left as they are. A NaN or an infinity
 * makes every result that it enters not finite; they enter none of other rows. So may, on the way, values of x from
 * 2^116 on.
 * rows < 2^25, N and K up to 2^20; rows * K and N * K below 2^36 each. */
typedef struct moe_w4_gemm_args {
    int32_t rows;             /* rows of x */
    int32_t by_token, swiglu;
    int32_t out_dtype;
    const moe_groups *g;      /* host pointer or NULL */
    const uint16_t *x;
    moe_w4_weights w;
    void *out;
} moe_w4_gemm_args;
int32_t moe_w4_gemm(const moe_w4_gemm_args *a, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* BLOCK_SCALED_MOE_W4_H */
