// block_quant.hip - quantisers to E4M3 with one fp32 scale per block of 128
// (include/moe_ops.h): rows (1 x 128), columns of sorted rows (128 x 1), weights (128 x 128).
//
// s = fl32(max |block| / 448) (1 for a zero block), code = E4M3(fl32(x / s)), nearest, ties to
// even. All are bound by memory: 2 bytes read and 1 written per value (2 by rows and by
// columns), one pass, the block's maximum taken in registers.
#include "formats.h"
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// fl32(x / s) with r = fl32(1 / s): for s in [2^-60, 2^60] one multiply and two fused
// multiply-adds give the correctly rounded quotient wherever it is not below 2^-12 (see
// quotient_by in formats.h), and smaller ones code to a signed zero either way; outside that range one division.
struct Divisor {
    float s, r;
    bool fast;
    __device__ __forceinline__ explicit Divisor(float amax) {
        s = amax > 0.0f ? amax / 448.0f : 1.0f;
        fast = s >= 0x1p-60f && s <= 0x1p60f;
        r = fast ? 1.0f / s : 0.0f;
    }
    __device__ __forceinline__ float quotient(float x) const { return fast ? quotient_by(x, s, r) : x / s; }
};

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    return e4m3_pack2<true>(e4m3_pack2<false>(0u, e4m3_clamp(a), e4m3_clamp(b)), e4m3_clamp(c), e4m3_clamp(d));
}

__device__ __forceinline__ void widen(uint32_t w, float &lo, float &hi) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
}

// ---- rows: 16 lanes per block, 8 values each. A workgroup takes four blocks of four rows at a
// time: a wave reads 1 KiB of one row, and each block's plane of codes gets 512 bytes in a row.
__global__ void __launch_bounds__(kThreads) rows_kernel(const BlockQuantArgs a) {
    const int32_t rows = a.offsets ? a.offsets[a.n] : a.rows;
    const int32_t kb = a.C / 128;
    const int sub = threadIdx.x & 15, quads = (kb + 3) / 4;
    const int64_t n = (int64_t)((rows + 3) / 4) * quads;
    for (int64_t w = blockIdx.x; w < n; w += gridDim.x) {
        const int64_t row = w / quads * 4 + (threadIdx.x >> 6);
        const int blk = (int)(w % quads) * 4 + ((threadIdx.x >> 4) & 3);
        if (row >= rows || blk >= kb) continue;
        const int64_t b = row * kb + blk;
        const uint4 u = reinterpret_cast<const uint4 *>(a.x)[b * 16 + sub];
        float x[8];
        widen(u.x, x[0], x[1]);
        widen(u.y, x[2], x[3]);
        widen(u.z, x[4], x[5]);
        widen(u.w, x[6], x[7]);
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
        const Divisor d(m);
        uint2 c;
        c.x = codes4(d.quotient(x[0]), d.quotient(x[1]), d.quotient(x[2]), d.quotient(x[3]));
        c.y = codes4(d.quotient(x[4]), d.quotient(x[5]), d.quotient(x[6]), d.quotient(x[7]));
        reinterpret_cast<uint2 *>(a.codes)[((int64_t)blk * a.rows + row) * 16 + sub] = c;
        if (sub == 0) a.scales[b] = d.s;
    }
}

// ---- columns (and rows): one workgroup takes a run of 128 sorted rows of one expert and
// kColumnTiles tiles of 128 columns. Thread (q, h) holds columns 4q..4q+3 of rows 16h..16h+15:
// its loads are 8 bytes, 256 consecutive bytes a row over 32 threads, and it stores the 16
// codes of one column as 16 bytes.
constexpr int kColumnTiles = 4;

__global__ void __launch_bounds__(kThreads) columns_kernel(const BlockQuantArgs a) {
    __shared__ float col_max[8][128];
    const int tid = threadIdx.x, q = tid & 31, h = tid >> 5;
    const int32_t run = blockIdx.x;
    // the run's expert: run b belongs to the last e with offsets[e] / 128 + e <= b
    int32_t first = 0, cnt = a.rows;  // the expert's first row and rows
    int32_t i = run;                  // run within the expert
    if (a.offsets) {
        int below = 0;
        for (int e0 = 0; e0 < a.n; e0 += 64) {
            const int e = e0 + (tid & 63);
            const bool le = e < a.n && a.offsets[e] / 128 + e <= run;
            below += __popcll(__ballot(le));
            if (!__all(le)) break;
        }
        const int e = below - 1;
        first = a.offsets[e];
        cnt = a.offsets[e + 1] - first;
        i = run - (first / 128 + e);
    }
    const int32_t left = cnt - 128 * i;  // rows of the run
    if (left <= 0) return;
    const int32_t r0 = first + 128 * i;
    const int kb = a.C / 128;
    int64_t src_row[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int row = 16 * h + r;
        const int32_t p = r0 + (row < left ? row : 0);
        src_row[r] = a.sorted_slot ? a.sorted_slot[p] / a.top_k : p;
    }
    for (int ct = blockIdx.y * kColumnTiles; ct < min(kb, (int)(blockIdx.y + 1) * kColumnTiles); ++ct) {
        uint2 u[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            u[r] = make_uint2(0u, 0u);
            if (16 * h + r < left) u[r] = *reinterpret_cast<const uint2 *>(a.x + src_row[r] * a.C + ct * 128 + 4 * q);
        }
        float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float x[4];
            widen(u[r].x, x[0], x[1]);
            widen(u[r].y, x[2], x[3]);
#pragma unroll
            for (int c = 0; c < 4; ++c) m[c] = fmaxf(m[c], fabsf(x[c]));
        }
        __syncthreads();  // the previous tile's reads of col_max
#pragma unroll
        for (int c = 0; c < 4; ++c) col_max[h][4 * q + c] = m[c];
        if (a.codes) {  // by rows: the 32 threads of a row are half a wave
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float x[4];
                widen(u[r].x, x[0], x[1]);
                widen(u[r].y, x[2], x[3]);
                float rm = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) rm = fmaxf(rm, __shfl_xor(rm, off));
                const Divisor d(rm);
                const int row = 16 * h + r;
                if (row < left) {
                    const int64_t p = r0 + row;
                    *reinterpret_cast<uint32_t *>(a.codes + ((int64_t)ct * a.rows + p) * 128 + 4 * q) =
                        codes4(d.quotient(x[0]), d.quotient(x[1]), d.quotient(x[2]), d.quotient(x[3]));
                    if (q == 0) a.scales[p * kb + ct] = d.s;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float cm = col_max[0][4 * q + c];
#pragma unroll
            for (int g = 1; g < 8; ++g) cm = fmaxf(cm, col_max[g][4 * q + c]);
            const Divisor d(cm);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t word = c < 2 ? u[4 * j + b].x : u[4 * j + b].y;
                    v[b] = d.quotient(__uint_as_float(c & 1 ? word & 0xffff0000u : word << 16));
                }
                w[j] = codes4(v[0], v[1], v[2], v[3]);
            }
            const int64_t col = ct * 128 + 4 * q + c;
            uint8_t *dst = a.col_codes + (int64_t)run * a.C * 128 + (col >> 5) * 4096 + (h >> 2) * 2048 + (h & 3) * 512 +
                           (col & 31) * 16;
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            if (h == 0) a.col_scales[(int64_t)run * a.C + col] = d.s;
        }
    }
}

// ---- weights: one workgroup per 128 x 128 block; thread (q, r) holds 16 columns (one
// quarter row of a 32 x 64 tile) of rows r, r + 32, r + 64, r + 96.
__global__ void __launch_bounds__(kThreads) weights_kernel(const uint16_t *__restrict__ w, int32_t N, int32_t K,
                                                           uint8_t *__restrict__ codes, float *__restrict__ scales) {
    __shared__ float part[kThreads / 64];
    const int tid = threadIdx.x, q = tid & 7, r = tid >> 3;
    const int kblocks = K / 128, nblocks = N / 128;
    const int64_t b = blockIdx.x;
    const int kb = (int)(b % kblocks), nb = (int)((b / kblocks) % nblocks);
    const int64_t e = b / ((int64_t)kblocks * nblocks);
    uint4 u[4][2];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 *src = reinterpret_cast<const uint4 *>(w + (e * N + nb * 128 + 32 * i + r) * K + kb * 128 + 16 * q);
        u[i][0] = src[0];
        u[i][1] = src[1];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t word[4] = {u[i][j].x, u[i][j].y, u[i][j].z, u[i][j].w};
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                float lo, hi;
                widen(word[d], lo, hi);
                m = fmaxf(m, fmaxf(fabsf(lo), fabsf(hi)));
            }
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    if ((tid & 63) == 0) part[tid >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const Divisor d(m);
    if (tid == 0) scales[b] = d.s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t word[4] = {u[i][j].x, u[i][j].y, u[i][j].z, u[i][j].w};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[4];
                widen(word[2 * h], v[0], v[1]);
                widen(word[2 * h + 1], v[2], v[3]);
                c[2 * j + h] = codes4(d.quotient(v[0]), d.quotient(v[1]), d.quotient(v[2]), d.quotient(v[3]));
            }
        }
        const int64_t tile = (int64_t)(nb * 4 + i) * (K / 64) + kb * 2 + (q >> 2);
        *reinterpret_cast<uint4 *>(codes + e * N * K + tile * 2048 + (q & 3) * 512 + r * 16) =
            make_uint4(c[0], c[1], c[2], c[3]);
    }
}

}  // namespace

hipError_t launch_block_quant_rows(const BlockQuantArgs &a, hipStream_t s) {
    const int64_t want = (int64_t)((a.rows + 3) / 4) * ((a.C / 128 + 3) / 4);
    hipLaunchKernelGGL(rows_kernel, dim3((unsigned)(want < 16384 ? want : 16384)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_block_quant_columns(const BlockQuantArgs &a, hipStream_t s) {
    const int64_t runs = a.offsets ? (int64_t)a.rows / 128 + a.n : ((int64_t)a.rows + 127) / 128;
    const int tiles = (a.C / 128 + kColumnTiles - 1) / kColumnTiles;
    hipLaunchKernelGGL(columns_kernel, dim3((unsigned)runs, (unsigned)tiles), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_block_quant_weights(const uint16_t *w, int32_t E, int32_t N, int32_t K, uint8_t *codes, float *scales,
                                      hipStream_t s) {
    const int64_t blocks = (int64_t)E * (N / 128) * (K / 128);
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(weights_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, w, N, K, codes, scales);
    return hipGetLastError();
}

}  // namespace moe
