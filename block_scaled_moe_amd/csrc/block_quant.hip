// block_quant.hip - quantisers to E4M3 with one fp32 scale per block of 128
// (include/moe_ops.h): rows (1 x 128), columns of sorted rows (128 x 1), weights (128 x 128).
//
// s = fl32(max |block| / 448) (1 for a zero block), code = E4M3(fl32(x / s)), nearest, ties to
// even. All are bound by memory: 2 bytes read and 1 written per value (2 by rows and by
// columns), one pass, the block's maximum taken in registers. 8191 x 4096 bf16: rows 23 to 25 us (4.1 to
// 4.5 TB/s), columns 25 us (4.1), both 36 us (3.8); weights 32 x 4096 x 4096 302 us (5.3). Runs that are
// mostly padding cost the whole run's time: 17108 rows of 4096 in 96 uneven groups by both 100 us, their
// input's 2560 columns by token 46 us.
#include "formats.h"
#include "ops_internal.h"

#include <type_traits>

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
        s = amax != 0.0f ? amax / 448.0f : 1.0f;  // a NaN stays one
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

// Maxima are taken of magnitudes as bit patterns, two bf16 values a word: they order like the values, and a
// NaN or an infinity, above them all, reaches the scale (a maximum of floats drops a NaN).
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) { return w & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ float max_of(uint32_t m) { return __uint_as_float(max(m & 0xffff0000u, m << 16)); }

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
        uint32_t m = max2(max2(magnitudes(u.x), magnitudes(u.y)), max2(magnitudes(u.z), magnitudes(u.w)));
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) m = max2(m, __shfl_xor(m, off));
        const Divisor d(max_of(m));
        uint2 c;
        c.x = codes4(d.quotient(x[0]), d.quotient(x[1]), d.quotient(x[2]), d.quotient(x[3]));
        c.y = codes4(d.quotient(x[4]), d.quotient(x[5]), d.quotient(x[6]), d.quotient(x[7]));
        reinterpret_cast<uint2 *>(a.codes)[((int64_t)blk * a.rows + row) * 16 + sub] = c;
        if (sub == 0) a.scales[row * scale_stride(a.C) + blk] = d.s;
    }
}

// ---- columns (and rows): one workgroup takes a run of 128 sorted rows of one expert and
// kColumnTiles tiles of 128 columns (one in small calls). Thread (q, h) holds columns 4q..4q+3 of rows 16h..16h+15:
// its loads are 8 bytes, 256 consecutive bytes a row over 32 threads, the next tile's issued
// before this one is quantised, and it stores the 16 codes of one column as 16 bytes. A block's
// two divisions are done once, by one lane, and reach the others through LDS.
constexpr int kColumnTiles = 4;

// v[r] holds this lane's part of the maxima of row r (its even and its odd columns') over the 16 lanes of a
// DPP row; returns the whole maxima of row (lane & 15). Each step gives half of its rows to a partner lane and takes
// the partner's part of the other half: partners l ^ 8, l ^ 7, l ^ 2, l ^ 1 reach all 16 lanes.
__device__ __forceinline__ uint32_t row_maxima(uint32_t (&v)[16], int lane) {
#define MOE_HALVE(COUNT, BIT, CTRL)                                                                               \
    _Pragma("unroll") for (int r = 0; r < COUNT; ++r) {                                                           \
        const uint32_t keep = (lane & BIT) ? v[r + COUNT] : v[r], give = (lane & BIT) ? v[r] : v[r + COUNT];      \
        v[r] = max2(keep, __builtin_amdgcn_update_dpp(0, give, CTRL, 0xF, 0xF, true));                            \
    }
    MOE_HALVE(8, 8, 0x128)  // row_ror:8
    MOE_HALVE(4, 4, 0x141)  // row_half_mirror
    MOE_HALVE(2, 2, 0x4E)   // quad_perm 2, 3, 0, 1
    MOE_HALVE(1, 1, 0xB1)   // quad_perm 1, 0, 3, 2
#undef MOE_HALVE
    return v[0];
}

// Four codes with the scale s, r = fl32(1 / s); FAST where the short quotient serves (r != 0)
template <bool FAST>
__device__ __forceinline__ uint32_t quotient_codes(const float (&x)[4], float s, float r) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = FAST ? quotient_by(x[i], s, r) : x[i] / s;
    return codes4(v[0], v[1], v[2], v[3]);
}

template <bool TOKEN, bool ROWS>
__global__ void __launch_bounds__(kThreads, 3) columns_kernel(const BlockQuantArgs a) {
    __shared__ __attribute__((aligned(16))) uint16_t col_max[8][128];  // magnitudes' bits
    __shared__ __attribute__((aligned(16))) float col_s[128], col_r[128];
    __shared__ __attribute__((aligned(16))) float row_s[8][16], row_r[8][16];
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
    int32_t token[TOKEN ? 16 : 1];
    if (TOKEN) {
#pragma unroll
        for (int r = 0; r < 16; ++r) token[r] = a.sorted_slot[r0 + (16 * h + r < left ? 16 * h + r : 0)] / a.top_k;
    }
    const uint16_t *src = a.x + (TOKEN ? 0 : (int64_t)(r0 + 16 * h) * a.C) + 4 * q;
    auto load = [&](uint2 (&u)[16], int ct) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            u[r] = make_uint2(0u, 0u);
            if (16 * h + r < left)
                u[r] = *reinterpret_cast<const uint2 *>(src + (TOKEN ? (int64_t)token[r] * a.C : (int64_t)r * a.C) + ct * 128);
        }
    };
    const int ct1 = min(kb, (int)(blockIdx.y + 1) * a.tiles);
    uint2 u[16], next[16];
    load(next, blockIdx.y * a.tiles);
#pragma clang loop unroll(disable)
    for (int ct = blockIdx.y * a.tiles; ct < ct1; ++ct) {
#pragma unroll
        for (int r = 0; r < 16; ++r) u[r] = next[r];
        if (ct + 1 < ct1) load(next, ct + 1);
        uint32_t m0 = 0, m1 = 0, rm[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const uint32_t a0 = magnitudes(u[r].x), a1 = magnitudes(u[r].y);
            m0 = max2(m0, a0);
            m1 = max2(m1, a1);
            rm[r] = max2(a0, a1);
        }
        *reinterpret_cast<uint2 *>(&col_max[h][4 * q]) = make_uint2(m0, m1);
        bool fast = true;
        if (ROWS) {  // the 32 threads of a row are half a wave
            uint32_t top = row_maxima(rm, tid & 15);
            top = max2(top, __shfl_xor(top, 16));
            const Divisor d(max_of(top));
            fast = __all(d.fast);
            if (q < 16) {
                row_s[h][q] = d.s;
                row_r[h][q] = d.r;
                if (16 * h + q < left) a.scales[(int64_t)(r0 + 16 * h + q) * scale_stride(a.C) + ct] = d.s;
            }
        }
        __syncthreads();
        if (tid < 128) {
            uint32_t cm = col_max[0][tid];
#pragma unroll
            for (int g = 1; g < 8; ++g) cm = max(cm, (uint32_t)col_max[g][tid]);
            const Divisor d(__uint_as_float(cm << 16));
            col_s[tid] = d.s;
            col_r[tid] = d.r;
            a.col_scales[(int64_t)run * a.C + ct * 128 + tid] = d.s;
        }
        if (ROWS) {
            auto store_rows = [&](auto fast_c) __attribute__((always_inline)) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float x[4];
                    widen(u[r].x, x[0], x[1]);
                    widen(u[r].y, x[2], x[3]);
                    const uint32_t c = quotient_codes<decltype(fast_c)::value>(x, row_s[h][r], row_r[h][r]);
                    if (16 * h + r < left)
                        *reinterpret_cast<uint32_t *>(a.codes + ((int64_t)ct * a.rows + r0 + 16 * h + r) * 128 + 4 * q) = c;
                }
            };
            if (fast) store_rows(std::true_type{});
            else store_rows(std::false_type{});
        }
        __syncthreads();
        uint8_t *dst = a.col_codes + (int64_t)run * a.C * 128 + ct * 16384 + (q >> 3) * 4096 + (h >> 2) * 2048 + (h & 3) * 512 +
                       (q & 7) * 64;
        const float4 cs = *reinterpret_cast<const float4 *>(&col_s[4 * q]), cr = *reinterpret_cast<const float4 *>(&col_r[4 * q]);
        auto store_columns = [&](auto fast_c) __attribute__((always_inline)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float s = c == 0 ? cs.x : c == 1 ? cs.y : c == 2 ? cs.z : cs.w;
                const float r = c == 0 ? cr.x : c == 1 ? cr.y : c == 2 ? cr.z : cr.w;
                uint32_t code[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint32_t word = c < 2 ? u[4 * j + b].x : u[4 * j + b].y;
                        x[b] = __uint_as_float(c & 1 ? word & 0xffff0000u : word << 16);
                    }
                    code[j] = quotient_codes<decltype(fast_c)::value>(x, s, r);
                }
                *reinterpret_cast<uint4 *>(dst + 16 * c) = make_uint4(code[0], code[1], code[2], code[3]);
            }
        };
        if (__all(cr.x != 0.0f && cr.y != 0.0f && cr.z != 0.0f && cr.w != 0.0f)) store_columns(std::true_type{});
        else store_columns(std::false_type{});
        __syncthreads();  // before the next tile writes the maxima and scales
    }
}

// ---- weights: one workgroup per 128 x 128 block; thread (q, r) holds 16 columns (one
// quarter row of a 32 x 64 tile) of rows r, r + 32, r + 64, r + 96.
__global__ void __launch_bounds__(kThreads) weights_kernel(const uint16_t *__restrict__ w, int32_t N, int32_t K,
                                                           uint8_t *__restrict__ codes, float *__restrict__ scales) {
    __shared__ uint32_t part[kThreads / 64];
    const int tid = threadIdx.x, q = tid & 7, r = tid >> 3;
    const int kblocks = K / 128, nblocks = N / 128;
    const int64_t b = blockIdx.x;
    const int kb = (int)(b % kblocks), nb = (int)((b / kblocks) % nblocks);
    const int64_t e = b / ((int64_t)kblocks * nblocks);
    uint4 u[4][2];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 *src = reinterpret_cast<const uint4 *>(w + (e * N + nb * 128 + 32 * i + r) * K + kb * 128 + 16 * q);
        u[i][0] = src[0];
        u[i][1] = src[1];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            m = max2(m, max2(max2(magnitudes(u[i][j].x), magnitudes(u[i][j].y)), max2(magnitudes(u[i][j].z), magnitudes(u[i][j].w))));
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = max2(m, __shfl_xor(m, off));
    if ((tid & 63) == 0) part[tid >> 6] = m;
    __syncthreads();
    m = max2(max2(part[0], part[1]), max2(part[2], part[3]));
    const Divisor d(max_of(m));
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

hipError_t launch_block_quant_columns(BlockQuantArgs a, hipStream_t s) {
    const int64_t runs = a.offsets ? (int64_t)a.rows / 128 + a.n : ((int64_t)a.rows + 127) / 128;
    const int kb = a.C / 128;
    // fewer than a workgroup or two a CU with one tile each: the run's latency counts (2400 rows of 256 by
    // both 11.3 -> 8.0 us)
    a.tiles = runs * kb < 512 ? 1 : kColumnTiles;
    const dim3 grid((unsigned)runs, (unsigned)((kb + a.tiles - 1) / a.tiles));
    if (a.sorted_slot) hipLaunchKernelGGL((columns_kernel<true, false>), grid, dim3(kThreads), 0, s, a);
    else if (a.codes) hipLaunchKernelGGL((columns_kernel<false, true>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((columns_kernel<false, false>), grid, dim3(kThreads), 0, s, a);
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
