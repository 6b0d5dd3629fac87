// w4_gemm.hip - grouped product of bf16 rows with 4-bit weights that have a scale (and a zero point) per group along
// the reduction (include/moe_w4.h, moe_w4_gemm), and the packing of such weights.
//
//   y[p][n] = sum over groups g of s[n][g] (sum over k in g of x[p][k] (16 + q[n][k])  -  (16 + z[n][g]) sum over k in g of x[p][k])
//
// 16 + q is a bf16 whose upper four mantissa bits are the code, so that two of the MFMA's operands come from a word of
// eight codes by one shift and one AND-OR; both sums, of x (16 + q) and of x itself, are fp32 sums of the bf16
// MFMA (the second against ones), and what 16 brings in is taken off group by group, where it is at most a few times
// larger than the group's own sum. Scales and zero points meet the sums in fp32: nothing of the weights is rounded.
#include "block_mma.h"
#include "w4_internal.h"

#include <type_traits>

namespace moe {
namespace {

using namespace block;

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- packing

__global__ void __launch_bounds__(256) pack_codes_kernel(const uint8_t *__restrict__ src, int32_t N, int32_t K, int32_t tiles,
                                                         int32_t steps, int64_t words, uint32_t *__restrict__ dst) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) {
        const int j = i & 3, lane = (i >> 2) & 63, half = (i >> 8) & 1;
        const int64_t at = i >> 9, step = at % steps, tile = at / steps % tiles, e = at / steps / tiles;
        const int64_t n = 16 * tile + (lane & 15), k = 256 * step + 128 * half + 32 * j + 8 * (lane >> 4);
        uint32_t r = 0;
        if (n < N && k < K) {  // K % 32 == 0: all eight
            const uint32_t b = *reinterpret_cast<const uint32_t *>(src + ((e * N + n) * K + k) / 2);
#pragma unroll
            for (int m = 0; m < 4; ++m) r |= ((b >> (8 * m)) & 15) << (4 * m) | ((b >> (8 * m + 4)) & 15) << (16 + 4 * m);
        }
        dst[i] = r << 3 | r >> 29;
    }
}

// scales (two bytes) or zero points (one): [E][N][groups] -> [E][N/16][K/256][16][per_step]
template <typename T>
__global__ void __launch_bounds__(256) pack_groups_kernel(const T *__restrict__ src, int32_t N, int32_t groups, int32_t per_step,
                                                          int32_t tiles, int32_t steps, int64_t n_out, T *__restrict__ dst) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n_out; i += (int64_t)gridDim.x * 256) {
        const int64_t g = i % per_step, row = i / per_step % 16, at = i / per_step / 16;
        const int64_t step = at % steps, tile = at / steps % tiles, e = at / steps / tiles;
        const int64_t n = 16 * tile + row, k = step * per_step + g;
        T v = 0;
        if (n < N && k < groups) v = src[(e * N + n) * groups + k];
        if constexpr (sizeof(T) == 1) v &= 15;
        dst[i] = v;
    }
}

// ---------------------------------------------------------------- few rows

// eight codes as 16 + q
__device__ __forceinline__ bf8 expand(uint32_t w) {
    const uint32_t mask = 0x00780078u, base = 0x41804180u;
    u32x4 r;
    r[0] = (w & mask) | base;
    r[1] = ((w >> 4) & mask) | base;
    r[2] = ((w >> 8) & mask) | base;
    r[3] = (__builtin_rotateright32(w, 12) & mask) | base;
    return __builtin_bit_cast(bf8, r);
}

template <bool HALF>
__device__ __forceinline__ float scale_value(uint32_t word, int upper) {
    const uint32_t u = upper ? word >> 16 : word & 0xFFFFu;
    if constexpr (HALF) return (float)__builtin_bit_cast(_Float16, (uint16_t)u);
    else return __uint_as_float(u << 16);
}

// Bound by the weights' bytes. A workgroup takes two column tiles of 16 (with swiglu one of the gate's columns and the
// same of the other half's) of one tile of rows, its four waves a quarter of the steps each, and the four partial sums meet
// in LDS in the waves' order. A wave's load of codes is 1 KiB in a row; those of the next step are in flight while the
// current one is multiplied.
template <int GROUP, bool HALF, bool ZEROS>
__global__ void __launch_bounds__(256, 3) stream_kernel(const W4GemmArgs p) {
    constexpr int kGroups = kW4Step / GROUP;      // per step
    constexpr int kWords = (kGroups + 1) / 2;     // of scales
    constexpr int kZeroWords = (kGroups + 3) / 4;
    __shared__ __attribute__((aligned(16))) float part[4][64][36];
    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int N = p.w.N, K = p.w.K;
    const int nb = p.swiglu ? (p.C + 15) / 16 : (p.C + 31) / 32;
    const int n_tiles = p.v.offsets ? scalar_load(&p.v.ctrl->n_tiles) : p.v.max_tiles;
    const int tile = blockIdx.x / nb, cb = blockIdx.x % nb;
    if (tile >= n_tiles) return;
    int e = 0, p0 = tile * kGroupTile, rows = p.v.rows - p0;
    if (p.v.offsets) {
        e = scalar_load(p.v.tile_expert + tile);
        p0 = scalar_load(p.v.tile_row0 + tile);
        rows = scalar_load(p.v.offsets + e + 1) - p0;
    }
    rows = min(rows, kGroupTile);
    const uint8_t *codes[2], *scales[2], *zeros[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        // this lane's weight row: past the end the last one, which is not stored
        const int n = p.swiglu ? min(16 * cb + i16, p.C - 1) + q * p.C : min(32 * cb + 16 * q + i16, N - 1);
        const int64_t at = ((int64_t)e * p.tiles + (n >> 4)) * p.steps, in = n & 15;
        codes[q] = reinterpret_cast<const uint8_t *>(p.w.codes) + at * 2048 + (16 * g + in) * 16;
        scales[q] = reinterpret_cast<const uint8_t *>(p.w.scales) + (at * 16 + in) * (2 * kGroups);
        zeros[q] = ZEROS ? p.w.zeros + (at * 16 + in) * kGroups : nullptr;
    }
    const int s0 = wave * p.steps / 4, s1 = (wave + 1) * p.steps / 4;

    struct Weights {
        u32x4 c[2][2];
        uint32_t s[2][kWords], z[2][kZeroWords];
    };
    auto load = [&](int s, Weights &w) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w.c[q][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(codes[q] + (int64_t)s * 2048 + h * 1024));
            const uint8_t *sp = scales[q] + (int64_t)s * (32 * kGroups);
            if constexpr (kWords == 1) {
                w.s[q][0] = *reinterpret_cast<const uint32_t *>(sp);
            } else if constexpr (kWords == 2) {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(sp);
                w.s[q][0] = v.x, w.s[q][1] = v.y;
            } else {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(sp);
#pragma unroll
                for (int i = 0; i < 4; ++i) w.s[q][i] = v[i];
            }
            if constexpr (ZEROS) {
                const uint8_t *zp = zeros[q] + (int64_t)s * (16 * kGroups);
                if constexpr (kGroups == 2) {
                    w.z[q][0] = *reinterpret_cast<const uint16_t *>(zp);
                } else if constexpr (kGroups == 4) {
                    w.z[q][0] = *reinterpret_cast<const uint32_t *>(zp);
                } else {
                    const u32x2 v = *reinterpret_cast<const u32x2 *>(zp);
                    w.z[q][0] = v.x, w.z[q][1] = v.y;
                }
            }
        }
    };

    // MT pieces of 16 rows from m0 on
    auto turn = [&](int m0, auto mt_c) __attribute__((always_inline)) {
        constexpr int MT = decltype(mt_c)::value;
        constexpr int kRuns = MT > 2 ? 4 : 8;  // of 32 columns whose rows are loaded together
        const uint16_t *x[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int pos = p0 + min(m0 + 16 * m + i16, rows - 1);
            const int64_t row = p.by_token ? p.v.sorted_slot[pos] / p.v.top_k : pos;
            x[m] = p.x + row * K + 8 * g;
        }
        f4 acc[MT][2] = {};
        Weights next;
        if (s0 < s1) load(s0, next);
        for (int s = s0; s < s1; ++s) {
            const Weights w = next;
            const int left = K / 32 - 8 * s;  // runs of 32 columns from here on
            const bf8 one = __builtin_bit_cast(bf8, (u32x4){0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
#pragma unroll
            for (int b = 0; b < 8 / kRuns; ++b) {
                u32x4 xv[kRuns][MT];
#pragma unroll
                for (int i = 0; i < kRuns; ++i)
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        xv[i][m] = (u32x4){0, 0, 0, 0};
                        if (kRuns * b + i < left) xv[i][m] = *reinterpret_cast<const u32x4 *>(x[m] + 256 * s + 32 * (kRuns * b + i));
                    }
                if (b == 0) load(min(s + 1, s1 - 1), next);
#pragma unroll
                for (int gr = b * (32 * kRuns / GROUP); gr < (b + 1) * (32 * kRuns / GROUP); ++gr) {
                    f4 sum[MT], d[MT][2];
#pragma unroll
                    for (int m = 0; m < MT; ++m) sum[m] = d[m][0] = d[m][1] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = gr * (GROUP / 32); i < (gr + 1) * (GROUP / 32); ++i) {
                        bf8 wv[2];
#pragma unroll
                        for (int q = 0; q < 2; ++q) wv[q] = expand(w.c[q][i >> 2][i & 3]);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const bf8 xo = __builtin_bit_cast(bf8, xv[i % kRuns][m]);
                            sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo, one, sum[m], 0, 0, 0);
#pragma unroll
                            for (int q = 0; q < 2; ++q) d[m][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo, wv[q], d[m][q], 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float f = scale_value<HALF>(w.s[q][gr / 2], gr & 1);
                        const float off = ZEROS ? 16.0f + (float)((w.z[q][gr / 4] >> (8 * (gr & 3))) & 255u) : 24.0f;
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int v = 0; v < 4; ++v) acc[m][q][v] = fmaf(fmaf(-off, sum[m][v], d[m][q][v]), f, acc[m][q][v]);
                    }
                }
            }
        }
        // accumulator v of (m, q): row 16 m + 4 g + v, column 16 q + i16
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int v = 0; v < 4; ++v) part[wave][16 * m + 4 * g + v][16 * q + i16] = acc[m][q][v];
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = 16 * m + (t >> 4);
            if (m0 + r >= rows) continue;
            float y[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int c = p.swiglu ? 16 * q + (t & 15) : 2 * (t & 15) + q;
                y[q] = part[0][r][c];
#pragma unroll
                for (int k = 1; k < 4; ++k) y[q] += part[k][r][c];
            }
            const int64_t row = (int64_t)(p0 + m0 + r) * p.C;
            if (p.swiglu) {
                const int c = 16 * cb + (t & 15);
                const float v = y[0] / (1.0f + expf(-y[0])) * y[1];
                if (c < p.C) {
                    if (p.out_dtype == MOE_DT_BF16) static_cast<uint16_t *>(p.out)[row + c] = __builtin_bit_cast(uint16_t, (__bf16)v);
                    else static_cast<float *>(p.out)[row + c] = v;
                }
            } else {
                const int c = 32 * cb + 2 * (t & 15);
                if (p.out_dtype == MOE_DT_BF16) {
                    uint16_t *o = static_cast<uint16_t *>(p.out) + row + c;
                    if (p.C % 2 == 0) {
                        if (c < p.C) *reinterpret_cast<uint32_t *>(o) = bf16_pair(y[0], y[1]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            if (c + q < p.C) o[q] = __builtin_bit_cast(uint16_t, (__bf16)y[q]);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (c + q < p.C) static_cast<float *>(p.out)[row + c + q] = y[q];
                }
            }
        }
    };
    using std::integral_constant;
    int m0 = 0;
    for (; rows - m0 > 32; m0 += 64) turn(m0, integral_constant<int, 4>{});
    if (rows - m0 > 16) turn(m0, integral_constant<int, 2>{});
    else if (rows > m0) turn(m0, integral_constant<int, 1>{});
}

// f is called with the group, whether scales are fp16, and whether there are zero points
template <typename F>
void by_form(const moe_w4_weights &w, F &&f) {
    using std::integral_constant;
    auto zeros = [&](auto group, auto half) {
        if (w.zeros) f(group, half, integral_constant<bool, true>{});
        else f(group, half, integral_constant<bool, false>{});
    };
    auto type = [&](auto group) {
        if (w.scale_type == MOE_W4_SCALE_FP16) zeros(group, integral_constant<bool, true>{});
        else zeros(group, integral_constant<bool, false>{});
    };
    if (w.group == 32) type(integral_constant<int, 32>{});
    else if (w.group == 64) type(integral_constant<int, 64>{});
    else type(integral_constant<int, 128>{});
}

unsigned grid_of(int64_t items) { return (unsigned)((items + 255) / 256 < 1 << 16 ? (items + 255) / 256 : 1 << 16); }

}  // namespace

hipError_t launch_w4_pack(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, const moe_w4_weights &w,
                          hipStream_t s) {
    const int32_t tiles = (int32_t)w4_tiles(w), steps = (int32_t)w4_steps(w), per_step = kW4Step / w.group, groups = w.K / w.group;
    const int64_t blocks = (int64_t)w.E * tiles * steps, n = blocks * 16 * per_step;
    hipLaunchKernelGGL(pack_codes_kernel, dim3(grid_of(blocks * 512)), dim3(256), 0, s, codes, w.N, w.K, tiles, steps, blocks * 512,
                       const_cast<uint32_t *>(w.codes));
    hipLaunchKernelGGL(pack_groups_kernel<uint16_t>, dim3(grid_of(n)), dim3(256), 0, s, scales, w.N, groups, per_step, tiles, steps, n,
                       const_cast<uint16_t *>(w.scales));
    if (zeros)
        hipLaunchKernelGGL(pack_groups_kernel<uint8_t>, dim3(grid_of(n)), dim3(256), 0, s, zeros, w.N, groups, per_step, tiles, steps, n,
                           const_cast<uint8_t *>(w.zeros));
    return hipGetLastError();
}

hipError_t launch_w4_gemm(const W4GemmArgs &a, hipStream_t s) {
    const int64_t nb = a.swiglu ? (a.C + 15) / 16 : (a.C + 31) / 32, groups = (int64_t)a.v.max_tiles * nb;
    if (groups >= 1 << 24) return hipErrorInvalidValue;  // a grid's threads are 32 bits
    by_form(a.w, [&](auto group, auto half, auto zeros) {
        constexpr int kGroup = decltype(group)::value;
        constexpr bool kHalf = decltype(half)::value, kZeros = decltype(zeros)::value;
        hipLaunchKernelGGL((stream_kernel<kGroup, kHalf, kZeros>), dim3((unsigned)groups), dim3(256), 0, s, a);
    });
    return hipGetLastError();
}

}  // namespace moe
