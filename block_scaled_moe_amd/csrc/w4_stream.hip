// w4_stream.hip - product of few rows a group with 4-bit weights (include/moe_w4.h, moe_w4_gemm; the arithmetic stands in
// w4_mma.h), and the choice between the kernels.
//
// Bound by the weights' bytes. A wave takes two column tiles of 16 (with swiglu one of the first half's columns and the same of
// the second half's) of one tile of rows; its load of codes is 1 KiB in a row, and those of the next step are in flight
// while the current one is multiplied. 64 tokens on 96 of 384 experts, 5120 x 4096, groups of 32 with zero points: 147 us, 6.0
// TB/s. One token, eight experts 4096 x 2560, groups of 128: 13.2 us for 41 MB; one row, 5120 x 4096: 8.1 us for 11.5 MB: a load's
// latency, the rows' way into LDS and the launch.
#include "w4_mma.h"

namespace moe {
namespace {

using namespace w4;

// A step of 256 columns of one weight row as a lane holds it: four words of codes of each half, the groups' scales and zero points.
template <int GROUP, bool ZEROS>
struct Step {
    static constexpr int kGroups = kW4Step / GROUP, kWords = (kGroups + 1) / 2, kZeroWords = (kGroups + 3) / 4;
    u32x4 c[2];
    uint32_t s[kWords], z[kZeroWords];
    // from the step's places in the packed arrays, and this lane's in them
    __device__ __forceinline__ void load(const uint8_t *codes, uint32_t code_at, const uint8_t *scales, const uint8_t *zeros,
                                         uint32_t scale_at) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            c[h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(codes + (code_at + h * 1024)));
        const uint8_t *sp = scales + scale_at;
        if constexpr (kWords == 1) {
            s[0] = *reinterpret_cast<const uint32_t *>(sp);
        } else if constexpr (kWords == 2) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(sp);
            s[0] = v.x, s[1] = v.y;
        } else {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(sp);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = v[i];
        }
        if constexpr (ZEROS) {
            const uint8_t *zp = zeros + scale_at / 2;
            if constexpr (kGroups == 2) {
                z[0] = *reinterpret_cast<const uint16_t *>(zp);
            } else if constexpr (kGroups == 4) {
                z[0] = *reinterpret_cast<const uint32_t *>(zp);
            } else {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(zp);
                z[0] = v.x, z[1] = v.y;
            }
        }
    }
};

// Up to 16 or 32 rows a turn: they go into LDS once for the workgroup's eight waves (in parts of the reduction where they
// do not fit), and KS waves share two column tiles, each with a part of the steps; their sums meet in LDS in the waves' order.
// 16 + z is a bf16 as 16 + q is, so it is taken off by a second MFMA on the same rows, which leaves four multiply-adds
// for four results and group.
constexpr int kStreamWaves = 8, kStreamX = 60 * 1024;  // waves, LDS bytes of rows of a workgroup: two of them a CU
template <int GROUP, bool HALF, bool ZEROS, int KS>
__global__ void __launch_bounds__(64 * kStreamWaves, 4) stream_kernel(const W4GemmArgs p) {
    constexpr int kGroups = kW4Step / GROUP;      // per step
    constexpr int kBlocks = kStreamWaves / KS;    // of two column tiles a workgroup
    // two pieces of 16 rows share the expanded codes where registers (not beside finest groups or zero points) and LDS (not
    // beside shared columns) allow it
    constexpr int kUnit = KS == 1 && GROUP > 32 && !ZEROS ? 32 : 16;
    __shared__ __attribute__((aligned(16))) uint8_t xs[kStreamX];
    __shared__ __attribute__((aligned(16))) float part[KS > 1 ? kStreamWaves : 1][KS > 1 ? 16 : 1][36];
    const Expander expand;
    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const int i16 = lane & 15, g = lane >> 4, ks = wave % KS;
    const int K = p.w.K, steps = p.steps;
    const int nb = p.swiglu ? (p.C + 15) / 16 : (p.C + 31) / 32, per_tile = (nb + kBlocks - 1) / kBlocks;
    // the later shares first: most are empty and leave at once, the others take longest
    const int share = p.shares - 1 - blockIdx.x / (p.v.max_tiles * per_tile), tile = blockIdx.x % (p.v.max_tiles * per_tile) / per_tile;
    const int cb = blockIdx.x % per_tile * kBlocks + wave / KS;
    int e = 0, p0 = tile * kGroupTile, rows = p.v.rows - p0;
    if (p.v.offsets) {
        // all at once: behind the last tile they are not used
        const int n_tiles = scalar_load(&p.v.ctrl->n_tiles);
        e = scalar_load(p.v.tile_expert + tile);
        p0 = scalar_load(p.v.tile_row0 + tile);
        if (tile >= n_tiles) return;
        rows = scalar_load(p.v.offsets + e + 1) - p0;
    }
    rows = min(rows, kGroupTile);
    if (share * kUnit >= rows) return;

    const uint8_t *codes[2], *scales[2], *zeros[2];  // of the column tile's first row
    uint32_t code_at[2], scale_at[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        // this lane's weight row: past the end the last one, which is not stored
        const int last = p.swiglu ? (q + 1) * p.C - 1 : p.C - 1;
        const int n0 = min(p.swiglu ? 16 * cb + q * p.C : 32 * cb + 16 * q, last), n = min(n0 + i16, last);
        const int64_t at = ((int64_t)e * p.tiles + (n0 >> 4)) * steps;
        const uint32_t next = (n >> 4) - (n0 >> 4), in = n & 15;  // the row may lie in the next packed tile
        codes[q] = uniform(reinterpret_cast<const uint8_t *>(p.w.codes) + at * 2048);
        code_at[q] = next * steps * 2048 + (16 * g + in) * 16;
        scales[q] = uniform(reinterpret_cast<const uint8_t *>(p.w.scales) + at * 32 * kGroups);
        zeros[q] = ZEROS ? uniform(p.w.zeros + at * 16 * kGroups) : nullptr;
        scale_at[q] = (next * steps * 16 + in) * (2 * kGroups);
    }

    typedef Step<GROUP, ZEROS> Weights[2];
    auto load = [&](int s, Weights &w) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            w[q].load(codes[q] + (int64_t)s * 2048, code_at[q], scales[q] + (int64_t)s * (32 * kGroups),
                      ZEROS ? zeros[q] + (int64_t)s * (16 * kGroups) : nullptr, scale_at[q]);
    };

    // MT pieces of 16 rows from m0 on
    auto turn = [&](int m0, auto mt_c) __attribute__((always_inline)) {
        constexpr int MT = decltype(mt_c)::value;
        const int have = min(rows - m0, 16 * MT);
        const int chunk = min(steps, (kStreamX / have - 16) / 512), pitch = chunk * 512 + 16;  // steps in LDS, bytes of a row
        // steps of this wave in the chunk that begins at c
        auto first = [&](int c) __attribute__((always_inline)) { return c + ks * min(chunk, steps - c) / KS; };
        auto behind = [&](int c) __attribute__((always_inline)) { return c + (ks + 1) * min(chunk, steps - c) / KS; };
        Weights next;
        bool loaded = first(0) < behind(0);
        if (loaded) load(first(0), next);
        f4 acc[MT][2] = {};
        uint32_t row[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) row[m] = min(16 * m + i16, have - 1) * pitch + 16 * g;
        for (int c = 0; c < steps; c += chunk) {
            if (c > 0 || m0 > share * kUnit) __syncthreads();
            {
                const int k0 = c * 256, pieces = min(chunk, steps - c) * 32;  // of 16 bytes; past the end the last ones
                for (int r = wave; r < have; r += kStreamWaves) {
                    const int pos = p0 + m0 + r;
                    const int64_t src = p.by_token ? token_of(p.v.sorted_slot[pos], p) : pos;
                    for (int i = lane; i < pieces; i += 64)
                        *reinterpret_cast<u32x4 *>(xs + r * pitch + i * 16) =
                            *reinterpret_cast<const u32x4 *>(p.x + src * K + min(k0 + 8 * i, K - 8));
                }
            }
            __syncthreads();
            const int c2 = c + chunk, s_end = behind(c);
            const bool more = c2 < steps && first(c2) < behind(c2);
            if (!loaded && first(c) < s_end) load(first(c), next);
            loaded = more && first(c) < s_end;
            for (int s = first(c); s < s_end; ++s) {
                const Step<GROUP, ZEROS> w[2] = {next[0], next[1]};
                load(s + 1 < s_end ? s + 1 : more ? first(c2) : s, next);
                const uint8_t *at = xs + (s - c) * 512;
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr) {
                    f4 d[MT][2] = {};
                    uint32_t off[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q)  // minus 16 minus the zero point, twice: its lower byte as it is stored, 0xC1
                        off[q] = ZEROS ? __builtin_amdgcn_perm(0xC1C1C1C1u, w[q].z[gr / 4], 0x04000400u | (gr & 3) * 0x00010001u) : 0xC1C0C1C0u;
#pragma unroll
                    for (int i = gr * (GROUP / 32); i < (gr + 1) * (GROUP / 32); ++i) {
                        bf8 w_op[2];
#pragma unroll
                        for (int q = 0; q < 2; ++q) w_op[q] = expand(w[q].c[i >> 2][i & 3]);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const bf8 xo = __builtin_bit_cast(bf8, *reinterpret_cast<const u32x4 *>(at + row[m] + 64 * i));
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                d[m][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo, w_op[q], d[m][q], 0, 0, 0);
                                d[m][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    xo, __builtin_bit_cast(bf8, (u32x4){off[q], off[q], off[q], off[q]}), d[m][q], 0, 0, 0);
                            }
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float f = scale_value<HALF>(w[q].s[gr / 2], gr & 1);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int v = 0; v < 4; ++v) acc[m][q][v] = fmaf(d[m][q][v], f, acc[m][q][v]);
                    }
                    if constexpr (MT > 1) __builtin_amdgcn_sched_barrier(0);  // one group's operands at a time: registers
                }
            }
        }
        // accumulator v of (m, q): row 16 m + 4 g + v, column 16 q + i16
        if constexpr (KS > 1) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int v = 0; v < 4; ++v) part[wave][4 * g + v][16 * q + i16] = acc[0][q][v];
            __syncthreads();
            // a block's waves take the rows 4 g + v of its sums in turn: a wave's lanes are 16 columns of four rows
            if (ks >= 4) return;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float y = part[wave - ks][4 * g + v][16 * q + i16];
#pragma unroll
                    for (int k = 1; k < KS; ++k) y += part[wave - ks + k][4 * g + v][16 * q + i16];
                    acc[0][q][v] = y;
                }
        }
        if (cb >= nb) return;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int r = 16 * m + 4 * g + v;
                if (r >= have || (KS > 1 && ks != v)) continue;
                const int64_t out = (int64_t)(p0 + m0 + r) * p.C;
                auto store = [&](int c, float y) __attribute__((always_inline)) {
                    if (c >= p.C) return;
                    if (p.out_dtype == MOE_DT_BF16) static_cast<uint16_t *>(p.out)[out + c] = __builtin_bit_cast(uint16_t, (__bf16)y);
                    else static_cast<float *>(p.out)[out + c] = y;
                };
                if (p.swiglu) {
                    store(16 * cb + i16, swiglu(acc[m][0][v], acc[m][1][v]));
                } else {
                    store(32 * cb + i16, acc[m][0][v]);
                    store(32 * cb + 16 + i16, acc[m][1][v]);
                }
            }
    };
    using std::integral_constant;
    for (int m0 = share * kUnit; m0 < rows; m0 += p.shares * kUnit) {
        if (kUnit > 16 && rows - m0 > 16) turn(m0, integral_constant<int, kUnit / 16>{});
        else turn(m0, integral_constant<int, 1>{});
    }
}

// 17 to kWideRows rows of the one weight there is (no groups, so x's rows are in order): a workgroup takes two column tiles, its
// waves a part of the steps each, and their partial sums meet in LDS in the waves' order. Turns of up to 64 rows, each of which
// reads the weights.
constexpr int kWideWaves = 8, kWidePieces = 4;  // of 16 rows in a turn
template <int GROUP, bool HALF, bool ZEROS>
__global__ void __launch_bounds__(64 * kWideWaves, 2) wide_stream_kernel(const W4GemmArgs p) {
    constexpr int kGroups = kW4Step / GROUP;      // per step
    __shared__ __attribute__((aligned(16))) float part[kWideWaves][16 * kWidePieces][36];
    const Expander expand;
    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int N = p.w.N, K = p.w.K;
    const int nb = p.swiglu ? (p.C + 15) / 16 : (p.C + 31) / 32;
    const int cb = blockIdx.x, rows = p.v.rows;
    const uint8_t *codes[2], *scales[2], *zeros[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        // this lane's weight row: past the end the last one, which is not stored
        const int n = p.swiglu ? min(16 * cb + i16, p.C - 1) + q * p.C : min(32 * cb + 16 * q + i16, N - 1);
        const int64_t at = (int64_t)(n >> 4) * p.steps, in = n & 15;
        codes[q] = reinterpret_cast<const uint8_t *>(p.w.codes) + at * 2048 + (16 * g + in) * 16;
        scales[q] = reinterpret_cast<const uint8_t *>(p.w.scales) + (at * 16 + in) * (2 * kGroups);
        zeros[q] = ZEROS ? p.w.zeros + (at * 16 + in) * kGroups : nullptr;
    }
    const int s0 = wave * p.steps / kWideWaves, s1 = (wave + 1) * p.steps / kWideWaves;

    typedef Step<GROUP, ZEROS> Weights[2];
    auto load = [&](int s, Weights &w) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            w[q].load(codes[q] + (int64_t)s * 2048, 0, scales[q] + (int64_t)s * (32 * kGroups),
                      ZEROS ? zeros[q] + (int64_t)s * (16 * kGroups) : nullptr, 0);
    };

    Weights first;
    if (s0 < s1) load(s0, first);

    // MT pieces of 16 rows from m0 on
    auto turn = [&](int m0, auto mt_c) __attribute__((always_inline)) {
        constexpr int MT = decltype(mt_c)::value;
        constexpr int kRuns = MT > 2 ? 4 : 8;  // of 32 columns whose rows are loaded together
        const uint16_t *x[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = p.x + (int64_t)min(m0 + 16 * m + i16, rows - 1) * K + 8 * g;
        f4 acc[MT][2] = {};
        Weights next = {first[0], first[1]};
        if (m0 > 0 && s0 < s1) load(s0, next);
        for (int s = s0; s < s1; ++s) {
            const Step<GROUP, ZEROS> w[2] = {next[0], next[1]};
#pragma unroll
            for (int b = 0; b < 8 / kRuns; ++b) {
                u32x4 xv[kRuns][MT];
#pragma unroll
                for (int i = 0; i < kRuns; ++i) {
                    const int k = min(256 * s + 32 * (kRuns * b + i), K - 32);
#pragma unroll
                    for (int m = 0; m < MT; ++m) xv[i][m] = *reinterpret_cast<const u32x4 *>(x[m] + k);
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
                        for (int q = 0; q < 2; ++q) wv[q] = expand(w[q].c[i >> 2][i & 3]);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const bf8 xo = __builtin_bit_cast(bf8, xv[i % kRuns][m]);
                            sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo, ones(), sum[m], 0, 0, 0);
#pragma unroll
                            for (int q = 0; q < 2; ++q) d[m][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo, wv[q], d[m][q], 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float f = scale_value<HALF>(w[q].s[gr / 2], gr & 1);
                        const float off = ZEROS ? 0.125f * (float)((w[q].z[gr / 4] >> (8 * (gr & 3))) & 255u) : 24.0f;
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int v = 0; v < 4; ++v) acc[m][q][v] = fmaf(fmaf(-off, sum[m][v], d[m][q][v]), f, acc[m][q][v]);
                    }
                    if ((gr + 1) * GROUP % 128 == 0) __builtin_amdgcn_sched_barrier(0);  // else more is alive at once than registers hold
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
        for (int r = t >> 4; r < min(16 * MT, rows - m0); r += 4 * kWideWaves) {
            float y[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int c = p.swiglu ? 16 * q + (t & 15) : 2 * (t & 15) + q;
                y[q] = part[0][r][c];
#pragma unroll
                for (int k = 1; k < kWideWaves; ++k) y[q] += part[k][r][c];
            }
            const int64_t row = (int64_t)(m0 + r) * p.C;
            if (p.swiglu) {
                const int c = 16 * cb + (t & 15);
                const float v = swiglu(y[0], y[1]);
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
    if (rows > m0) turn(m0, integral_constant<int, 2>{});
}

}  // namespace

// Kernels by the rows of a group (for an even routing, or of the one group). One group, 5120 x 4096, groups of 128, us of this
// kernel, the wide one and the tiles: 16 rows 10.0, 11.6, 24.8; 32 rows 17.0, 13.9, 25.9; 128 rows 58, 38, 46; 192 rows 90, 55, 47.
// 4096 x 2560, groups of 32 and zero points: 16 rows 8.2, 10.6, 24.3; 192 rows 66, 44, 54; 256 rows 78, 53, 54. Evenly routed
// over 96 experts, this one and the tiles: 16 rows each 241, 300 and 183, 290; 21 rows 256, 302 and 219, 294; 32 rows 345, 322 and
// 304, 342; 42 rows 474, 352 and 373, 378; unevenly (the largest group of five to thirty times the mean) 10 rows 220, 273 and 167,
// 270; 21 rows 322, 348 and 187, 294; 42 rows 444, 424 and 311, 360.
constexpr int kStreamMean = 24, kStreamRows = 16, kWideRows = 160;
// Waves that share a block of two column tiles, by the blocks of a call: eight up to kBlocksOfEight, four up to kBlocksOfFour,
// then each its own. us of eight, four and one: one row, K 4096, 256 blocks 8.2, 8.8, 18.3; 384 blocks 10.8, 9.5, 18.8; 2048
// blocks 42, 32, 34. One token of eight experts, K 2560, 256 blocks 7.1, 7.8, 13.4; 384 blocks 9.0, 8.4, 13.6; 1024 blocks 16.9,
// 12.9, 16.1; 1536 blocks 24.1, 20.7, 17.5. 48 tokens on 48 experts, K 2048, 392 blocks 9.0, 8.7, 13.3; 784 blocks 14.9, 12.1,
// 13.4; 1176 blocks 19.8, 17.6, 14.6; 6272 blocks 83, 64, 50.
constexpr int kBlocksOfEight = 320, kBlocksOfFour = 1024;

hipError_t launch_w4_gemm(const W4GemmArgs &args, hipStream_t s) {
    W4GemmArgs a = args;
    const int rows = a.v.mean_rows;
    const int64_t nb = a.swiglu ? (a.C + 15) / 16 : (a.C + 31) / 32, blocks = (int64_t)a.v.max_tiles * nb;
    // a grid's threads are 32 bits; the tiles' grid is one workgroup a CU
    if (rows > (a.v.offsets ? kStreamMean : kWideRows) || blocks >= 1 << 22) return launch_w4_tile(a, s);
    // An expert that far more tokens chose than the others takes several turns: four workgroups share them (256 tokens, 161 of
    // them for one expert of 60, 5120 x 4096: 284 -> 186 us; evenly routed, where most of them are empty, 202 -> 208 us).
    a.shares = a.v.offsets && a.v.rows / a.v.top_k > 64 ? 4 : 1;
    by_form(a.w, [&](auto group, auto half, auto zeros) {
        constexpr int kGroup = decltype(group)::value;
        constexpr bool kHalf = decltype(half)::value, kZeros = decltype(zeros)::value;
        auto go = [&](auto kernel, int per_group) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)(a.v.max_tiles * a.shares * ((nb + per_group - 1) / per_group))), dim3(512), 0, s, a);
        };
        if (!a.v.offsets && rows > kStreamRows) go(wide_stream_kernel<kGroup, kHalf, kZeros>, 1);
        else if (blocks > kBlocksOfFour) go(stream_kernel<kGroup, kHalf, kZeros, 1>, 8);
        else if (blocks > kBlocksOfEight) go(stream_kernel<kGroup, kHalf, kZeros, 4>, 2);
        else go(stream_kernel<kGroup, kHalf, kZeros, 8>, 1);
    });
    return hipGetLastError();
}

}  // namespace moe
