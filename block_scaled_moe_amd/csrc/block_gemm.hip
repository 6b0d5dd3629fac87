// block_gemm.hip - grouped product of E4M3 rows with E4M3 expert weights, a scale per 1 x 128
// block of the rows and per 128 x 128 block of the weights (include/moe_ops.h, moe_block_gemm),
// and the same with the weights transposed.
//
//   out[p][c] = sum over blocks b of (sx[p][b] sw[b, c / 128]) * sum over the block of cx * cw
//
// tile_kernel: 256 rows x 256 output columns per work item, 8 waves as 2 (rows) x 4 (columns),
// a wave 16 MFMA tiles of 16 rows apart by two (the tile's 16-row pieces alternate between the
// two row waves, so a partial tile splits evenly) x 64 columns. The weights are the MFMA's A
// operand, so a lane's accumulators are consecutive outputs of one row, its block factor is
// one value per piece, and the factor costs one multiply per 16 results.
//  - Per block of 128 the item needs 32 KiB of row codes and 32 KiB of weight codes. Both go
//    straight from memory into LDS, two buffers each. Row codes are copied one block ahead;
//    weight codes, which come from HBM, two ahead: every wave reads its 64 columns' codes of
//    the block into registers before its second piece of rows, and the buffer is refilled
//    from there on (the barrier in the middle of a step).
//  - The row scales of 32 blocks (4096 values of the reduction) are kept in LDS as
//    [block][row], loaded once per item (again every 32 blocks for longer reductions).
//  - One workgroup per CU (160 KiB of LDS) walks its work items; each XCD takes a contiguous
//    range of them, expert by expert with the column blocks outside, so an expert's rows and
//    weights meet in one L2.
// Transposed, the reduction runs along the weights' rows: the same bytes are copied, and the
// operand is read with the transposing LDS read (8 rows x 16 columns per 16 lanes).
//
// stream_kernel: few rows per group (decode). Bound by the weights' bytes from HBM: a
// workgroup takes 32 output columns of one expert, its four waves a quarter of the blocks each,
// weights go straight into registers, and the four partial sums meet in LDS in a fixed order.
#include "block_mma.h"
#include "ops_internal.h"

#include <type_traits>

namespace moe {
namespace {

using namespace block;

constexpr int kThreads = 512, kBM = kGroupTile, kBN = 256;
constexpr int kOperand = 256 * 128;  // LDS bytes of one operand of one block
constexpr int kSeg = 32;             // blocks whose row scales are in LDS
constexpr int kMaxGrid = 256;        // workgroups: one per CU
static_assert(4 * kOperand + kSeg * kBM * 4 <= 160 * 1024, "LDS");

// Work item w: its tile of rows and block of columns. Items of one expert are consecutive,
// its tiles in groups of up to four with the column blocks outside.
__device__ __forceinline__ bool work_item(const GroupView &v, int n_tiles, int w, int nb, int &tile, int &cb) {
    if (w >= n_tiles * nb) return false;
    const int tq = w / nb;
    int t0 = 0, te = n_tiles;
    if (v.offsets) {
        const int e = scalar_load(v.tile_expert + tq), o = scalar_load(v.offsets + e);
        t0 = tq - (scalar_load(v.tile_row0 + tq) - o) / kBM;
        te = (scalar_load(v.offsets + e + 1) - o + kBM - 1) / kBM;
    }
    const int local = w - nb * t0, g = local / (4 * nb), r = local % (4 * nb);
    const int gs = min(4, te - 4 * g);
    tile = t0 + 4 * g + r % gs;
    cb = r / gs;
    return true;
}

template <bool TRANS>
__global__ void __launch_bounds__(kThreads) tile_kernel(const BlockGemmArgs p) {
    // row codes (two buffers), weight codes (two buffers), row scales [block][row]
    __shared__ __attribute__((aligned(16))) uint8_t xb[2 * kOperand];
    __shared__ __attribute__((aligned(16))) uint8_t wb[2 * kOperand];
    __shared__ __attribute__((aligned(16))) float sc[kSeg * kBM];

    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int i16 = lane & 15, g = lane >> 4;
    const int R = p.R, C = p.C, n = R / 128;
    const int nb = (C + kBN - 1) / kBN;
    const int n_tiles = p.v.offsets ? p.v.ctrl->n_tiles : p.v.max_tiles;
    const int per_xcd = (n_tiles * nb + 7) / 8;
    const int step = (gridDim.x + 7) / 8;
    const uint32_t x_lds = lds_address(xb) + wave * 4096, w_lds = lds_address(wb) + wave * 4096;

    for (int it = blockIdx.x >> 3; it < per_xcd; it += step) {
        int tile, cb;
        if (!work_item(p.v, n_tiles, (blockIdx.x & 7) * per_xcd + it, nb, tile, cb)) break;
        int e = 0, p0 = tile * kBM, rows = p.v.rows - p0;
        if (p.v.offsets) {
            e = scalar_load(p.v.tile_expert + tile);
            p0 = scalar_load(p.v.tile_row0 + tile);
            rows = scalar_load(p.v.offsets + e + 1) - p0;
        }
        rows = uniform(min(rows, kBM));
        const int n_sub = (rows + 15) / 16;
        const int c0 = cb * kBN;
        auto src_row = [&](int r) -> int64_t {
            const int pos = p0 + min(r, rows - 1);
            return p.by_token ? p.v.sorted_slot[pos] / p.v.top_k : pos;
        };

        // ---- sources of this lane's copies: four pieces of rows; the wave's weights and the
        // lane's offset in them
        uint32_t x_lane[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x_lane[j] = (uint32_t)src_row(32 * wave + 8 * j + (lane >> 3)) * 128 + (((lane & 7) ^ (lane >> 3)) * 16);
        const int64_t x_step = (int64_t)p.x_rows * 128;
        const int x_copies = min(4, max(0, 2 * n_sub - 4 * wave));  // of 8 rows each that hold rows
        const uint8_t *ws = p.w_codes + e * p.w_expert_bytes;
        uint32_t w_lane;
        if (TRANS) {
            int kc = c0 / 64 + 2 * (wave & 1);
            if (kc * 64 >= C) kc = c0 / 64;  // half a column block: its first half again, unused
            ws += ((int64_t)(wave >> 1) * (C / 64) + kc) * 2048;
            w_lane = lane * 16;
        } else {
            int rb = c0 / 32 + wave;
            if (rb * 32 >= C) rb -= 4;
            ws += (int64_t)rb * (R / 64) * 2048;
            w_lane = (lane >> 5) * 512 + swizzled_row(lane & 31) * 16;
        }
        ws = uniform(ws);
        const int64_t w_step = TRANS ? (int64_t)C * 128 : 4096;
        auto copy_x = [&](int s) __attribute__((always_inline)) {
            const uint32_t dst = x_lds + (s & 1) * kOperand;
            const uint8_t *src = p.x_codes + s * x_step;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < x_copies) copy_to_lds(src, x_lane[j], dst + j * 1024);
        };
        auto copy_w = [&](int s) __attribute__((always_inline)) {
            const uint32_t dst = w_lds + (s & 1) * kOperand;
            const uint8_t *src = ws + s * w_step;
#pragma unroll
            for (int j = 0; j < 4; ++j) copy_to_lds(src + j * 1024, w_lane, dst + j * 1024);
        };

        const int col_block = min(c0 / 128 + (wn >> 1), C / 128 - 1);
        const float *sw = p.w_scales + (int64_t)e * p.w_expert_scales + (TRANS ? col_block : col_block * p.w_kb);

        auto run = [&](auto msa_c) __attribute__((always_inline)) {
            constexpr int MSA = decltype(msa_c)::value;  // this wave's pieces of 16 rows
            f4 acc[MSA > 0 ? MSA : 1][4];
#pragma unroll
            for (int i = 0; i < MSA; ++i)
#pragma unroll
                for (int s = 0; s < 4; ++s) acc[i][s] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
            // Block sums of two pieces of rows: a piece's are added to its accumulators behind
            // the MFMAs of the next one, the last piece's behind those of the next block's first
            // (where the two do not fall on the same registers)
            constexpr bool kCarry = MSA % 2 == 0;
            f4 d[2][4];
            float fd = 0.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q) d[0][q] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
            auto add = [&](int i, int b, int q, float f) __attribute__((always_inline)) {
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][q][v] = fmaf(d[b][q][v], f, acc[i][q][v]);
                pin(acc[i][q]);
            };

            copy_x(0);
            copy_w(0);
            if (n > 1) copy_w(1);
            for (int seg = 0; seg < n; seg += kSeg) {
                // ---- scales of blocks seg ..: the rows' to LDS, the weights' one per lane
                if (seg > 0) lds_barrier();  // the last segment's reads
                const int bw = min(seg + (lane & 31), n - 1);
                const float swv = sw[TRANS ? (int64_t)bw * p.w_kb : bw];
                {
                    const float *sx = p.x_scales + src_row(t >> 1) * n;
                    const int b0 = 16 * (t & 1);
                    f4 v[4];
                    if (n % 4 == 0) {
#pragma unroll
                        for (int h = 0; h < 4; ++h) v[h] = *reinterpret_cast<const f4 *>(sx + min(seg + b0 + 4 * h, n - 4));
                    } else {
#pragma unroll
                        for (int h = 0; h < 16; ++h) v[h >> 2][h & 3] = sx[min(seg + b0 + h, n - 1)];
                    }
#pragma unroll
                    for (int h = 0; h < 16; ++h) sc[(b0 + h) * kBM + (t >> 1)] = v[h >> 2][h & 3];
                }
                const int end = min(seg + kSeg, n);
#pragma clang loop unroll(disable)
                for (int s = seg; s < end; ++s) {
                    // this block's copies are all but the weights of block s + 1
                    if (s + 1 < n) wait_copies<4>();
                    else wait_copies<0>();
                    lds_barrier();
                    if (s + 1 < n) copy_x(s + 1);
                    if constexpr (MSA > 0) {
                        const uint8_t *x = xb + (s & 1) * kOperand, *w = wb + (s & 1) * kOperand;
                        const float *fs = sc + (s - seg) * kBM + 16 * wm + i16;
                        const float fw = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(swv), s - seg));
                        auto x_operand = [&](int i) __attribute__((always_inline)) -> v8i {
                            const uint8_t *q = x + (16 * wm + i16) * 128 + i * 4096;
                            return operand(*reinterpret_cast<const u32x4 *>(q + ((g ^ (i16 & 7)) * 16)),
                                           *reinterpret_cast<const u32x4 *>(q + (((4 + g) ^ (i16 & 7)) * 16)));
                        };
                        v8i wf[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if constexpr (TRANS) {
                                // columns 16 q + i16 of tile column wn; block rows 16 g .. and 64 + 16 g ..
                                const uint8_t *a = w + (g >> 1) * 8192 + wn * 2048 + q * 512 + (g & 1) * 256 + i16 * 8;
                                auto tr = [&](int at) {
                                    return __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                                        (__attribute__((address_space(3))) v2i *)(a + at));
                                };
                                const v2i a0 = tr(0), a1 = tr(128), a2 = tr(2 * 8192), a3 = tr(2 * 8192 + 128);
                                wf[q] = (v8i){a0.x, a0.y, a1.x, a1.y, a2.x, a2.y, a3.x, a3.y};
                            } else {
                                const uint8_t *a = w + (2 * wn + (q >> 1)) * 4096 + g * 512 + swizzled_row(a_row(i16, q)) * 16;
                                wf[q] = operand(*reinterpret_cast<const u32x4 *>(a),
                                                *reinterpret_cast<const u32x4 *>(a + 2048));
                            }
                        }
                        v8i xf = x_operand(0);
                        float f = fs[0] * fw;
#pragma unroll
                        for (int i = 0; i < MSA; ++i) {
                            const v8i xi = xf;
                            const float fi = f;
                            if (i + 1 < MSA) {
                                xf = x_operand(i + 1);
                                f = fs[32 * (i + 1)] * fw;
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                d[(MSA - 1 - i) & 1][q] = block_dot(wf[q], xi);
                                pin(d[(MSA - 1 - i) & 1][q]);
                                if (i > 0 || kCarry) add(i > 0 ? i - 1 : MSA - 1, (MSA - i) & 1, q, fd);
                                __builtin_amdgcn_sched_barrier(0);
                            }
                            fd = fi;
                            if (i == 0) {  // every wave holds its columns' codes: refill their buffer
                                lds_barrier();
                                if (s + 2 < n) copy_w(s + 2);
                            }
                        }
                        if (!kCarry) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) add(MSA - 1, 0, q, fd);
                        }
                    } else {
                        lds_barrier();
                        if (s + 2 < n) copy_w(s + 2);
                    }
                }
            }

            if constexpr (MSA > 0 && kCarry) {
#pragma unroll
                for (int q = 0; q < 4; ++q) add(MSA - 1, 0, q, fd);
            }

            // ---- outputs
            if (c0 + 64 * wn < C) {
#pragma unroll
                for (int i = 0; i < MSA; ++i) {
                    const int m = 16 * (2 * i + wm) + i16;
                    if (m < rows) {
                        uint16_t *o = p.out + (int64_t)(p0 + m) * C + c0 + 64 * wn;
                        if (TRANS) {  // read s holds columns 16 s + 4 g ..
#pragma unroll
                            for (int s = 0; s < 4; ++s)
                                *reinterpret_cast<uint2 *>(o + 16 * s + 4 * g) = make_uint2(
                                    bf16_pair(acc[i][s][0], acc[i][s][1]), bf16_pair(acc[i][s][2], acc[i][s][3]));
                        } else {  // reads 2 h, 2 h + 1 hold columns 32 h + 8 g ..
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                *reinterpret_cast<uint4 *>(o + 32 * h + 8 * g) =
                                    make_uint4(bf16_pair(acc[i][2 * h][0], acc[i][2 * h][1]),
                                               bf16_pair(acc[i][2 * h][2], acc[i][2 * h][3]),
                                               bf16_pair(acc[i][2 * h + 1][0], acc[i][2 * h + 1][1]),
                                               bf16_pair(acc[i][2 * h + 1][2], acc[i][2 * h + 1][3]));
                        }
                    }
                }
            }
        };
        lds_barrier();  // the previous item's reads
        // pieces 2 i + wm < n_sub; every wave runs the same copies and barriers
        switch ((n_sub - wm + 1) / 2) {
            case 0: run(std::integral_constant<int, 0>{}); break;
            case 1: run(std::integral_constant<int, 1>{}); break;
            case 2: run(std::integral_constant<int, 2>{}); break;
            case 3: run(std::integral_constant<int, 3>{}); break;
            case 4: run(std::integral_constant<int, 4>{}); break;
            case 5: run(std::integral_constant<int, 5>{}); break;
            case 6: run(std::integral_constant<int, 6>{}); break;
            case 7: run(std::integral_constant<int, 7>{}); break;
            default: run(std::integral_constant<int, 8>{}); break;
        }
    }
}

}  // namespace

hipError_t launch_block_gemm(const BlockGemmArgs &a, bool transposed, hipStream_t s) {
    const int64_t items = (int64_t)a.v.max_tiles * ((a.C + kBN - 1) / kBN);
    if (items > INT32_MAX - 8) return hipErrorInvalidValue;
    const unsigned grid = (unsigned)(items >= kMaxGrid ? kMaxGrid : (items + 7) / 8 * 8);
    if (transposed) hipLaunchKernelGGL(tile_kernel<true>, dim3(grid), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL(tile_kernel<false>, dim3(grid), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
