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
        const int e = v.tile_expert[tq], o = v.offsets[e];
        t0 = tq - (v.tile_row0[tq] - o) / kBM;
        te = (v.offsets[e + 1] - o + kBM - 1) / kBM;
    }
    const int local = w - nb * t0, g = local / (4 * nb), r = local % (4 * nb);
    const int gs = min(4, te - 4 * g);
    tile = t0 + 4 * g + r % gs;
    cb = r / gs;
    return true;
}

template <bool TRANS>
__global__ void __launch_bounds__(kThreads) tile_kernel(const BlockGemmArgs p) {
    __shared__ __attribute__((aligned(16))) uint8_t xb0[kOperand];
    __shared__ __attribute__((aligned(16))) uint8_t xb1[kOperand];
    __shared__ __attribute__((aligned(16))) uint8_t wb0[kOperand];
    __shared__ __attribute__((aligned(16))) uint8_t wb1[kOperand];
    __shared__ __attribute__((aligned(16))) float sc[kSeg * kBM];

    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wm = wave >> 2, wn = wave & 3;
    const int i16 = lane & 15, g = lane >> 4;
    const int R = p.R, C = p.C, n = R / 128;
    const int nb = (C + kBN - 1) / kBN;
    const int n_tiles = p.v.offsets ? p.v.ctrl->n_tiles : p.v.max_tiles;
    const int per_xcd = (n_tiles * nb + 7) / 8;
    const int step = (gridDim.x + 7) / 8;

    for (int it = blockIdx.x >> 3; it < per_xcd; it += step) {
        int tile, cb;
        if (!work_item(p.v, n_tiles, (blockIdx.x & 7) * per_xcd + it, nb, tile, cb)) break;
        int e = 0, p0 = tile * kBM, rows = p.v.rows - p0;
        if (p.v.offsets) {
            e = p.v.tile_expert[tile];
            p0 = p.v.tile_row0[tile];
            rows = p.v.offsets[e + 1] - p0;
        }
        rows = min(rows, kBM);
        const int n_sub = (rows + 15) / 16, msa = (n_sub - wm + 1) / 2;
        const int c0 = cb * kBN;
        auto src_row = [&](int r) -> int64_t {
            const int pos = p0 + min(r, rows - 1);
            return p.by_token ? p.v.sorted_slot[pos] / p.v.top_k : pos;
        };

        // ---- sources of this lane's copies
        const uint8_t *xs[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            xs[j] = p.x_codes + src_row(32 * wave + 8 * j + (lane >> 3)) * R + (((lane & 7) ^ (lane >> 3)) * 16);
        const uint8_t *ws = p.w_codes + e * p.w_expert_bytes;
        if (TRANS) {
            int kc = c0 / 64 + 2 * (wave & 1);
            if (kc * 64 >= C) kc = c0 / 64;  // half a column block: its first half again, unused
            ws += ((int64_t)(wave >> 1) * (C / 64) + kc) * 2048 + lane * 16;
        } else {
            int rb = c0 / 32 + wave;
            if (rb * 32 >= C) rb -= 4;
            ws += (int64_t)rb * (R / 64) * 2048 + (lane >> 5) * 512 + swizzled_row(lane & 31, wave) * 16;
        }
        const int64_t w_step = TRANS ? (int64_t)C * 128 : 4096;
        auto copy_x = [&](uint8_t *dst, int s) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (32 * wave + 8 * j < 16 * n_sub) copy_to_lds(xs[j] + s * 128, dst + wave * 4096 + j * 1024);
        };
        auto copy_w = [&](uint8_t *dst, int s) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) copy_to_lds(ws + s * w_step + j * 1024, dst + wave * 4096 + j * 1024);
        };

        // ---- scales of blocks seg .. seg + 31: the rows' to LDS, the weights' one per lane
        const int col_block = min(c0 / 128 + (wn >> 1), C / 128 - 1);
        const float *sw = p.w_scales + (int64_t)e * p.w_expert_scales + (TRANS ? col_block : col_block * p.w_kb);
        const float *sx = p.x_scales + src_row(t >> 1) * n;
        float swv = 0.0f;
        auto load_scales = [&](int seg) {
            const int b = min(seg + (lane & 31), n - 1);
            swv = sw[TRANS ? (int64_t)b * p.w_kb : b];
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = sx[min(seg + 16 * (t & 1) + j, n - 1)];
#pragma unroll
            for (int j = 0; j < 16; ++j) sc[(16 * (t & 1) + j) * kBM + (t >> 1)] = v[j];
        };

        f4 acc[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s) acc[i][s] = (f4){0.0f, 0.0f, 0.0f, 0.0f};

        // the wave's operand for its columns, read s of 4
        auto w_operand = [&](const uint8_t *w, int s) __attribute__((always_inline)) -> v8i {
            if constexpr (TRANS) {
                // columns 16 s + i16 of tile column wn; block rows 16 g .. and 64 + 16 g ..
                const uint8_t *q = w + (g >> 1) * 8192 + wn * 2048 + s * 512 + (g & 1) * 256 + i16 * 8;
                auto tr = [&](int at) {
                    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) v2i *)(q + at));
                };
                const v2i a = tr(0), b = tr(128), c = tr(2 * 8192), d = tr(2 * 8192 + 128);
                return (v8i){a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
            } else {
                const int rt = 2 * wn + (i16 >> 3);  // 32-row tile
                const int r = 16 * ((i16 >> 2) & 1) + 4 * s + (i16 & 3);
                const uint8_t *q = w + rt * 4096 + g * 512 + swizzled_row(r, rt) * 16;
                return operand(*reinterpret_cast<const u32x4 *>(q), *reinterpret_cast<const u32x4 *>(q + 2048));
            }
        };
        auto x_operand = [&](const uint8_t *x, int i) __attribute__((always_inline)) -> v8i {
            const int r = 16 * (2 * i + wm) + i16;
            const uint8_t *q = x + r * 128;
            return operand(*reinterpret_cast<const u32x4 *>(q + ((g ^ (r & 7)) * 16)),
                           *reinterpret_cast<const u32x4 *>(q + (((4 + g) ^ (r & 7)) * 16)));
        };

        // block s from buffers x, w
        auto block_step = [&](const uint8_t *x, uint8_t *x_next, uint8_t *w, int s) __attribute__((always_inline)) {
            // this block's copies are all but the weights of block s + 1
            if (s + 1 < n) wait_copies<4>();
            else wait_copies<0>();
            lds_barrier();
            if ((s & (kSeg - 1)) == 0 && s > 0) {
                load_scales(s);
                lds_barrier();
            }
            if (s + 1 < n) copy_x(x_next, s + 1);
            v8i wf[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) wf[q] = w_operand(w, q);
            const float fw = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(swv), s & (kSeg - 1)));
            const float *fs = sc + (s & (kSeg - 1)) * kBM;
            v8i xf = x_operand(x, 0);
            float f = fs[16 * wm + i16] * fw;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i < msa) {
                    const v8i xi = xf;
                    const float fi = f;
                    if (i + 1 < 8) {
                        xf = x_operand(x, i + 1);
                        f = fs[16 * (2 * (i + 1) + wm) + i16] * fw;
                    }
                    f4 d[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) d[q] = block_dot(wf[q], xi);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[i][q][v] = fmaf(d[q][v], fi, acc[i][q][v]);
                }
                if (i == 0) {  // every wave holds its columns' codes: refill their buffer
                    lds_barrier();
                    if (s + 2 < n) copy_w(w, s + 2);
                }
            }
        };

        lds_barrier();  // the previous item's reads
        load_scales(0);
        copy_x(xb0, 0);
        copy_w(wb0, 0);
        if (n > 1) copy_w(wb1, 1);
        for (int s = 0; s < n; s += 2) {
            block_step(xb0, xb1, wb0, s);
            if (s + 1 < n) block_step(xb1, xb0, wb1, s + 1);
        }

        // ---- outputs
        if (c0 + 64 * wn < C) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int m = 16 * (2 * i + wm) + i16;
                if (i < msa && m < rows) {
                    uint16_t *o = p.out + (int64_t)(p0 + m) * C + c0 + 64 * wn;
                    if (TRANS) {  // read s holds columns 16 s + 4 g ..
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            *reinterpret_cast<uint2 *>(o + 16 * s + 4 * g) =
                                make_uint2(bf16_pair(acc[i][s][0], acc[i][s][1]), bf16_pair(acc[i][s][2], acc[i][s][3]));
                    } else {  // read s holds columns 16 g + 4 s ..
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            *reinterpret_cast<uint4 *>(o + 16 * g + 8 * h) =
                                make_uint4(bf16_pair(acc[i][2 * h][0], acc[i][2 * h][1]),
                                           bf16_pair(acc[i][2 * h][2], acc[i][2 * h][3]),
                                           bf16_pair(acc[i][2 * h + 1][0], acc[i][2 * h + 1][1]),
                                           bf16_pair(acc[i][2 * h + 1][2], acc[i][2 * h + 1][3]));
                    }
                }
            }
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
