// block_gemm.hip - grouped product of E4M3 rows with E4M3 expert weights, a scale per 1 x 128
// block of the rows and per 128 x 128 block of the weights (include/moe_ops.h, moe_block_gemm),
// and the same with the weights transposed.
//
//   out[p][c] = sum over blocks b of (sx[p][b] sw[b, c / 128]) * sum over the block of cx * cw
//
// 224 rows x 256 output columns per work item, 8 waves as 2 (rows) x 4 (columns), a wave up to 7
// pieces of 16 rows (the tile's pieces alternate between the two row waves, so that a partial
// tile splits evenly) x 64 columns. The weights are the MFMA's A operand, so a lane's accumulators
// are consecutive outputs of one row, its block factor is one value per piece, and the factor
// costs one multiply per 16 results.
//  - Per block of 128 the item needs 28 KiB of row codes with their scales and 32 KiB of weight
//    codes. All of it goes straight from memory into LDS: rows into two buffers, one block ahead;
//    weights, which come from HBM, into three. A wave reads its weights of block s + 1 into
//    registers while it multiplies block s, so their buffer takes block s + 4 at the next block's
//    start and a copy has two blocks' time to arrive; one barrier a block covers everything.
//  - 224 rows are what 160 KiB of LDS and 256 registers a lane leave beside that.
//  - A block sum is added to its accumulator two MFMAs later, behind the next ones.
//  - One workgroup per CU walks its work items; each XCD takes a contiguous range of them,
//    expert by expert with the column blocks outside, so an expert's rows and weights meet in
//    one L2.
// Transposed, the reduction runs along the weights' rows: the same bytes are copied, and the
// operand is read with the transposing LDS read (8 rows x 16 columns per 16 lanes).
//
// One group of 8191 rows, 5120 x 4096: 176 us (1.95 PFLOP/s), of which the products alone take 130 us, the
// barriers 8, the stores 15, the copies 24. 96 groups of about 170 rows, 5120 x 4096: 467 us (1.47 PFLOP/s,
// 4.8 TB/s of weights, rows and results; a group's last tile is as long in copies as a full one). Transposed
// on 17108 unevenly grouped rows, 4096 x 2560: 278 us.
// stream_kernel below takes over where groups have few rows.
#include "block_mma.h"
#include "ops_internal.h"

#include <type_traits>

namespace moe {
namespace {

using namespace block;

constexpr int kThreads = 512, kBM = kGroupTile, kBN = 256;
constexpr int kX = kBM * 128, kW = kBN * 128;  // LDS bytes of one block's codes
constexpr int kXCopies = kBM / 8;              // copies of 8 rows, dealt to the waves in turn
constexpr int kMaxGrid = 256;                  // workgroups: one per CU
static_assert(2 * kX + 3 * kW + 2 * 16 * kBM + 4 * kBM <= 160 * 1024 && kBM % 32 == 0 && kBM <= 256, "LDS");

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
    __shared__ __attribute__((aligned(16))) uint8_t xb[2 * kX];
    __shared__ __attribute__((aligned(16))) uint8_t wb[3 * kW];
    __shared__ __attribute__((aligned(16))) float sb[2 * 4 * kBM];  // scales of the rows, four blocks: [row][4]
    __shared__ int32_t slots[kBM];                                  // of the next item's rows

    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int i16 = lane & 15, g = lane >> 4;
    const int R = p.R, C = p.C, n = R / 128;
    const int nb = (C + kBN - 1) / kBN;
    const int n_tiles = p.v.offsets ? p.v.ctrl->n_tiles : p.v.max_tiles;
    const int per_xcd = (n_tiles * nb + 7) / 8;
    const int step = (gridDim.x + 7) / 8;
    const uint32_t x_lds = lds_address(xb) + wave * 1024, w_lds = lds_address(wb) + wave * 4096;
    const uint32_t s_lds = lds_address(sb) + (wave & 3) * 1024;

    struct Item {
        int e, p0, rows, c0;
    };
    auto fetch = [&](int it, Item &a) __attribute__((always_inline)) -> bool {
        int tile, cb;
        if (it >= per_xcd || !work_item(p.v, n_tiles, (blockIdx.x & 7) * per_xcd + it, nb, tile, cb)) return false;
        a.e = 0;
        a.p0 = tile * kBM;
        a.rows = p.v.rows - a.p0;
        if (p.v.offsets) {
            a.e = scalar_load(p.v.tile_expert + tile);
            a.p0 = scalar_load(p.v.tile_row0 + tile);
            a.rows = scalar_load(p.v.offsets + a.e + 1) - a.p0;
        }
        a.rows = min(a.rows, kBM);
        a.c0 = cb * kBN;
        return true;
    };
    const uint32_t w_lane = TRANS ? lane * 16 : (lane >> 5) * 512 + swizzled_row(lane & 31) * 16;
    const int64_t w_step = TRANS ? (int64_t)C * 128 : 4096, x_step = (int64_t)p.x_rows * 128;

    // ---- sources of the current item: the wave's weights and their scales; this lane's place in up
    // to four copies of 8 rows (waves 4 to 7 three, and every fourth block four blocks' scales of 64
    // rows)
    const uint8_t *ws;
    const float *sw;
    uint32_t x_lane[4], s_lane;
    auto weight_scale = [&](int s) { return scalar_load(sw + (TRANS ? (int64_t)min(s, n - 1) * p.w_kb : min(s, n - 1))); };
    // the rows' slots (by token) are in `slots` for an item that was announced
    auto sources = [&](const Item &a, bool announced) __attribute__((always_inline)) {
        ws = p.w_codes + a.e * p.w_expert_bytes;
        if (TRANS) {
            int kc = a.c0 / 64 + 2 * (wave & 1);
            if (kc * 64 >= C) kc = a.c0 / 64;  // half a column block: its first half again, unused
            ws += ((int64_t)(wave >> 1) * (C / 64) + kc) * 2048;
        } else {
            int rb = a.c0 / 32 + wave;
            if (rb * 32 >= C) rb -= 4;
            ws += (int64_t)rb * (R / 64) * 2048;
        }
        ws = uniform(ws);
        const int col_block = min(a.c0 / 128 + (wn >> 1), C / 128 - 1);
        sw = uniform(p.w_scales + (int64_t)a.e * p.w_expert_scales + (TRANS ? col_block : col_block * p.w_kb));
        uint32_t row[5];
#pragma unroll
        for (int j = 0; j < 5; ++j) {
            const int r = min(j < 4 ? 8 * (wave + 8 * j) + (lane >> 3) : 64 * (wave & 3) + lane, a.rows - 1);
            row[j] = a.p0 + r;
            if (p.by_token) row[j] = (uint32_t)(announced ? slots[r] : p.v.sorted_slot[a.p0 + r]) / (uint32_t)p.v.top_k;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x_lane[j] = row[j] * 128 + (((lane & 7) ^ (lane >> 3)) * 16);
        s_lane = row[4] * (uint32_t)scale_stride(R) * 4;
    };
    auto announce = [&](const Item &a) __attribute__((always_inline)) {
        const int r = 64 * (wave & 3) + lane;
        if (p.by_token && wave >= 4 && r < kBM)
            copy4_to_lds(reinterpret_cast<const uint8_t *>(p.v.sorted_slot + a.p0), min(r, a.rows - 1) * 4,
                         lds_address(slots) + (wave & 3) * 256);
    };
    auto copy_x = [&](const Item &a, int s) __attribute__((always_inline)) {
        const uint32_t b = (s & 1) * kX;
        const uint8_t *src = p.x_codes + s * x_step;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (wave + 8 * j < min((a.rows + 15) / 16 * 2, kXCopies)) copy_to_lds(src, x_lane[j], x_lds + b + j * 8192);
    };
    // scales of blocks s .. s + 3 (s % 4 == 0)
    auto copy_s = [&](const Item &a, int s) __attribute__((always_inline)) {
        if (wave >= 4 && 64 * (wave - 4) < a.rows && 64 * (wave - 4) + lane < kBM)
            copy_to_lds(reinterpret_cast<const uint8_t *>(p.x_scales + s), s_lane, s_lds + (s & 4) * 4 * kBM);
    };
    auto copy_w = [&](int s, int buffer) __attribute__((always_inline)) {
        const uint32_t dst = w_lds + buffer * kW;
        const uint8_t *src = ws + s * w_step;
#pragma unroll
        for (int j = 0; j < 4; ++j) copy_to_lds(src + j * 1024, w_lane, dst + j * 1024);
    };
    // an item's first copies; wait_first leaves the last of them, and `stores` behind them, in flight
    auto copy_first = [&](const Item &a) __attribute__((always_inline)) {
        copy_s(a, 0);
        copy_x(a, 0);
        if (n > 1) copy_x(a, 1);
        copy_w(0, 0);
        if (n > 1) copy_w(1, 1);
        if (n > 2) copy_w(2, 2);
    };
    auto wait_newer = [&](int newer) __attribute__((always_inline)) {  // rounded down to a multiple of four
        if (newer >= 16) wait_copies<16>();
        else if (newer >= 12) wait_copies<12>();
        else if (newer >= 8) wait_copies<8>();
        else if (newer >= 4) wait_copies<4>();
        else wait_copies<0>();
    };

    int it = blockIdx.x >> 3;
    Item cur, next;
    if (!fetch(it, cur)) return;
    sources(cur, false);
    copy_first(cur);
    int stores = 0;  // of the last item by this wave (or fewer), behind the first copies of this one
    for (;;) {
        it += step;
        const bool more = fetch(it, next);
        const int n_sub = (cur.rows + 15) / 16;

        auto run = [&](auto msa_c) __attribute__((always_inline)) {
            constexpr int MSA = decltype(msa_c)::value;  // this wave's pieces of 16 rows
            constexpr int U = 4 * MSA;                   // MFMAs of a block
            f4 acc[MSA > 0 ? MSA : 1][4], d[4];
#pragma unroll
            for (int i = 0; i < MSA; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][q] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < 4; ++q) d[q] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
            float f_last = 0.0f;
            auto add = [&](int u, float f) __attribute__((always_inline)) {
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[u / 4][u % 4][v] = fmaf(d[u % 4][v], f, acc[u / 4][u % 4][v]);
                pin(acc[u / 4][u % 4]);
            };
            // the wave's operand for its columns, read q of 4, from weight buffer b
            auto w_operand = [&](int b, int q) __attribute__((always_inline)) -> v8i {
                const uint8_t *w = wb + b * kW;
                if constexpr (TRANS) {
                    // columns 16 q + i16 of tile column wn; block rows 16 g .. and 64 + 16 g ..
                    const uint8_t *a = w + (g >> 1) * 8192 + wn * 2048 + q * 512 + (g & 1) * 256 + i16 * 8;
                    auto tr = [&](int at) {
                        return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) v2i *)(a + at));
                    };
                    const v2i a0 = tr(0), a1 = tr(128), a2 = tr(2 * 8192), a3 = tr(2 * 8192 + 128);
                    return (v8i){a0.x, a0.y, a1.x, a1.y, a2.x, a2.y, a3.x, a3.y};
                } else {
                    const uint8_t *a = w + (2 * wn + (q >> 1)) * 4096 + g * 512 + swizzled_row(a_row(i16, q)) * 16;
                    return operand(*reinterpret_cast<const u32x4 *>(a), *reinterpret_cast<const u32x4 *>(a + 2048));
                }
            };

            v8i wf[2][4];
            float fw_next = weight_scale(0);
            int wr = 1, wc = 0;  // weight buffers of block s + 1 (read) and of block s (copied into)
            // block s with the weights wf[H], those of block s + 1 into wf[H ^ 1]
            auto block = [&](int s, auto h_c) __attribute__((always_inline)) {
                constexpr int H = decltype(h_c)::value;
                // all copies but the weights of block s + 2 have arrived, and every wave is done
                // with block s - 1 and has its weights of block s
                if (s == 1) wait_newer((n > 3 ? 4 : 0) + stores);
                else if (s + 2 < n && s > 0) wait_copies<4>();
                else if (s > 0) wait_copies<0>();
                lds_barrier();
                if ((s & 3) == 0 && s + 4 < n) copy_s(cur, s + 4);
                if (s > 0 && s + 1 < n) copy_x(cur, s + 1);
                if (MSA < 2 && s + 3 < n) copy_w(s + 3, wc);
                if (s == 0 && more) announce(next);
                if constexpr (MSA > 0) {
                    const uint8_t *x = xb + (s & 1) * kX + (16 * wm + i16) * 128;
                    const float *fs = sb + (s & 4) * kBM + (16 * wm + i16) * 4 + (s & 3);
                    const float fw = fw_next;
                    fw_next = weight_scale(s + 1);
                    auto x_operand = [&](int i) __attribute__((always_inline)) -> v8i {
                        const uint8_t *q = x + i * 4096;
                        return operand(*reinterpret_cast<const u32x4 *>(q + ((g ^ (i16 & 7)) * 16)),
                                       *reinterpret_cast<const u32x4 *>(q + (((4 + g) ^ (i16 & 7)) * 16)));
                    };
                    v8i xf = x_operand(0);
                    float f = fs[0], f_prev = f_last;
#pragma unroll
                    for (int i = 0; i < MSA; ++i) {
                        const v8i xi = xf;
                        const float fi = f * fw;
                        if (i + 1 < MSA) {
                            xf = x_operand(i + 1);
                            f = fs[128 * (i + 1)];  // times fw a piece later, when it is there
                        }
                        // the next block's weights: one read a piece, the rest with the last
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (q == i || (i == MSA - 1 && q > i)) wf[H ^ 1][q] = w_operand(wr, q);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int u = 4 * i + q;
                            d[q] = block_dot(wf[H][q], xi);
                            pin(d[q]);
                            __builtin_amdgcn_sched_barrier(0);  // the sums behind the MFMA, not before it
                            if (q < 2) add((u + U - 2) % U, f_prev);
                            else add(u - 2, fi);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                        f_prev = fi;
                        if (i == 1 && s + 3 < n) copy_w(s + 3, wc);  // not in one burst with the rows
                    }
                    f_last = f_prev;
                }
                wr = wr == 2 ? 0 : wr + 1;
                wc = wc == 2 ? 0 : wc + 1;
            };

            wait_newer((n > 2 ? 4 : 0) + stores);
            lds_barrier();
            if constexpr (MSA > 0) {
#pragma unroll
                for (int q = 0; q < 4; ++q) wf[0][q] = w_operand(0, q);
            }
#pragma clang loop unroll(disable)
            for (int s = 0; s < n; s += 2) {
                block(s, std::integral_constant<int, 0>{});
                if (s + 1 < n) block(s + 1, std::integral_constant<int, 1>{});
            }
            if (n < 3) wait_copies<0>();  // the announced slots: from block 2 on they are waited for with its copies
            lds_barrier();  // every wave is done with the buffers
            if (more) {
                sources(next, true);
                copy_first(next);
            }
            if constexpr (MSA > 0) {
                add(U - 2, f_last);
                add(U - 1, f_last);
            }

            // ---- outputs: 16 bytes a lane, whole 128-byte lines an instruction
            stores = cur.c0 + 64 * wn < C && MSA > 0 ? 2 * MSA - 1 : 0;
            if (cur.c0 + 64 * wn < C) {
                const bool odd = i16 & 1;
#pragma unroll
                for (int i = 0; i < MSA; ++i) {
                    const int m = 16 * (2 * i + wm) + (i16 & ~1);  // of a pair of rows
                    u32x4 v[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint2 a = make_uint2(bf16_pair(acc[i][2 * h][0], acc[i][2 * h][1]),
                                                   bf16_pair(acc[i][2 * h][2], acc[i][2 * h][3]));
                        const uint2 b = make_uint2(bf16_pair(acc[i][2 * h + 1][0], acc[i][2 * h + 1][1]),
                                                   bf16_pair(acc[i][2 * h + 1][2], acc[i][2 * h + 1][3]));
                        // columns 32 h + 8 g ..; transposed 16 (2 h + g % 2) + 8 (g / 2) ..
                        v[h] = TRANS ? swap_groups(a, b) : (u32x4){a.x, a.y, b.x, b.y};
                    }
                    const int col = (odd ? 32 : 0) + (TRANS ? 16 * (g & 1) + 8 * (g >> 1) : 8 * g);
                    const RowPair r = swap_rows(v[0], v[1], odd);
                    uint16_t *o = p.out + (int64_t)(cur.p0 + m) * C + cur.c0 + 64 * wn + col;
                    if (m < cur.rows) *reinterpret_cast<u32x4 *>(o) = r.x[0];
                    if (m + 1 < cur.rows) *reinterpret_cast<u32x4 *>(o + C) = r.x[1];
                }
            }
        };
        // pieces 2 i + wm < n_sub; every wave runs the same copies and barriers
        switch ((n_sub - wm + 1) / 2) {
            case 0: run(std::integral_constant<int, 0>{}); break;
            case 1: run(std::integral_constant<int, 1>{}); break;
            case 2: run(std::integral_constant<int, 2>{}); break;
            case 3: run(std::integral_constant<int, 3>{}); break;
            case 4: run(std::integral_constant<int, 4>{}); break;
            case 5: run(std::integral_constant<int, 5>{}); break;
            case 6: run(std::integral_constant<int, 6>{}); break;
            default: run(std::integral_constant<int, 7>{}); break;
        }
        if (!more) break;
        cur = next;
    }
}

// Few rows per group (decode): bound by the weights' bytes, and the tile kernel's items of 256
// columns are too few to go round the CUs. A workgroup takes 32 columns of one tile of rows, its
// four waves a quarter of the blocks each; weights go straight into registers, 16 bytes a lane from
// 512 consecutive bytes an instruction's half, and the four partial sums meet in LDS in the waves'
// order. Up to 32 rows have two blocks' loads ahead of the products, more rows share a turn's
// weights in four pieces with one block ahead: 134 registers, three workgroups a CU (four blocks
// ahead of two pieces or two of four cost that and 5 %, four ahead of one piece 1 us of 28). One token
// through 8 of 64 experts, 5120 x 4096: 27.7 us for 168 MB (6.1 TB/s); two tokens 52 us (6.4 TB/s); 64
// tokens that meet 71 of 96 local experts of 384: 212 us for 1.49 GB (7.0 TB/s).
__global__ void __launch_bounds__(256, 3) stream_kernel(const BlockGemmArgs p) {
    __shared__ __attribute__((aligned(16))) float part[4][64][36];
    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int n = p.R / 128, nb = p.C / 32;
    const int n_tiles = p.v.offsets ? scalar_load(&p.v.ctrl->n_tiles) : p.v.max_tiles;
    const int tile = blockIdx.x / nb, cb = blockIdx.x % nb;
    if (tile >= n_tiles) return;
    int e = 0, p0 = tile * kBM, rows = p.v.rows - p0;
    if (p.v.offsets) {
        e = scalar_load(p.v.tile_expert + tile);
        p0 = scalar_load(p.v.tile_row0 + tile);
        rows = scalar_load(p.v.offsets + e + 1) - p0;
    }
    rows = min(rows, kBM);
    // columns 16 q + i16 of the 32, pieces g of both halves of a block
    const uint8_t *w = uniform(p.w_codes + e * p.w_expert_bytes + (int64_t)cb * (p.R / 64) * 2048);
    const uint32_t w_lane = g * 512 + i16 * 16;
    const float *sw = uniform(p.w_scales + (int64_t)e * p.w_expert_scales + cb / 4 * p.w_kb);
    const int64_t x_step = (int64_t)p.x_rows * 128;
    // MT pieces of 16 rows from m0 on, UNROLL blocks' loads ahead of the products
    auto turn = [&](int m0, auto mt_c, auto unroll_c) __attribute__((always_inline)) {
        constexpr int MT = decltype(mt_c)::value, UNROLL = decltype(unroll_c)::value;
        const uint8_t *x[MT];
        const float *sx[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int pos = p0 + min(m0 + 16 * m + i16, rows - 1);
            const uint32_t row = p.by_token ? p.v.sorted_slot[pos] / p.v.top_k : pos;
            x[m] = p.x_codes + row * 128 + g * 16;
            sx[m] = p.x_scales + (int64_t)row * scale_stride(p.R);
        }
        f4 acc[MT][2] = {};
        for (int b0 = wave; b0 < n; b0 += 4 * UNROLL) {
            u32x4 wv[UNROLL][4], xv[UNROLL][MT][2];
            float f[UNROLL][MT];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int b = min(b0 + 4 * u, n - 1);  // past the end: the last block again, with factor 0
                const uint8_t *wb = w + (int64_t)b * 4096;
#pragma unroll
                for (int j = 0; j < 4; ++j)  // column half j / 2, block half j % 2
                    wv[u][j] = __builtin_nontemporal_load(
                        reinterpret_cast<const u32x4 *>(wb + w_lane + (j >> 1) * 256 + (j & 1) * 2048));
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    xv[u][m][0] = *reinterpret_cast<const u32x4 *>(x[m] + b * x_step);
                    xv[u][m][1] = *reinterpret_cast<const u32x4 *>(x[m] + b * x_step + 64);
                    f[u][m] = b0 + 4 * u < n ? sx[m][b] * sw[b] : 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const v8i xo = operand(xv[u][m][0], xv[u][m][1]);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const f4 d = block_dot(operand(wv[u][2 * q], wv[u][2 * q + 1]), xo);
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[m][q][v] = fmaf(d[v], f[u][m], acc[m][q][v]);
                    }
                }
        }
        // accumulator v of read q: column 16 q + 4 g + v of row 16 m + i16
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q) *reinterpret_cast<f4 *>(&part[wave][16 * m + i16][16 * q + 4 * g]) = acc[m][q];
        __syncthreads();
        const int c = 2 * (t & 15);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = 16 * m + (t >> 4);
            if (m0 + r < rows) {
                float a = part[0][r][c], b = part[0][r][c + 1];
#pragma unroll
                for (int k = 1; k < 4; ++k) {
                    a += part[k][r][c];
                    b += part[k][r][c + 1];
                }
                *reinterpret_cast<uint32_t *>(p.out + (int64_t)(p0 + m0 + r) * p.C + 32 * cb + c) = bf16_pair(a, b);
            }
        }
    };
    using std::integral_constant;
    int m0 = 0;
    for (; rows - m0 > 32; m0 += 64) turn(m0, integral_constant<int, 4>{}, integral_constant<int, 1>{});
    if (rows - m0 > 16) turn(m0, integral_constant<int, 2>{}, integral_constant<int, 2>{});
    else if (rows > m0) turn(m0, integral_constant<int, 1>{}, integral_constant<int, 2>{});
}

}  // namespace

// The stream kernel from here down; 5120 x 4096, stream against tile kernel. 96 experts of 384, top 8,
// even routing: 64 tokens 202 : 243 us, 256 292 : 350, 384 303 : 347; but with a few hot experts (rows
// of one group take turns over its weights) 256 tokens 295 : 292, 448 403 : 338, so the grouped limit
// stays below the even crossing. One group: 16 rows 9.1 : 18.7, 64 17.3 : 25.9, 96 26.4 : 30.0, 128
// 32.1 : 33.3. Both limits come from this one shape and go by rows alone: other shapes are not measured, and
// a few experts of 6 to 96 rows each in groups take the tile kernel, which one such group alone loses by
// (64 rows: 25.9 for 17.3 us). Transposed there is no kernel for few rows: one group of 16 takes 33 us, 64 42.
constexpr int kStreamMean = 5, kStreamRows = 96;

hipError_t launch_block_gemm(const BlockGemmArgs &a, bool transposed, hipStream_t s) {
    const int64_t groups = (int64_t)a.v.max_tiles * (a.C / 32);  // 2^24 workgroups are a grid's limit
    if (!transposed && a.v.mean_rows <= (a.v.offsets ? kStreamMean : kStreamRows) && groups < 1 << 24) {
        hipLaunchKernelGGL(stream_kernel, dim3((unsigned)groups), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const int64_t items = (int64_t)a.v.max_tiles * ((a.C + kBN - 1) / kBN);
    if (items > INT32_MAX - 8) return hipErrorInvalidValue;
    const unsigned grid = (unsigned)(items >= kMaxGrid ? kMaxGrid : (items + 7) / 8 * 8);
    if (transposed) hipLaunchKernelGGL(tile_kernel<true>, dim3(grid), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL(tile_kernel<false>, dim3(grid), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
