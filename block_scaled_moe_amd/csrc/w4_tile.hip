// w4_tile.hip - product of many rows a group with 4-bit weights (include/moe_w4.h, moe_w4_gemm; the arithmetic stands in
// w4_mma.h).
//
// 128 rows x 64 NF columns a workgroup, 8 waves as 2 (rows) x 4 (columns), a wave up to 4 pieces of 16 rows (the tile's pieces
// alternate between the two row waves, so that a partial tile splits evenly) x 16 NF columns; with swiglu half of a wave's
// columns are the first half's and half the same ones of the second half, so that both meet in one lane.
//  - Stages of 128 of the reduction. Rows (gathered by token) and codes go straight from memory into LDS, three buffers
//    each, scales and zero points into two buffers of 256 of the reduction; one barrier a stage covers everything. It
//    stands before the last quarter of a stage's products, whose operands are in registers by then: its buffers take the stage
//    three ahead at once, and the next stage's operands are read and expanded behind those products.
//  - The sums of x per row and group are the same for all columns: each wave forms those of one piece of 16 rows, two stages
//    ahead, and leaves them in LDS, from where they are the products' first addends.
//  - MFMAs (16 clocks) and other vector instructions (4 clocks) are about as much work, so each MFMA stands beside the
//    instructions that expand a later operand or add an earlier group's sum.
//  - A workgroup a CU (157 KiB of LDS) walks its items, parts with many rows first. Where the next part's rows are is found out
//    while this one's first stages arrive: three loads in a row, each of which needs the one before, no longer begin a part.
// Bound by waits: on 8192 rows of 96 experts, 5120 x 4096, groups of 128, the matrix cores are busy 33% of the cycles and other vector
// instructions take 36%; a wave issues in 36% of its time, waits for its turn in 24%, and in 40% for LDS and for the other waves at a
// stage's barrier, which two waves a SIMD do not hide. About 8 us of an item are its beginning and end. That product: 538 us in the
// median, 514 at best (0.64 to 0.67 PFLOP/s; 1920 items, of which a workgroup takes seven or eight). 3003 rows of 60 experts (1 to 553
// each), 1002 x 2592, groups of 32: 104 us; a fourth more with the parts in the list's order, a tenth once they are spread over
// the XCDs. Evenly routed the order costs 2%.
#include "w4_mma.h"
#include "w4_parts.h"

namespace moe {
namespace {

using namespace w4;

constexpr int kThreads = 512, kBM = kW4PartRows, kStage = 128;
constexpr int kGrid = 256;  // workgroups: one a CU
constexpr int kX = kBM * kStage * 2;  // LDS bytes of a stage's rows

// copy_to_lds from any address
__device__ __forceinline__ void copy_from(const void *src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(uniform((int)dst)), "v"(src) : "memory");
}

// a word a lane
__device__ __forceinline__ void copy_words(const void *src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, off" ::"s"(uniform((int)dst)), "v"(src) : "memory");
}

template <int GROUP, bool HALF, bool ZEROS, int NF>
__global__ void __launch_bounds__(kThreads) tile_kernel(const W4GemmArgs p) {
    constexpr int kBN = 64 * NF;
    constexpr int kTiles = kBN / 16 + (NF == 2 ? 1 : 0);      // packed tiles: a second half may start inside one
    constexpr int kGroups = kW4Step / GROUP, kIn = kStage / GROUP;  // groups per step, per stage
    constexpr int kW = kTiles * 1024;                         // LDS bytes of a stage's codes
    constexpr int kS = kTiles * 32 * kGroups, kZ = ZEROS ? kS / 2 : 0;  // of a step's scales and zero points
    constexpr int kLds = 3 * (kX + kW) + 2 * (kS + kZ) + 3 * kIn * kBM * 4 + 2 * kBM * 4 + 4 * kThreads;
    constexpr int kWCopies = kBN / 16 / 8;  // of codes by every wave in a stage (the first one: perhaps one more)
    constexpr int kSWaves = (kS + 1023) / 1024, kZWaves = (kZ + 1023) / 1024;
    static_assert(kLds <= 160 * 1024 && kSWaves + kZWaves <= 8, "LDS");
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
    uint8_t *const xb = lds, *const wb = lds + 3 * kX, *const sb = wb + 3 * kW, *const zb = sb + 2 * kS;
    float *const sums = reinterpret_cast<float *>(zb + 2 * kZ);
    int32_t *const slots = reinterpret_cast<int32_t *>(sums + 3 * kIn * kBM);  // of the rows of this part and of the next one
    uint16_t *const order = reinterpret_cast<uint16_t *>(slots + 2 * kBM);

    const Expander expand;
    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const int i16 = lane & 15, g = lane >> 4, wm = wave >> 2, wn = wave & 3;
    const int K = p.w.K, stages = (K + kStage - 1) / kStage;
    const int width = p.swiglu ? kBN / 2 : kBN;  // output columns a workgroup
    const int nb = (p.C + width - 1) / width;

    // ---- work items: parts of 128 rows (a tile of the groups' list is one or two) times column blocks, those with most rows
    // first: workgroups then take about as much work each, however uneven the groups are. kThreads tiles of the list are brought
    // into that order at a time: its parts by the number of their pieces, in `order` as 2 * tile + part.
    const int n_tiles = p.v.offsets ? scalar_load(&p.v.ctrl->n_tiles) : (p.v.rows + kBM - 1) / kBM;
    auto sort_parts = [&](int tile0) __attribute__((always_inline)) -> int {
        int *const count = reinterpret_cast<int *>(sums), *const place = count + 64;  // by pieces (8 first), then waves
        int pieces[2] = {0, 0};  // of this thread's tile's parts
        if (tile0 + t < n_tiles) {
            const int left = p.v.offsets[p.v.tile_expert[tile0 + t] + 1] - p.v.tile_row0[tile0 + t];
            pieces[0] = (w4_part_rows(left, kGroupTile, 0) + 15) / 16;
            pieces[1] = (w4_part_rows(left, kGroupTile, 1) + 15) / 16;
        }
        int before[2] = {0, 0};  // parts of as many pieces before it in its wave
        const uint64_t lower = (1ull << lane) - 1;
#pragma unroll
        for (int n = 1; n <= 8; ++n) {
            const uint64_t b0 = __ballot(pieces[0] == n), b1 = __ballot(pieces[1] == n);
            if (pieces[0] == n) before[0] = __popcll(b0 & lower);
            if (pieces[1] == n) before[1] = __popcll(b0) + __popcll(b1 & lower);
            if (lane == 0) count[(8 - n) * 8 + wave] = __popcll(b0) + __popcll(b1);
        }
        __syncthreads();
        if (wave == 0) {
            const int own = count[lane];
            int sum = own;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int v = __shfl_up(sum, off);
                if (lane >= off) sum += v;
            }
            place[lane] = sum - own;
            if (lane == 63) place[64] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (pieces[i] > 0) order[place[(8 - pieces[i]) * 8 + wave] + before[i]] = (uint16_t)(2 * t + i);
        const int n = uniform(place[64]);
        __syncthreads();
        return n;
    };
    struct Part {
        int item, e, part, p0, end;  // expert; which of its tile; first row, the one behind the last
    };
    int parity = 0;
    for (int tile0 = 0; tile0 < n_tiles; tile0 += p.v.offsets ? kThreads : n_tiles) {
    // Up to two parts' items in a row, whose rows and codes then meet in one L2, go to each XCD (workgroups 8 apart) in turn, each
    // time from another one on.
    const int items = (p.v.offsets ? sort_parts(tile0) : n_tiles) * nb, unit = min(2 * nb, max(items / 32, 1));
    // this workgroup's j-th item, -1: none, but there may be more; items: no more
    auto item_of = [&](int j) __attribute__((always_inline)) -> int {
        const int turn = j / unit;
        if (turn * 8 * unit >= items) return items;
        const int item = (8 * turn + ((blockIdx.x - turn) & 7)) * unit + j % unit;
        return item < items ? item : -1;
    };
    auto first_of = [&](int item, Part &q) __attribute__((always_inline)) {
        q.item = item;
        if (p.v.offsets) {
            const int at = uniform((int)order[item / nb]), tile = tile0 + at / 2;
            q.e = scalar_load(p.v.tile_expert + tile);
            q.part = at % 2;
            q.p0 = scalar_load(p.v.tile_row0 + tile) + q.part * kBM;
        } else {
            q.e = q.part = 0, q.p0 = item / nb * kBM;
        }
    };
    auto end_of = [&](Part &q) __attribute__((always_inline)) {
        const int left = (p.v.offsets ? scalar_load(p.v.offsets + q.e + 1) : p.v.rows) - (q.p0 - q.part * kBM);
        q.end = uniform(q.p0 + w4_part_rows(left, kGroupTile, q.part));
    };
    auto copy_slots = [&](const Part &q, int buffer) __attribute__((always_inline)) {
        if (p.by_token && wave < kBM / 64)
            copy_words(p.v.sorted_slot + min(q.p0 + 64 * wave + lane, q.end - 1), lds_address(slots + buffer * kBM + 64 * wave));
    };
    auto following = [&](int &j) __attribute__((always_inline)) -> int {
        int item;
        do {
            item = item_of(j);
            j += gridDim.x >> 3;
        } while (item < 0);
        return item;
    };
    int j_next = blockIdx.x >> 3;
    Part part, next;
    part.item = following(j_next);
    if (part.item >= items) continue;
    first_of(part.item, part);
    end_of(part);
    copy_slots(part, parity);
    wait_copies<0>();
    lds_barrier();
    for (;;) {
    // what says where the next part's rows are arrives beside this one's rows
    next.item = following(j_next);
    if (next.item < items) first_of(next.item, next);
    const int e = part.e, cb = part.item % nb, p0 = part.p0, rows = part.end - p0;

    // ---- sources. Rows: copies wave + 8 j of four rows of 256 bytes; a row's 16-byte pieces are swapped by the row's last
    // four bits, so that sixteen rows' pieces of one place lie in different banks.
    const int n_sub = (rows + 15) / 16;
    const uint16_t *x[4];
    const int x_at = ((lane & 15) ^ ((4 * wave + (lane >> 4)) & 15)) * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int in = min(4 * (wave + 8 * j) + (lane >> 4), rows - 1);
        const uint32_t row = p.by_token ? token_of(slots[parity * kBM + in], p) : p0 + in;
        x[j] = p.x + (int64_t)row * K;
    }
    // Packed tiles in LDS order; past the end the last one, whose columns are not stored.
    auto packed_tile = [&](int j) __attribute__((always_inline)) -> int64_t {
        int tile = cb * (width / 16) + j;
        if (p.swiglu && j >= kBN / 32) tile = (p.C + cb * width) / 16 + j - kBN / 32;
        return ((int64_t)e * p.tiles + min(tile, p.tiles - 1)) * p.steps;
    };
    const uint8_t *codes[kWCopies + 1];
#pragma unroll
    for (int j = 0; j <= kWCopies; ++j)
        codes[j] = uniform(reinterpret_cast<const uint8_t *>(p.w.codes) + packed_tile(min(wave + 8 * j, kTiles - 1)) * 2048);
    // 16 bytes a lane of the step's scales (waves from 0 on) or zero points (the next ones)
    const bool side_z = wave >= kSWaves;
    const int side_lane = (side_z ? wave - kSWaves : wave) * 64 + lane;
    const bool side_on = side_lane < (side_z ? kZ : kS) / 16;
    const int side_bytes = side_z ? 16 * kGroups : 32 * kGroups;  // of a tile
    const uint8_t *side = side_z ? p.w.zeros : reinterpret_cast<const uint8_t *>(p.w.scales);
    if (side_on) side += packed_tile(side_lane * 16 / side_bytes) * side_bytes + side_lane * 16 % side_bytes;

    const uint32_t x_lds = lds_address(xb) + wave * 1024, w_lds = lds_address(wb) + wave * 1024;
    const uint32_t side_lds = lds_address(side_z ? zb : sb) + (side_z ? wave - kSWaves : wave) * 1024;
    auto copy_side = [&](int step) __attribute__((always_inline)) {
        if (side_on) copy_from(side + (int64_t)step * side_bytes, side_lds + (step & 1) * (side_z ? kZ : kS));
    };
    auto copy_x = [&](int s, int buffer) __attribute__((always_inline)) {
        const int k = min(s * kStage + x_at, K - 8);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (wave + 8 * j < 4 * n_sub) copy_from(x[j] + k, x_lds + buffer * kX + j * 8192);
    };
    auto copy_w = [&](int s, int buffer) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j <= kWCopies; ++j)
            if (wave + 8 * j < kTiles && (j < kWCopies || p.swiglu))
                copy_to_lds(codes[j] + (int64_t)s * 1024, lane * 16, w_lds + buffer * kW + j * 8192);
    };

    // ---- this lane's columns: row of the packed tiles in LDS
    int w_row[NF], w_at[NF];  // and place in its codes
#pragma unroll
    for (int q = 0; q < NF; ++q) {
        w_row[q] = (wn * NF + q) * 16 + i16;
        if (p.swiglu) {
            const int in = (wn * (NF / 2) + q % (NF / 2)) * 16 + i16;
            w_row[q] = q < NF / 2 ? in : kBN / 2 + ((p.C + cb * width) & 15) + in;
        }
        w_at[q] = (w_row[q] >> 4) * 1024 + (16 * g + (w_row[q] & 15)) * 16;
    }

    // sums of x over the groups of stage s for the 16 rows of piece `wave`, times minus 24, or with zero points, which
    // are read times 8, times minus 1 / 8
    auto row_sums = [&](int buffer) __attribute__((always_inline)) {
        if (wave >= n_sub) return;
        const uint8_t *row = xb + buffer * kX + (16 * wave + i16) * 256;
#pragma unroll
        for (int gr = 0; gr < kIn; ++gr) {
            f4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int r = gr * (GROUP / 32); r < (gr + 1) * (GROUP / 32); ++r)
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf8, *reinterpret_cast<const u32x4 *>(row + ((4 * r + g) ^ i16) * 16)), ones(), d, 0, 0, 0);
            if (i16 == 0) *reinterpret_cast<f4 *>(sums + (buffer * kIn + gr) * kBM + 16 * wave + 4 * g) = d * (ZEROS ? -0.125f : -24.0f);
        }
    };

    copy_side(0);
    if (stages > 2) copy_side(1);
#pragma unroll
    for (int s = 0; s < 3; ++s)
        if (s < stages) copy_x(s, s);
#pragma unroll
    for (int s = 0; s < 3; ++s)
        if (s < stages) copy_w(s, s);
    if (next.item < items) {
        asm volatile("" : "+s"(next.e), "+s"(next.p0));
        end_of(next);
        asm volatile("" : "+s"(next.end));
    }
    if (stages > 2) wait_copies<2 * kWCopies>();
    else wait_copies<0>();
    lds_barrier();
    if (next.item < items) copy_slots(next, parity ^ 1);
    row_sums(0);
    if (stages > 1) row_sums(1);
    lds_barrier();

    auto run = [&](auto mf_c) __attribute__((always_inline)) {
        constexpr int MF = decltype(mf_c)::value, kRuns = GROUP / 32;  // this wave's pieces of 16 rows; MFMAs in a row of a group
        f4 acc[MF][NF], d[MF][NF];  // d: of the group that is summed
        float f_last[NF];           // and its scales
#pragma unroll
        for (int q = 0; q < NF; ++q) {
            f_last[q] = 0.0f;
#pragma unroll
            for (int i = 0; i < MF; ++i) acc[i][q] = d[i][q] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
        }
        // what a stage's products need of its columns
        struct Columns {
            u32x4 raw[NF];
            uint32_t s[NF][(kIn + 1) / 2], z[NF];
        };
        auto read_columns = [&](int s, int buffer, Columns &c) __attribute__((always_inline)) {
#pragma unroll
            for (int q = 0; q < NF; ++q) {
                c.raw[q] = *reinterpret_cast<const u32x4 *>(wb + buffer * kW + w_at[q]);
                const uint8_t *sp = sb + ((s >> 1) & 1) * kS + w_row[q] * (2 * kGroups) + (s & 1) * (2 * kIn);
                if constexpr (kIn == 1) c.s[q][0] = *reinterpret_cast<const uint16_t *>(sp);
                else if constexpr (kIn == 2) c.s[q][0] = *reinterpret_cast<const uint32_t *>(sp);
                else c.s[q][0] = reinterpret_cast<const u32x2 *>(sp)->x, c.s[q][1] = reinterpret_cast<const u32x2 *>(sp)->y;
                if constexpr (ZEROS) {
                    const uint8_t *zp = zb + ((s >> 1) & 1) * kZ + w_row[q] * kGroups + (s & 1) * kIn;
                    if constexpr (kIn == 1) c.z[q] = *zp;
                    else if constexpr (kIn == 2) c.z[q] = *reinterpret_cast<const uint16_t *>(zp);
                    else c.z[q] = *reinterpret_cast<const uint32_t *>(zp);
                }
            }
        };
        const uint8_t *const rows_at = xb + (16 * wm + i16) * 256;
        // operand n = MF r + i of the stage in `buffer`: rows of piece i, columns 32 r ..
        auto read_rows = [&](int buffer, int n) __attribute__((always_inline)) -> bf8 {
            return __builtin_bit_cast(bf8, *reinterpret_cast<const u32x4 *>(rows_at + buffer * kX + n % MF * 8192 + ((4 * (n / MF) + g) ^ i16) * 16));
        };
        Columns c, cn;
        bf8 x0 = read_rows(0, 0), x1 = read_rows(0, 1);
        u32x4 w[NF];
        read_columns(0, 0, c);
#pragma unroll
        for (int q = 0; q < NF; ++q) w[q] = __builtin_bit_cast(u32x4, expand(c.raw[q][0]));
        int b0 = 0, b1 = 1, b2 = 2;  // buffers of stages s (and s + 3), s + 1, s + 2
#pragma clang loop unroll(disable)
        for (int s = 0; s < stages; ++s) {
            const float *sum_at = sums + b0 * kIn * kBM + 16 * wm + 4 * g;
            bf8 x[4 * MF];
            u32x4 wn[NF];
            x[0] = x0, x[1] = x1;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int gr = r / kRuns;
                if (r == 3) {
                    // everything but the codes of stage s + 2 has arrived, and every wave is done with the buffers of stage s
                    if (s + 2 < stages) wait_copies<kWCopies>();
                    else wait_copies<0>();
                    lds_barrier();
                    if (s + 3 < stages) {
                        if (s & 1) copy_side((s + 3) / 2);
                        copy_x(s + 3, b0);
                        copy_w(s + 3, b0);
                    }
                    read_columns(s + 1, b1, cn);  // behind the last stage what is there, unused
                    x0 = read_rows(b1, 0), x1 = read_rows(b1, 1);
                }
                float f[NF], off[NF];
                if (r % kRuns == 0) {
#pragma unroll
                    for (int q = 0; q < NF; ++q) {
                        f[q] = scale_value<HALF>(c.s[q][gr / 2], gr & 1);
                        if constexpr (ZEROS) off[q] = (float)((c.z[q] >> (8 * gr)) & 255u);  // times 8
                    }
                }
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    const int n = MF * r + i;
                    if (n + 2 < 3 * MF) x[n + 2] = read_rows(b0, n + 2);
                    if (r == 2) x[3 * MF + i] = read_rows(b0, 3 * MF + i);
                    f4 sum;
                    if (r % kRuns == 0) sum = *reinterpret_cast<const f4 *>(sum_at + gr * kBM + 32 * i);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int q = 0; q < NF; ++q) {
                        const f4 last = d[i][q];
                        d[i][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            x[n], __builtin_bit_cast(bf8, w[q]), r % kRuns != 0 ? last : ZEROS ? sum * off[q] : sum, 0, 0, 0);
                        pin(d[i][q]);
                        __builtin_amdgcn_sched_barrier(0);  // what follows behind the MFMA, not before it
                        if (r % kRuns == 0) {               // the group before is done
#pragma unroll
                            for (int v = 0; v < 4; ++v) acc[i][q][v] = fmaf(last[v], f_last[q], acc[i][q][v]);
                            pin(acc[i][q]);
                        }
                        // the next operands of the columns, in equal parts
                        const int slot = i * NF + q;
#pragma unroll
                        for (int e = 0; e < 4 * NF; ++e)
                            if (e >= slot * 4 / MF && e < (slot + 1) * 4 / MF) {
                                wn[e / 4][e % 4] = expand.pair(r < 3 ? c.raw[e / 4][r < 3 ? r + 1 : 0] : cn.raw[e / 4][0], e % 4);
                                asm volatile("" ::"v"(wn[e / 4][e % 4]));
                            }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
#pragma unroll
                for (int q = 0; q < NF; ++q) {
                    w[q] = wn[q];
                    if (r % kRuns == 0) f_last[q] = f[q];
                }
            }
            if (s + 2 < stages) row_sums(b2);
            c = cn;
            const int b = b0;
            b0 = b1, b1 = b2, b2 = b;
        }
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int q = 0; q < NF; ++q)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][q][v] = fmaf(d[i][q][v], f_last[q], acc[i][q][v]);

        // ---- outputs: accumulator v of (i, q): row 16 (2 i + wm) + 4 g + v, column 16 q + i16
        auto store = [&](auto swiglu_c) __attribute__((always_inline)) {
            constexpr bool kSwiglu = decltype(swiglu_c)::value;
            constexpr int kOut = kSwiglu ? NF / 2 : NF;
            const int c0 = cb * (kSwiglu ? kBN / 2 : kBN) + wn * kOut * 16;  // the wave's first column
            auto value = [&](int i, int q) __attribute__((always_inline)) -> f4 {
                f4 y = acc[i][q];
                if constexpr (kSwiglu) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) y[v] = swiglu(y[v], acc[i][q + kOut][v]);
                }
                return y;
            };
            if (p.out_dtype != MOE_DT_BF16) {
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    const int m = 16 * (2 * i + wm) + 4 * g;
                    float *o = static_cast<float *>(p.out) + (int64_t)(p0 + m) * p.C + c0 + i16;
#pragma unroll
                    for (int q = 0; q < kOut; ++q) {
                        const f4 y = value(i, q);
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            if (m + v < rows && c0 + 16 * q + i16 < p.C) o[(int64_t)v * p.C + 16 * q] = y[v];
                    }
                }
                return;
            }
            // four lanes exchange their four rows of four columns: each then stores four columns of one row
            const bool odd = i16 & 1, upper = i16 & 2;
            const int col = c0 + (i16 & ~3);
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                const int m = 16 * (2 * i + wm) + 4 * g + (i16 & 3);
                uint16_t *o = static_cast<uint16_t *>(p.out) + (int64_t)(p0 + m) * p.C + col;
#pragma unroll
                for (int q = 0; q < kOut; ++q) {
                    const f4 y = value(i, q);
                    uint32_t pair[2];  // columns 2 (i16 / 2), + 1 of rows 2 h + i16 % 2
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float give = odd ? y[2 * h] : y[2 * h + 1];
                        const float got = __uint_as_float(
                            __builtin_amdgcn_update_dpp(0, __float_as_uint(give), 0xB1, 0xF, 0xF, true));  // quad_perm 1, 0, 3, 2
                        pair[h] = bf16_pair(odd ? got : y[2 * h], odd ? y[2 * h + 1] : got);
                    }
                    const uint32_t got = __builtin_amdgcn_update_dpp(0, upper ? pair[0] : pair[1], 0x4E, 0xF, 0xF, true);  // 2, 3, 0, 1
                    const u32x2 out = upper ? (u32x2){got, pair[1]} : (u32x2){pair[0], got};
                    if (m >= rows) continue;
                    if (p.C % 4 == 0) {
                        if (col + 16 * q < p.C) *reinterpret_cast<u32x2 *>(o + 16 * q) = out;
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (col + 16 * q + j < p.C) o[16 * q + j] = (uint16_t)(out[j / 2] >> (16 * (j & 1)));
                    }
                }
            }
        };
        if (p.swiglu) store(std::integral_constant<bool, true>{});
        else store(std::integral_constant<bool, false>{});
    };
    using std::integral_constant;
    switch ((n_sub - wm + 1) / 2) {
        case 4: run(integral_constant<int, 4>{}); break;
        case 3: run(integral_constant<int, 3>{}); break;
        case 2: run(integral_constant<int, 2>{}); break;
        default: run(integral_constant<int, 1>{}); break;  // none: beside the other waves, nothing of it is stored
    }
    lds_barrier();  // every wave is done with the buffers
    parity ^= 1;
    if (next.item >= items) break;
    part = next;
    }
    }
}

}  // namespace

hipError_t launch_w4_tile(const W4GemmArgs &a, hipStream_t s) {
    const int64_t tiles = a.v.offsets ? a.v.max_tiles : (a.v.rows + kBM - 1) / kBM;
    auto items = [&](int columns) { return tiles * ((a.C + columns - 1) / columns); };
    // A second half that starts inside a packed tile needs one more of them, for which only the narrow tile has room, as for the
    // sums of groups of 32. Else by the items of a call, us of the narrow tiles and the wide: 50 rows each of 64 experts, K 2560,
    // 156 items 30.6, 44.1; 390 items 66.6, 71.3; 624 items 86, 77; 1248 items 171, 144. One weight, K 2560, 96 items 35, 51; 320
    // items 92, 99; 576 items 152, 145 (between them, where the narrow ones begin one round of the CUs more, the wide are up to a
    // sixth faster: 256 items 66, 57).
    const bool narrow = a.w.group == 32 || (a.swiglu && a.C % 16) || items(a.swiglu ? 128 : 256) < 512;
    const int64_t n = ((a.v.offsets ? 2 : 1) * items(narrow ? (a.swiglu ? 64 : 128) : (a.swiglu ? 128 : 256)) + 7) / 8 * 8;
    if (n > INT32_MAX) return hipErrorInvalidValue;
    const int64_t grid = n < kGrid ? n : kGrid;
    w4::by_form(a.w, [&](auto group, auto half, auto zeros) {
        constexpr int kGroup = decltype(group)::value;
        constexpr bool kHalf = decltype(half)::value, kZeros = decltype(zeros)::value;
        if constexpr (kGroup > 32) {
            if (!narrow) {
                hipLaunchKernelGGL((tile_kernel<kGroup, kHalf, kZeros, 4>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
                return;
            }
        }
        hipLaunchKernelGGL((tile_kernel<kGroup, kHalf, kZeros, 2>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
    });
    return hipGetLastError();
}

}  // namespace moe
