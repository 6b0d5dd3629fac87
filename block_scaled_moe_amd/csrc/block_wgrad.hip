// block_wgrad.hip - gradient of the expert weights from E4M3 column forms of the output
// gradient and of the input (include/moe_ops.h, moe_block_wgrad).
//
//   dw[e][n][k] = sum over e's runs b of 128 rows of sg[b][n] sx[b][k] * sum over the run of cg * cx
//
// 256 (n) x 256 (k) outputs per work item, 8 waves as 2 (n) x 4 (k), 16-column pieces of n
// alternating between the two. The input's columns are the MFMA's A operand, so a lane's
// accumulators are consecutive k of one n. Both operands of a run are contiguous in the column
// form and go straight into LDS with their scales (two buffers).
//
// An expert has few runs (its rows / 128), so an item is mostly its 128 KiB of output: bound by
// the writes of dw, with the copies of a run (64 KiB) and its products behind them. One workgroup
// per CU walks its items; the runs of all of them make one sequence of steps. A step's copies go to
// the buffer of the step before it, a quarter behind each of the first pieces' products of the step
// in between: one barrier a step, and no burst of copies that the waves wait to issue. A wave's vector memory
// operations complete in order, so a step waits for its own copies by the number of stores issued
// behind them, and the stores of an item drain under the next steps. A lane swaps half its outputs
// with its neighbour, so that every store instruction writes whole 128-byte lines, which go past
// L2 (non-temporal) and leave the operands there.
//
// 96 experts of 4096 x 2560, 17108 rows unevenly routed: 504 us, of which the stores alone are 340 to
// 380 us (2.0 GB, up to 5.9 TB/s), the copies alone 130 us and the products about 200 us (as many
// cycles of the vector unit: each MFMA's four results take four products of scales and four multiply-adds).
// Stores overlap with products, but hardly with copies of the same CU: stores spread over the next
// item's first step, among its copies, took 615 us, a step's copies in one burst behind the step before
// 590 us; tiles of 128 x 256 with two workgroups a CU 600 us, sweeps along k that keep the block of n
// in LDS 700 us (uneven experts), ordinary stores 546 us, an expert on one XCD instead of eight 603 us.
#include "block_mma.h"
#include "ops_internal.h"

#include <type_traits>

namespace moe {
namespace {

using namespace block;

constexpr int kThreads = 512, kB = 256, kOperand = kB * 128, kMaxGrid = 256;

__global__ void __launch_bounds__(kThreads) wgrad_kernel(const BlockWgradArgs p) {
    __shared__ __attribute__((aligned(16))) uint8_t gb[2 * kOperand];
    __shared__ __attribute__((aligned(16))) uint8_t xb[2 * kOperand];
    __shared__ __attribute__((aligned(16))) float sgb[2 * kB], sxb[2 * kB];

    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int i16 = lane & 15, g = lane >> 4;
    const int N = p.N, K = p.K;
    const int nbk = (K + kB - 1) / kB, tiles = (N + kB - 1) / kB * nbk;

    // An expert's tiles are split over `split` XCDs and the experts dealt to the 8 / split sets of
    // XCDs, so that many experts of very different size load them evenly; a part has four tiles or
    // more, which share operands in the XCD's L2. With fewer experts than sets the other sets have
    // nothing to do, and few tiles in all leave most CUs idle: one group of 8192 rows takes 559 us
    // at 512 x 512 (one workgroup works), 281 at 1024 x 1024 (eight), 160 at 4096 x 2560, 328 at 5120 x 4096.
    const int split = tiles >= 32 ? 8 : tiles >= 16 ? 4 : tiles >= 8 ? 2 : 1;
    const int xcd = blockIdx.x & 7, sets = 8 / split, part = (tiles + split - 1) / split;
    const int r0 = xcd % split * part, mine = min(part, tiles - r0), e0 = xcd / split;
    const int end = mine > 0 && e0 < p.n ? (p.n - e0 + sets - 1) / sets * mine : 0;
    const int step = gridDim.x >> 3;

    const uint32_t g_lds = lds_address(gb) + wave * 4096, x_lds = lds_address(xb) + wave * 4096;
    const uint32_t sx_lds = lds_address(sxb), sg_lds = lds_address(sgb);
    const uint32_t x_lane = (lane >> 5) * 512 + swizzled_row(lane & 31) * 16;

    struct Item {
        int it, e, n0, k0, runs;
        int64_t run0;
    };
    auto item = [&](int it) __attribute__((always_inline)) {
        Item a;
        const int r = r0 + it % mine;
        a.it = it;
        a.e = e0 + it / mine * sets;
        a.n0 = r / nbk * kB;
        a.k0 = r % nbk * kB;
        int o = 0, cnt = p.rows;
        if (p.offsets) {
            o = scalar_load(p.offsets + a.e);
            cnt = scalar_load(p.offsets + a.e + 1) - o;
        }
        a.runs = (cnt + 127) / 128;
        a.run0 = p.offsets ? o / 128 + a.e : 0;
        return a;
    };
    // Only 128 of a block's 256 columns may exist: they are copied twice then.
    auto n_half = [&](const Item &a) { return a.n0 + 128 >= N; };
    auto k_half = [&](const Item &a) { return a.k0 + 128 >= K; };
    // a quarter of a step's copies
    auto copy = [&](const Item &a, int s, int buffer, int j) __attribute__((always_inline)) {
        const int64_t run = a.run0 + s;
        const uint32_t b = buffer * kOperand, f = buffer * kB * 4;
        const uint8_t *x = p.x_codes + run * K * 128 + (int64_t)(a.k0 / 32 + (k_half(a) ? wave & 3 : wave)) * 4096;
        const uint8_t *n = p.g_codes + run * N * 128 + (int64_t)(a.n0 / 32 + (n_half(a) ? wave & 3 : wave)) * 4096;
        copy_to_lds(x + j * 1024, x_lane, x_lds + b + j * 1024);
        copy_to_lds(n + j * 1024, lane * 16, g_lds + b + j * 1024);
        if (j == 0 && wave == 0)
            copy_to_lds(reinterpret_cast<const uint8_t *>(p.x_scales + run * K + a.k0), (k_half(a) ? lane & 31 : lane) * 16,
                        sx_lds + f);
        if (j == 0 && wave == 1)
            copy_to_lds(reinterpret_cast<const uint8_t *>(p.g_scales + run * N + a.n0), (n_half(a) ? lane & 31 : lane) * 16,
                        sg_lds + f);
    };
    // at most `newer` (a multiple of 8; 40 stands for more) of the wave's operations outstanding
    auto wait = [&](int newer) __attribute__((always_inline)) {
        if (newer >= 40) wait_copies<40>();
        else if (newer >= 32) wait_copies<32>();
        else if (newer >= 24) wait_copies<24>();
        else if (newer >= 16) wait_copies<16>();
        else if (newer >= 8) wait_copies<8>();
        else wait_copies<0>();
    };

    int it = blockIdx.x >> 3;
    if (it >= end) return;
    Item cur = item(it);
    // the next step to copy: run cs of item c; experts without rows have no steps
    Item c = cur;
    int cs = -1;
    bool left = true;
    auto advance = [&]() __attribute__((always_inline)) {
        ++cs;
        while (left && cs >= c.runs) {
            left = c.it + step < end;
            if (left) c = item(c.it + step);
            cs = 0;
        }
    };
    advance();
    if (left) {
#pragma unroll
        for (int j = 0; j < 4; ++j) copy(c, cs, 0, j);
        advance();
    }
    int buffer = 0, behind = 0;  // operations behind the copies of the next step to compute
    for (;;) {
        f4 acc[8][4];
        // the first step sets the accumulators, the others add to them
        auto run_step = [&](auto first_c) __attribute__((always_inline)) {
            constexpr bool FIRST = decltype(first_c)::value;
            wait(behind);
            lds_barrier();  // and every wave is done with the other buffer
            behind = 0;
            const uint8_t *xl = xb + buffer * kOperand, *gl = gb + buffer * kOperand;
            const float *sx = sxb + buffer * kB, *sg = sgb + buffer * kB + 16 * wm + i16;
            // n = n0 + 16 (2 i + wm) + i16, k = k0 + 64 wn + 32 (q / 2) + 8 g + 4 (q % 2) + v
            v8i xf[4];
            f4 fx[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint8_t *a = xl + (2 * wn + (q >> 1)) * 4096 + g * 512 + swizzled_row(a_row(i16, q)) * 16;
                xf[q] = operand(*reinterpret_cast<const u32x4 *>(a), *reinterpret_cast<const u32x4 *>(a + 2048));
                fx[q] = *reinterpret_cast<const f4 *>(sx + 64 * wn + 32 * (q >> 1) + 8 * g + 4 * (q & 1));
            }
            auto g_operand = [&](int i) __attribute__((always_inline)) -> v8i {
                const uint8_t *b = gl + i * 4096 + g * 512 + (16 * wm + i16) * 16;
                return operand(*reinterpret_cast<const u32x4 *>(b), *reinterpret_cast<const u32x4 *>(b + 2048));
            };
            // block sums are added to their accumulators two MFMAs later
            f4 d[3];
            float f[8];
            auto add = [&](int m) __attribute__((always_inline)) {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    acc[m / 4][m % 4][v] = FIRST ? d[m % 3][v] * (fx[m % 4][v] * f[m / 4])
                                                 : fmaf(d[m % 3][v], fx[m % 4][v] * f[m / 4], acc[m / 4][m % 4][v]);
                pin(acc[m / 4][m % 4]);
            };
            v8i gv = g_operand(0);
            f[0] = sg[0];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const v8i gi = gv;
                if (i + 1 < 8) {
                    gv = g_operand(i + 1);
                    f[i + 1] = sg[32 * (i + 1)];
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int m = 4 * i + q;
                    d[m % 3] = block_dot(xf[q], gi);
                    pin(d[m % 3]);
                    __builtin_amdgcn_sched_barrier(0);  // the sums behind the MFMA, not before it
                    if (m >= 2) add(m - 2);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (i < 4 && left) copy(c, cs, buffer ^ 1, i);
            }
            add(30);
            add(31);
            if (left) advance();
            buffer ^= 1;
        };
        if (cur.runs > 0) {
            run_step(std::true_type{});
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][q] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma clang loop unroll(disable)
        for (int s = 1; s < cur.runs; ++s) run_step(std::false_type{});

        if (!k_half(cur) || wn < 2) {
            const int stores = n_half(cur) ? 8 : 16;
            behind += stores;
            uint8_t *o = reinterpret_cast<uint8_t *>(p.dw + ((int64_t)cur.e * N + cur.n0) * K + cur.k0);
            // row pair i16 & ~1 of a piece, this lane's eight of its 64 k
            const bool odd = i16 & 1;
            const uint32_t at = ((uint32_t)(16 * wm + (i16 & ~1)) * K + 64 * wn + (odd ? 32 : 0) + 8 * g) * 2;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i < 4 || !n_half(cur)) {
                    u32x4 v[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        v[h] = (u32x4){bf16_pair(acc[i][2 * h][0], acc[i][2 * h][1]),
                                       bf16_pair(acc[i][2 * h][2], acc[i][2 * h][3]),
                                       bf16_pair(acc[i][2 * h + 1][0], acc[i][2 * h + 1][1]),
                                       bf16_pair(acc[i][2 * h + 1][2], acc[i][2 * h + 1][3])};
                    const RowPair r = swap_rows(v[0], v[1], odd);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        __builtin_nontemporal_store(r.x[h], reinterpret_cast<u32x4 *>(o + (int64_t)(64 * i + 2 * h) * K + at));
                }
            }
        }
        it += step;
        if (it >= end) break;
        cur = item(it);
    }
}

}  // namespace

hipError_t launch_block_wgrad(const BlockWgradArgs &a, hipStream_t s) {
    const int64_t items = (int64_t)a.n * ((a.N + kB - 1) / kB) * ((a.K + kB - 1) / kB);
    if (items > INT32_MAX / 2) return hipErrorInvalidValue;
    hipLaunchKernelGGL(wgrad_kernel, dim3((unsigned)(items >= kMaxGrid ? kMaxGrid : (items + 7) / 8 * 8)), dim3(kThreads), 0,
                       s, a);
    return hipGetLastError();
}

}  // namespace moe
