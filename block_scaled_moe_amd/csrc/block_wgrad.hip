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
// the writes of dw. One workgroup per CU walks its items, and the first two runs of the next item
// are copied before the outputs of the last are stored: a wave's vector memory operations
// complete in order, so the copies can be waited for while the stores drain behind them.
#include "block_mma.h"
#include "ops_internal.h"

namespace moe {
namespace {

using namespace block;

constexpr int kThreads = 512, kB = 256, kMaxGrid = 256;
constexpr int kOperand = kB * 128;
#ifndef NT
#define NT 0
#endif
#define MOE_WGRAD_STORE(v, p) do { if (NT) __builtin_nontemporal_store(v, p); else *(p) = v; } while (0)

__global__ void __launch_bounds__(kThreads) wgrad_kernel(const BlockWgradArgs p) {
    __shared__ __attribute__((aligned(16))) uint8_t gb[2 * kOperand];
    __shared__ __attribute__((aligned(16))) uint8_t xb[2 * kOperand];
    __shared__ __attribute__((aligned(16))) float sg[2 * kB], sx[2 * kB];

    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int i16 = lane & 15, g = lane >> 4;
    const int N = p.N, K = p.K;
    const int nbn = (N + kB - 1) / kB, nbk = (K + kB - 1) / kB;
    const int items = p.n * nbn * nbk, per_xcd = (items + 7) / 8;  // each XCD: a contiguous range
    const int step = (gridDim.x + 7) / 8;
    const uint32_t g_lds = lds_address(gb) + wave * 4096, x_lds = lds_address(xb) + wave * 4096;
    const uint32_t s_lds = wave == 0 ? lds_address(sx) : lds_address(sg);
    const uint32_t x_lane = (lane >> 5) * 512 + swizzled_row(lane & 31) * 16;

    struct Item {
        int e, n0, k0, runs;
        bool n_half, k_half;  // only 128 of the 256 columns exist: the first half is copied twice
        const uint8_t *g, *x, *s;  // this wave's 32 columns of both operands; scales (waves 0, 1)
    };
    auto item = [&](int w) __attribute__((always_inline)) {
        Item a;
        a.e = w / (nbn * nbk);
        const int r = w % (nbn * nbk);
        a.n0 = r / nbk * kB;
        a.k0 = r % nbk * kB;
        int first = 0, cnt = p.rows;
        if (p.offsets) {
            first = scalar_load(p.offsets + a.e);
            cnt = scalar_load(p.offsets + a.e + 1) - first;
        }
        a.runs = (cnt + 127) / 128;
        const int64_t run0 = p.offsets ? first / 128 + a.e : 0;
        a.n_half = a.n0 + 128 >= N;
        a.k_half = a.k0 + 128 >= K;
        a.g = p.g_codes + run0 * N * 128 + (int64_t)(a.n0 / 32 + (a.n_half ? wave & 3 : wave)) * 4096;
        a.x = p.x_codes + run0 * K * 128 + (int64_t)(a.k0 / 32 + (a.k_half ? wave & 3 : wave)) * 4096;
        a.s = reinterpret_cast<const uint8_t *>(wave == 0 ? p.x_scales + run0 * K + a.k0 : p.g_scales + run0 * N + a.n0);
        a.g = uniform(a.g);
        a.x = uniform(a.x);
        a.s = uniform(a.s);
        return a;
    };
    constexpr int kCopies = 8;  // of a run by a wave (nine by the two that copy scales)
    auto copy = [&](const Item &a, int s) __attribute__((always_inline)) {
        const uint8_t *gsrc = a.g + (int64_t)s * N * 128, *xsrc = a.x + (int64_t)s * K * 128;
        const uint32_t b = (s & 1) * kOperand;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            copy_to_lds(gsrc + j * 1024, lane * 16, g_lds + b + j * 1024);
            copy_to_lds(xsrc + j * 1024, x_lane, x_lds + b + j * 1024);
        }
        if (wave < 2) {
            const bool half = wave == 0 ? a.k_half : a.n_half;
            copy_to_lds(a.s + (int64_t)s * (wave == 0 ? K : N) * 4, (half ? lane & 31 : lane) * 16, s_lds + (s & 1) * kB * 4);
        }
    };
    // at most `newer` (rounded down to 0, 8, 16, 24) of the wave's operations outstanding
    auto wait = [&](int newer) __attribute__((always_inline)) {
        if (newer >= 24) wait_copies<24>();
        else if (newer >= 16) wait_copies<16>();
        else if (newer >= 8) wait_copies<8>();
        else wait_copies<0>();
    };

    int it = blockIdx.x >> 3;
    const int base = (blockIdx.x & 7) * per_xcd, end = min(per_xcd, items - base);
    if (it >= end) return;
    Item cur = item(base + it);
    if (cur.runs > 0) copy(cur, 0);
    if (cur.runs > 1) copy(cur, 1);
    int stores = 0;  // of the last item by this wave, issued behind the copies of cur's first two runs
    for (;;) {
        it += step;
        const bool more = it < end;
        const Item next = item(base + (more ? it : end - 1));

        f4 acc[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][q] = (f4){0.0f, 0.0f, 0.0f, 0.0f};

#pragma clang loop unroll(disable)
        for (int s = 0; s < cur.runs; ++s) {
            const int ahead = s + 1 < cur.runs ? kCopies : 0;  // the next run's copies
            wait(s < 2 ? ahead + stores : ahead);
            lds_barrier();
            const uint8_t *xl = xb + (s & 1) * kOperand, *gl = gb + (s & 1) * kOperand;
            const float *fsx = sx + (s & 1) * kB, *fsg = sg + (s & 1) * kB;
            // n = n0 + 16 (2 i + wm) + i16, k = k0 + 64 wn + 32 (q / 2) + 8 g + 4 (q % 2) + v
            v8i xf[4];
            f4 fx[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint8_t *a = xl + (2 * wn + (q >> 1)) * 4096 + g * 512 + swizzled_row(a_row(i16, q)) * 16;
                xf[q] = operand(*reinterpret_cast<const u32x4 *>(a), *reinterpret_cast<const u32x4 *>(a + 2048));
                fx[q] = *reinterpret_cast<const f4 *>(fsx + 64 * wn + 32 * (q >> 1) + 8 * g + 4 * (q & 1));
            }
            auto g_operand = [&](int i) __attribute__((always_inline)) -> v8i {  // columns 16 (2 i + wm) ..
                const uint8_t *b = gl + i * 4096 + g * 512 + (16 * wm + i16) * 16;
                return operand(*reinterpret_cast<const u32x4 *>(b), *reinterpret_cast<const u32x4 *>(b + 2048));
            };
            // block sums are added to their accumulators two MFMAs later
            f4 d[3];
            float f[8];
            auto add = [&](int u) __attribute__((always_inline)) {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    acc[u / 4][u % 4][v] = fmaf(d[u % 3][v], fx[u % 4][v] * f[u / 4], acc[u / 4][u % 4][v]);
                pin(acc[u / 4][u % 4]);
            };
            v8i gv = g_operand(0);
            f[0] = fsg[16 * wm + i16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const v8i gi = gv;
                if (i + 1 < 8) {
                    gv = g_operand(i + 1);
                    f[i + 1] = fsg[32 * (i + 1) + 16 * wm + i16];
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int u = 4 * i + q;
                    d[u % 3] = block_dot(xf[q], gi);
                    pin(d[u % 3]);
                    if (u >= 2) add(u - 2);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            add(30);
            add(31);
            lds_barrier();  // every wave is done with the buffer
            if (s + 2 < cur.runs) copy(cur, s + 2);
        }

        if (more && next.runs > 0) copy(next, 0);
        if (more && next.runs > 1) copy(next, 1);
        stores = 0;
        if (!cur.k_half || wn < 2) {
            stores = cur.n_half ? 8 : 16;
            uint8_t *o = reinterpret_cast<uint8_t *>(p.dw + ((int64_t)cur.e * N + cur.n0) * K + cur.k0);
            const uint32_t at = ((uint32_t)(16 * wm + i16) * K + 64 * wn + 8 * g) * 2;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i < 4 || !cur.n_half) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const u32x4 v = {bf16_pair(acc[i][2 * h][0], acc[i][2 * h][1]),
                                         bf16_pair(acc[i][2 * h][2], acc[i][2 * h][3]),
                                         bf16_pair(acc[i][2 * h + 1][0], acc[i][2 * h + 1][1]),
                                         bf16_pair(acc[i][2 * h + 1][2], acc[i][2 * h + 1][3])};
                        MOE_WGRAD_STORE(v, reinterpret_cast<u32x4 *>(o + (int64_t)64 * i * K + 64 * h + at));
                    }
                }
            }
        }
        if (!more) break;
        cur = next;
    }
}

}  // namespace

hipError_t launch_block_wgrad(const BlockWgradArgs &a, hipStream_t s) {
    const int64_t items = (int64_t)a.n * ((a.N + kB - 1) / kB) * ((a.K + kB - 1) / kB);
    if (items > INT32_MAX - 8) return hipErrorInvalidValue;
    const unsigned grid = (unsigned)(items >= kMaxGrid ? kMaxGrid : (items + 7) / 8 * 8);
    hipLaunchKernelGGL(wgrad_kernel, dim3(grid), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
