// block_wgrad.hip - gradient of the expert weights from E4M3 column forms of the output
// gradient and of the input (include/moe_ops.h, moe_block_wgrad).
//
//   dw[e][n][k] = sum over e's runs b of 128 rows of sg[b][n] sx[b][k] * sum over the run of cg * cx
//
// 128 (n) x 256 (k) outputs per workgroup of four waves, a wave 128 x 64. The input's columns
// are the MFMA's A operand, so a lane's accumulators are consecutive k of one n. Both operands
// of a run are contiguous in the column form and go straight into LDS, with their scales. An
// expert has few runs (its rows / 128), so a workgroup is mostly its 64 KiB of output: bound by
// the writes of dw. Two workgroups share a CU (one buffer of 50 KiB, 256 registers a lane), one
// loading or storing while the other multiplies.
#include "block_mma.h"
#include "ops_internal.h"

namespace moe {
namespace {

using namespace block;

constexpr int kThreads = 256, kBN = 128, kBK = 128;

__global__ void __launch_bounds__(kThreads, 4) wgrad_kernel(const BlockWgradArgs p) {
    __shared__ __attribute__((aligned(16))) uint8_t gl[kBN * 128];
    __shared__ __attribute__((aligned(16))) uint8_t xl[kBK * 128];
    __shared__ __attribute__((aligned(16))) float sg[kBN], sx[kBK];

    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6), wm = wave >> 1, wn = wave & 1;
    const int i16 = lane & 15, g = lane >> 4;
    const int N = p.N, K = p.K;
    const int nbn = N / kBN, nbk = K / kBK;
    // each XCD takes a contiguous range of items, expert by expert
    const int items = p.n * nbn * nbk, per_xcd = (items + 7) / 8;
    const int w = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
    if (w >= items) return;
    const int e = w / (nbn * nbk), r = w % (nbn * nbk);
    const int n0 = r / nbk * kBN, k0 = r % nbk * kBK;

    int first = 0, cnt = p.rows;
    if (p.offsets) {
        first = p.offsets[e];
        cnt = p.offsets[e + 1] - first;
    }
    const int runs = (cnt + 127) / 128;
    const int64_t run0 = p.offsets ? first / 128 + e : 0;

    // a wave copies 32 columns of n and of k, wave 0 the scales
    const uint8_t *gs = uniform(p.g_codes + run0 * N * 128 + (int64_t)(n0 / 32 + wave) * 4096);
    const uint8_t *xs = uniform(p.x_codes + run0 * K * 128 + (int64_t)(k0 / 32 + wave) * 4096);
    const uint32_t x_lane = (lane >> 5) * 512 + swizzled_row(lane & 31) * 16;
    const uint8_t *gf = uniform(reinterpret_cast<const uint8_t *>(p.g_scales + run0 * N + n0));
    const uint8_t *xf32 = uniform(reinterpret_cast<const uint8_t *>(p.x_scales + run0 * K + k0));
    const uint32_t g_lds = lds_address(gl) + wave * 4096, x_lds = lds_address(xl) + wave * 4096;
    const uint32_t sg_lds = lds_address(sg), sx_lds = lds_address(sx);
    auto copy = [&](int s) __attribute__((always_inline)) {
        const uint8_t *gsrc = gs + (int64_t)s * N * 128, *xsrc = xs + (int64_t)s * K * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            copy_to_lds(gsrc + j * 1024, lane * 16, g_lds + j * 1024);
            copy_to_lds(xsrc + j * 1024, x_lane, x_lds + j * 1024);
        }
        if (wave == 0 && lane < 32) {
            copy_to_lds(xf32 + (int64_t)s * K * 4, lane * 16, sx_lds);
            copy_to_lds(gf + (int64_t)s * N * 4, lane * 16, sg_lds);
        }
    };

    f4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s) acc[i][s] = (f4){0.0f, 0.0f, 0.0f, 0.0f};

#pragma clang loop unroll(disable)
    for (int s = 0; s < runs; ++s) {
        if (s > 0) lds_barrier();  // the last run's reads
        copy(s);
        wait_copies<0>();
        lds_barrier();
        // n = n0 + 64 wm + 16 i + i16, k = k0 + 64 wn + 32 (q / 2) + 8 g + 4 (q % 2) + v
        v8i xf[4];
        f4 fx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint8_t *a = xl + (2 * wn + (q >> 1)) * 4096 + g * 512 + swizzled_row(a_row(i16, q)) * 16;
            xf[q] = operand(*reinterpret_cast<const u32x4 *>(a), *reinterpret_cast<const u32x4 *>(a + 2048));
            fx[q] = *reinterpret_cast<const f4 *>(sx + 64 * wn + 32 * (q >> 1) + 8 * g + 4 * (q & 1));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t *b = gl + (2 * wm + (i >> 1)) * 4096 + g * 512 + (16 * (i & 1) + i16) * 16;
            const v8i gv = operand(*reinterpret_cast<const u32x4 *>(b), *reinterpret_cast<const u32x4 *>(b + 2048));
            const float fg = sg[64 * wm + 16 * i + i16];
            f4 d[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) d[q] = block_dot(xf[q], gv);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][q][v] = fmaf(d[q][v], fx[q][v] * fg, acc[i][q][v]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint16_t *o = p.dw + ((int64_t)e * N + n0 + 64 * wm + 16 * i + i16) * K + k0 + 64 * wn + 8 * g;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 v = {bf16_pair(acc[i][2 * h][0], acc[i][2 * h][1]), bf16_pair(acc[i][2 * h][2], acc[i][2 * h][3]),
                                 bf16_pair(acc[i][2 * h + 1][0], acc[i][2 * h + 1][1]),
                                 bf16_pair(acc[i][2 * h + 1][2], acc[i][2 * h + 1][3])};
                *reinterpret_cast<u32x4 *>(o + 32 * h) = v;
            }
        }
    }
}

}  // namespace

hipError_t launch_block_wgrad(const BlockWgradArgs &a, hipStream_t s) {
    const int64_t items = (int64_t)a.n * (a.N / kBN) * (a.K / kBK);
    if (items > INT32_MAX - 8) return hipErrorInvalidValue;
    hipLaunchKernelGGL(wgrad_kernel, dim3((unsigned)((items + 7) / 8 * 8)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
