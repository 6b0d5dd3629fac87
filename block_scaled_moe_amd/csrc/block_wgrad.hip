// block_wgrad.hip - gradient of the expert weights from E4M3 column forms of the output
// gradient and of the input (include/moe_ops.h, moe_block_wgrad).
//
//   dw[e][n][k] = sum over e's runs b of 128 rows of sg[b][n] sx[b][k] * sum over the run of cg * cx
//
// 256 (n) x 256 (k) outputs per work item, 8 waves as 2 (n) x 4 (k), 16-column pieces of n
// alternating between the two. The input's columns are the MFMA's A operand, so a lane's
// accumulators are consecutive k of one n. Both operands of a run are contiguous 32 KiB in the
// column form and go straight into one of two LDS buffers. An expert has few runs (its rows /
// 128), so the item is mostly its 128 KiB of output: bound by the writes of dw.
#include "block_mma.h"
#include "ops_internal.h"

namespace moe {
namespace {

using namespace block;

constexpr int kThreads = 512, kBN = 256;
constexpr int kOperand = 256 * 128;

__global__ void __launch_bounds__(kThreads) wgrad_kernel(const BlockWgradArgs p) {
    __shared__ __attribute__((aligned(16))) uint8_t gb0[kOperand];
    __shared__ __attribute__((aligned(16))) uint8_t gb1[kOperand];
    __shared__ __attribute__((aligned(16))) uint8_t xb0[kOperand];
    __shared__ __attribute__((aligned(16))) uint8_t xb1[kOperand];

    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wm = wave >> 2, wn = wave & 3;
    const int i16 = lane & 15, g = lane >> 4;
    const int N = p.N, K = p.K;
    const int nbn = (N + kBN - 1) / kBN, nbk = (K + kBN - 1) / kBN;
    const int64_t w = blockIdx.x;
    const int e = (int)(w / (nbn * nbk)), r = (int)(w % (nbn * nbk));
    const int n0 = r / nbk * kBN, k0 = r % nbk * kBN;

    int first = 0, cnt = p.rows;
    if (p.offsets) {
        first = p.offsets[e];
        cnt = p.offsets[e + 1] - first;
    }
    const int runs = (cnt + 127) / 128;
    const int64_t run0 = p.offsets ? first / 128 + e : 0;

    // this wave's 32 columns of both operands (half a block of columns: its first half again)
    int gt = n0 / 32 + wave, xt = k0 / 32 + wave;
    if (gt * 32 >= N) gt -= 4;
    if (xt * 32 >= K) xt -= 4;
    const uint8_t *gs = p.g_codes + run0 * N * 128 + (int64_t)gt * 4096 + lane * 16;
    const uint8_t *xs = p.x_codes + run0 * K * 128 + (int64_t)xt * 4096 + (lane >> 5) * 512 + swizzled_row(lane & 31, wave) * 16;
    auto copy = [&](uint8_t *gd, uint8_t *xd, int s) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            copy_to_lds(gs + (int64_t)s * N * 128 + j * 1024, gd + wave * 4096 + j * 1024);
            copy_to_lds(xs + (int64_t)s * K * 128 + j * 1024, xd + wave * 4096 + j * 1024);
        }
    };
    // scales of this lane's outputs: n = n0 + 16 (2 i + wm) + i16, k = k0 + 64 wn + 16 g + 4 s + v
    const bool k_in = k0 + 64 * wn < K;
    const float *sg = p.g_scales + run0 * N, *sx = p.x_scales + run0 * K + (k_in ? k0 + 64 * wn + 16 * g : 0);
    auto n_of = [&](int i) { return n0 + 16 * (2 * i + wm) + i16; };

    f4 acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s) acc[i][s] = (f4){0.0f, 0.0f, 0.0f, 0.0f};

    auto run_step = [&](const uint8_t *gl, const uint8_t *xl, uint8_t *g_next, uint8_t *x_next, int s)
                        __attribute__((always_inline)) {
        wait_copies<0>();
        lds_barrier();
        f4 fx[4];
        float fg[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) fx[q] = *reinterpret_cast<const f4 *>(sx + (int64_t)s * K + 4 * q);
#pragma unroll
        for (int i = 0; i < 8; ++i) fg[i] = sg[(int64_t)s * N + min(n_of(i), N - 1)];
        if (s + 1 < runs) copy(g_next, x_next, s + 1);
        v8i xf[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int rt = 2 * wn + (i16 >> 3), row = 16 * ((i16 >> 2) & 1) + 4 * q + (i16 & 3);
            const uint8_t *a = xl + rt * 4096 + g * 512 + swizzled_row(row, rt) * 16;
            xf[q] = operand(*reinterpret_cast<const u32x4 *>(a), *reinterpret_cast<const u32x4 *>(a + 2048));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 16 * (2 * i + wm);  // column of the item
            const uint8_t *b = gl + (c >> 5) * 4096 + g * 512 + ((c & 31) + i16) * 16;
            const v8i gf = operand(*reinterpret_cast<const u32x4 *>(b), *reinterpret_cast<const u32x4 *>(b + 2048));
            f4 d[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) d[q] = block_dot(xf[q], gf);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][q][v] = fmaf(d[q][v], fx[q][v] * fg[i], acc[i][q][v]);
        }
        lds_barrier();  // every wave is done with the buffer before it is refilled
    };

    if (runs > 0) {
        copy(gb0, xb0, 0);
        for (int s = 0; s < runs; s += 2) {
            run_step(gb0, xb0, gb1, xb1, s);
            if (s + 1 < runs) run_step(gb1, xb1, gb0, xb0, s + 1);
        }
    }

    if (k_in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int nn = n_of(i);
            if (nn < N) {
                uint16_t *o = p.dw + ((int64_t)e * N + nn) * K + k0 + 64 * wn + 16 * g;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<uint4 *>(o + 8 * h) =
                        make_uint4(bf16_pair(acc[i][2 * h][0], acc[i][2 * h][1]), bf16_pair(acc[i][2 * h][2], acc[i][2 * h][3]),
                                   bf16_pair(acc[i][2 * h + 1][0], acc[i][2 * h + 1][1]),
                                   bf16_pair(acc[i][2 * h + 1][2], acc[i][2 * h + 1][3]));
            }
        }
    }
}

}  // namespace

hipError_t launch_block_wgrad(const BlockWgradArgs &a, hipStream_t s) {
    const int64_t items = (int64_t)a.n * ((a.N + kBN - 1) / kBN) * ((a.K + kBN - 1) / kBN);
    if (items > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(wgrad_kernel, dim3((unsigned)items), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
