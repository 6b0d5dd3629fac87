// w4_pack.hip - 4-bit weights of a checkpoint into the packed form (include/moe_w4.h, moe_w4_pack).
#include "w4_internal.h"

namespace moe {
namespace {

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

// scales (two bytes) or zero points (one, as the lower byte of the bf16 16 + zero): [E][N][groups] -> [E][N/16][K/256][16][per_step]
template <typename T>
__global__ void __launch_bounds__(256) pack_groups_kernel(const T *__restrict__ src, int32_t N, int32_t groups, int32_t per_step,
                                                          int32_t tiles, int32_t steps, int64_t n_out, T *__restrict__ dst) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n_out; i += (int64_t)gridDim.x * 256) {
        const int64_t g = i % per_step, row = i / per_step % 16, at = i / per_step / 16;
        const int64_t step = at % steps, tile = at / steps % tiles, e = at / steps / tiles;
        const int64_t n = 16 * tile + row, k = step * per_step + g;
        T v = 0;
        if (n < N && k < groups) v = src[(e * N + n) * groups + k];
        if constexpr (sizeof(T) == 1) v = 0x80 | (v & 15) << 3;
        dst[i] = v;
    }
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

}  // namespace moe
