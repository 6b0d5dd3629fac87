// block_mma.h - pieces shared by the products of E4M3 codes with a scale per block of 128
// (block_gemm.hip, block_wgrad.hip).
//
// One v_mfma_f32_16x16x128 takes a whole block of 128 of the reduction: D[i][j] = sum over k of
// A[i][k] B[j][k], lane l holding 32 codes of row l % 16 of A and of B and accumulator v =
// D[4 (l / 16) + v][l % 16]. A lane's codes are two pieces of 16: 16 g .. 16 g + 15 and
// 64 + 16 g .. 64 + 16 g + 15 of the block for g = l / 16 (any order serves, the same for A and
// B), the two quarters g of the block's 64-value halves in the tiled layout. The MFMA starts
// from zero and its result is added to the fp32 accumulator times the block's two scales.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace block {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v8i operand(u32x4 lo, u32x4 hi) {
    return (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// sum over one block of 128 (E8M0 scale operands 127: 2^0)
__device__ __forceinline__ f4 block_dot(v8i a, v8i b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, (f4){0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 127, 0, 127);
}

// 16 bytes per lane from global memory straight into LDS at dst + 16 * lane (dst the same for
// the wave) from base + offset, the base the same for the wave. Written in
// assembly, as it has no register to wait for: behind the builtin the compiler puts a wait for
// every copy in flight before the next LDS read, which a ring of buffers cannot have. The
// caller waits (wait_copies) and meets its workgroup (lds_barrier) before the bytes are read.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
// p, the same for every lane of the wave, as a scalar
template <typename T>
__device__ __forceinline__ T *uniform(T *p) {
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);  // unsigned: it comes back as an int
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (T *)((uint64_t)hi << 32 | lo);
}
// *p through the scalar cache, the address the same for the wave: a vector load would have to
// wait for every copy and store in flight before it. For data no kernel writes while this one runs.
template <typename T>
__device__ __forceinline__ T scalar_load(const T *p) {
    return *(const __attribute__((address_space(4))) T *)(uint64_t)uniform(p);
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)uniform((int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p);
}
__device__ __forceinline__ void copy_to_lds(const uint8_t *base, uint32_t offset, uint32_t dst) {
    // m0 (nothing else here uses it) holds the LDS address; five wait states between a vector
    // instruction that wrote base and the copy that reads it
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(uniform((int)dst)), "v"(offset),
                 "s"(uniform(base))
                 : "memory");
}

// the same with 4 bytes per lane, at dst + 4 * lane
__device__ __forceinline__ void copy4_to_lds(const uint8_t *base, uint32_t offset, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, %2" ::"s"(uniform((int)dst)), "v"(offset),
                 "s"(uniform(base))
                 : "memory");
}

// Workgroup barrier that leaves the wave's copies into LDS in flight (__syncthreads waits for
// them all); LDS reads and writes complete first.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// at most N of the wave's vector loads, copies and stores outstanding
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Keeps v's computation above this point: the compiler otherwise sinks a loop's MFMAs behind the
// barriers and copies that follow them, with all of their operands held in registers.
__device__ __forceinline__ void pin(const f4 &v) { asm volatile("" ::"v"(v)); }

typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
// nearest, ties to even, in one instruction (two scalar conversions take four)
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, bf2));
}

// Lane l and lane l ^ 1 hold 16 bytes each, a and b, of two rows (l even: the first); after the
// swap the even lane holds a of both rows and the odd lane b of both: x[0] of the first row, x[1]
// of the second. Eight lanes then store 128 bytes of one row in one instruction.
struct RowPair {
    u32x4 x[2];
};
__device__ __forceinline__ RowPair swap_rows(u32x4 a, u32x4 b, bool odd) {
    RowPair r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t give = odd ? a[j] : b[j];
        const uint32_t got = __builtin_amdgcn_update_dpp(0, give, 0xB1, 0xF, 0xF, true);  // quad_perm 1, 0, 3, 2
        r.x[0][j] = odd ? got : a[j];
        r.x[1][j] = odd ? b[j] : got;
    }
    return r;
}

// 8 bytes per lane, a of one and b of another run of 16 outputs, lane group g (of 16 lanes) holding
// outputs 4 g .. 4 g + 3 of each: after the swap with the neighbouring group a lane holds 16 bytes,
// outputs 8 (g / 2) .. 8 (g / 2) + 7 of run a (g even) or b (g odd).
__device__ __forceinline__ u32x4 swap_groups(uint2 a, uint2 b) {
    const auto x = __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false);
    const auto y = __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false);
    return (u32x4){x[0], y[0], x[1], y[1]};
}

// The MFMA's A operand is read so that a lane's accumulators of four reads q, over 64 columns in
// two tiles of 32, are outputs 32 h + 8 g .. 32 h + 8 g + 7 (h = q / 2): 16 bytes of bf16, and
// the four g of a row 64 bytes in a row. Lane i then takes row 8 (i / 4) + 4 (q % 2) + i % 4 of
// tile q / 2.
__device__ __forceinline__ int a_row(int i, int q) { return 8 * (i >> 2) + 4 * (q & 1) + (i & 3); }
// Row of a 32-row tile kept at position `pos` of its quarter in LDS (an involution): 16 lanes of
// such a read take four runs of 64 bytes, which the swap puts at four different 64-byte
// offsets of 256.
__device__ __forceinline__ int swizzled_row(int pos) { return pos ^ (((pos >> 4) & 1) << 2); }

}  // namespace block
}  // namespace moe
