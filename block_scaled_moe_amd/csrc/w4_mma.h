// w4_mma.h - pieces shared by the products with 4-bit weights (w4_stream.hip, w4_tile.hip).
//
//   y[p][n] = sum over groups g of s[n][g] (sum over k in g of x[p][k] (16 + q[n][k])  -  (16 + z[n][g]) sum over k in g of x[p][k])
//
// 16 + q is a bf16 whose upper four mantissa bits are the code, so that two of the MFMA's operands come from a word of
// eight codes by one shift and one AND-OR; both sums, of x (16 + q) and of x itself, are fp32 sums of the bf16
// MFMA (the second against ones), and what 16 brings in is taken off group by group, where it is at most a few times
// larger than the group's own sum. Scales and zero points meet the sums in fp32: nothing of the weights is rounded.
// Rows and columns past the end of a matrix are filled up with zero scales, so whatever stands in the rows' places there
// (the last values of the same row) adds nothing.
#pragma once
#include "block_mma.h"
#include "w4_internal.h"

#include <type_traits>

namespace moe {
namespace w4 {

using namespace block;

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// eight codes as 16 + q, by one AND-OR of each pair. The constants are held in registers: as literals they cannot go into that
// instruction, and the compiler takes it apart into two.
struct Expander {
    uint32_t mask, base;
    __device__ __forceinline__ Expander() {
        asm("s_mov_b32 %0, 0x00780078" : "=s"(mask));
        asm("v_mov_b32 %0, 0x41804180" : "=v"(base));
    }
    // codes 2 i and 2 i + 1
    __device__ __forceinline__ uint32_t pair(uint32_t w, int i) const {
        return ((i == 0 ? w : i < 3 ? w >> (4 * i) : __builtin_rotateright32(w, 12)) & mask) | base;
    }
    __device__ __forceinline__ bf8 operator()(uint32_t w) const {
        return __builtin_bit_cast(bf8, (u32x4){pair(w, 0), pair(w, 1), pair(w, 2), pair(w, 3)});
    }
};

template <bool HALF>
__device__ __forceinline__ float scale_value(uint32_t word, int upper) {
    const uint32_t u = upper ? word >> 16 : word & 0xFFFFu;
    if constexpr (HALF) return (float)__builtin_bit_cast(_Float16, (uint16_t)u);
    else return __uint_as_float(u << 16);
}

__device__ __forceinline__ bf8 ones() {
    return __builtin_bit_cast(bf8, (u32x4){0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
}
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// f is called with the group, whether scales are fp16, and whether there are zero points
template <typename F>
void by_form(const moe_w4_weights &w, F &&f) {
    using std::integral_constant;
    auto zeros = [&](auto group, auto half) {
        if (w.zeros) f(group, half, integral_constant<bool, true>{});
        else f(group, half, integral_constant<bool, false>{});
    };
    auto type = [&](auto group) {
        if (w.scale_type == MOE_W4_SCALE_FP16) zeros(group, integral_constant<bool, true>{});
        else zeros(group, integral_constant<bool, false>{});
    };
    if (w.group == 32) type(integral_constant<int, 32>{});
    else if (w.group == 64) type(integral_constant<int, 64>{});
    else type(integral_constant<int, 128>{});
}

}  // namespace w4
}  // namespace moe
