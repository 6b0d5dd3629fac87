// w4_internal.h - launchers of the operators declared in include/moe_w4.h, shared between their kernel
// files and the host API (w4_api.hip). Every launcher enqueues on `stream` and returns hipGetLastError().
#pragma once
#include "../../include/moe_w4.h"
#include "ops_internal.h"

namespace moe {

constexpr int32_t kW4Rows = 16, kW4Step = 256;  // of a tile, columns of a step of the packed form

inline int64_t w4_tiles(const moe_w4_weights &w) { return ((int64_t)w.N + kW4Rows - 1) / kW4Rows; }
inline int64_t w4_steps(const moe_w4_weights &w) { return ((int64_t)w.K + kW4Step - 1) / kW4Step; }

hipError_t launch_w4_pack(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, const moe_w4_weights &w,
                          hipStream_t s);

struct W4GemmArgs {
    GroupView v;
    int32_t by_token, swiglu, out_dtype;
    const uint16_t *x;
    moe_w4_weights w;
    int32_t tiles, steps;  // of the packed form
    int32_t C;             // columns of out
    int32_t shares;        // workgroups that share the turns over a tile's rows (set by the launcher)
    uint32_t slot_factor;  // 2^31 / top_k rounded up
    void *out;
};
// Token of a slot below 2^28 (x has fewer than 2^25 rows): the factor is less than 8 / 2^31 too large, relative to 1 / top_k,
// which does not reach the next whole number.
__device__ __forceinline__ uint32_t token_of(uint32_t slot, const W4GemmArgs &a) { return __umulhi(2 * slot, a.slot_factor); }
hipError_t launch_w4_gemm(const W4GemmArgs &a, hipStream_t s);
hipError_t launch_w4_tile(const W4GemmArgs &a, hipStream_t s);  // groups of many rows

}  // namespace moe
