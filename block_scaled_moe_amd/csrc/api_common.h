// api_common.h - argument checks that the host sides of the operators' C ABIs share.
#pragma once
#include <stdint.h>

#include <initializer_list>

#include "../../include/moe_ops.h"

namespace moe {

inline bool aligned(const void *p, uintptr_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
inline bool type_ok(int32_t dtype) { return dtype == MOE_DT_BF16 || dtype == MOE_DT_FP32; }
inline int64_t type_bytes(int32_t dtype) { return dtype == MOE_DT_BF16 ? 2 : 4; }
inline int32_t status_of(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// A buffer of a call: n items of `item` bytes at p (NULL: not given).
struct Extent {
    const void *p;
    int64_t n, item;
};
inline bool meet(const Extent &a, const Extent &b) {
    typedef unsigned __int128 wide;  // sizes that no memory holds are compared too
    const wide a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a.p && b.p && a.n && b.n && a0 < b0 + (wide)b.n * (wide)b.item && b0 < a0 + (wide)a.n * (wide)a.item;
}
// An output meets another output or an input.
inline bool outputs_meet(std::initializer_list<Extent> outputs, std::initializer_list<Extent> inputs) {
    for (auto o = outputs.begin(); o != outputs.end(); ++o) {
        for (auto p = o + 1; p != outputs.end(); ++p)
            if (meet(*o, *p)) return true;
        for (const Extent &i : inputs)
            if (meet(*o, i)) return true;
    }
    return false;
}

}  // namespace moe
