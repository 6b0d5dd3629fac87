// tokens.hip - rows of the sorted order from token rows and back, with weights, and the
// gradients of both (include/moe_ops.h, moe_gather .. moe_combine_backward).
//
//   spread   rows[pos(t, j)] = x[t]                          (moe_gather)
//            d_y[pos] = w[t][j] d_out[t], d_w[t][j] = <d_out[t], y[pos]>   (moe_combine_backward)
//   join     out[t] = sum over j ascending of w[t][j] y[pos(t, j)]  (moe_combine; with weights
//            of 1 moe_gather_backward), fp32 fused multiply-adds in slot order, one rounding
//
// Each is bound by memory: a token's row is read or written once and its sorted rows once,
// with no arithmetic to speak of. So work is laid out by token: a thread owns one piece of
// 16 bytes (one element where rows do not end on 16 bytes) of a token's row, finds the
// token's positions, and touches all of its sorted rows; every output is written once by one
// thread, without atomics, so results do not depend on the order of workgroups. 16384 tokens in
// eight slots, 4096 bf16 values: 4.8 to 5.8 TB/s (below, at load_row); one token 3 us, a launch.
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct Bf16 {
    uint16_t u;
};
__device__ __forceinline__ float to_f32(Bf16 v) { return __uint_as_float((uint32_t)v.u << 16); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ Bf16 from_f32<Bf16>(float v) {  // nearest, ties to even
    return {__builtin_bit_cast(uint16_t, (__bf16)v)};
}

// V consecutive elements, loaded and stored in pieces of at most 16 bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V > 16 ? 16 : sizeof(T) * V) Piece {
    T v[V];
};

// Rows are read once and written once here, and the sorted ones of a long batch fill the caches many
// times over: pieces of 16 bytes go past them (16384 tokens of 4096 bf16 values in eight slots:
// gather 276 -> 238 us, join 290 -> 208 us, the gradient of combine 554 -> 472 us: 4.8 to 5.8 TB/s).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <typename P>
__device__ __forceinline__ P load_row(const P *p) {
    if constexpr (sizeof(P) % 16 == 0) {
        P r;
#pragma unroll
        for (int i = 0; i < (int)sizeof(P) / 16; ++i)
            reinterpret_cast<u32x4 *>(&r)[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p) + i);
        return r;
    } else {
        return *p;
    }
}
template <typename P>
__device__ __forceinline__ void store_row(P *p, const P &v) {
    if constexpr (sizeof(P) % 16 == 0) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(P) / 16; ++i)
            __builtin_nontemporal_store(reinterpret_cast<const u32x4 *>(&v)[i], reinterpret_cast<u32x4 *>(p) + i);
    } else {
        *p = v;
    }
}

// Where a workgroup's threads stand: `lanes` (a power of two) threads share a token's row.
struct Span {
    int32_t log_lanes;  // of threads per token
    int32_t pieces;     // per row
    int32_t per_block;  // pieces of a row that one workgroup of grid.y takes
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gather_kernel(int32_t n_tokens, int32_t k, Span sp,
                                                          const int32_t *__restrict__ slot_pos,
                                                          const T *__restrict__ x, T *__restrict__ rows) {
    using P = Piece<T, V>;
    const int lanes = 1 << sp.log_lanes;
    const int64_t t = ((int64_t)blockIdx.x << (8 - sp.log_lanes)) + (threadIdx.x >> sp.log_lanes);
    if (t >= n_tokens) return;
    int32_t pos[8];
    int any = -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        pos[j] = j < k ? slot_pos[t * k + j] : -1;
        any = max(any, pos[j]);
    }
    if (any < 0) return;
    const P *src = reinterpret_cast<const P *>(x) + t * sp.pieces;
    P *dst = reinterpret_cast<P *>(rows);
    const int c0 = blockIdx.y * sp.per_block, c1 = min(c0 + sp.per_block, sp.pieces);
    for (int c = c0 + (threadIdx.x & (lanes - 1)); c < c1; c += lanes) {
        const P v = src[c];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (pos[j] >= 0) store_row(dst + (int64_t)pos[j] * sp.pieces + c, v);
    }
}

template <typename TY, typename TO, int V, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads) join_kernel(int32_t n_tokens, int32_t k, Span sp,
                                                        const int32_t *__restrict__ slot_pos,
                                                        const float *__restrict__ w, const TY *__restrict__ y,
                                                        TO *__restrict__ out) {
    using PY = Piece<TY, V>;
    using PO = Piece<TO, V>;
    const int lanes = 1 << sp.log_lanes;
    const int64_t t = ((int64_t)blockIdx.x << (8 - sp.log_lanes)) + (threadIdx.x >> sp.log_lanes);
    if (t >= n_tokens) return;
    int32_t pos[8];
    float wj[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        pos[j] = j < k ? slot_pos[t * k + j] : -1;
        wj[j] = WEIGHTED && j < k ? w[t * k + j] : 1.0f;
    }
    const PY *src = reinterpret_cast<const PY *>(y);
    PO *dst = reinterpret_cast<PO *>(out) + t * sp.pieces;
    const int c0 = blockIdx.y * sp.per_block, c1 = min(c0 + sp.per_block, sp.pieces);
    for (int c = c0 + (threadIdx.x & (lanes - 1)); c < c1; c += lanes) {
        PY v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (pos[j] >= 0) v[j] = load_row(src + (int64_t)pos[j] * sp.pieces + c);
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (pos[j] >= 0) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    acc[i] = WEIGHTED ? fmaf(wj[j], to_f32(v[j].v[i]), acc[i]) : acc[i] + to_f32(v[j].v[i]);
            }
        PO o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.v[i] = from_f32<TO>(acc[i]);
        store_row(dst + c, o);
    }
}

// One token's rows are read whole by its threads, whose partial dot products meet in a
// fixed tree: lanes of a wave by exchange, the waves of a wide token through LDS.
template <typename TY, typename TO, int V>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(int32_t n_tokens, int32_t k, Span sp,
                                                                    const int32_t *__restrict__ slot_pos,
                                                                    const float *w,  // may be d_w
                                                                    const TO *__restrict__ d_out,
                                                                    const TY *__restrict__ y, TY *__restrict__ d_y,
                                                                    float *d_w) {
    using PY = Piece<TY, V>;
    using PO = Piece<TO, V>;
    __shared__ float part[kThreads / 64][8];
    const int lanes = 1 << sp.log_lanes, lane = threadIdx.x & (lanes - 1);
    const int64_t t = ((int64_t)blockIdx.x << (8 - sp.log_lanes)) + (threadIdx.x >> sp.log_lanes);
    const bool valid = t < n_tokens;
    int32_t pos[8];
    float wj[8], dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        pos[j] = valid && j < k ? slot_pos[t * k + j] : -1;
        wj[j] = valid && j < k ? w[t * k + j] : 0.0f;
        dot[j] = 0.0f;
    }
    if (valid) {
        const PO *src = reinterpret_cast<const PO *>(d_out) + t * sp.pieces;
        const PY *ys = reinterpret_cast<const PY *>(y);
        PY *dst = reinterpret_cast<PY *>(d_y);
        for (int c = lane; c < sp.pieces; c += lanes) {
            const PO g = src[c];
            PY v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (pos[j] >= 0) v[j] = load_row(ys + (int64_t)pos[j] * sp.pieces + c);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (pos[j] >= 0) {
                    PY o;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float gi = to_f32(g.v[i]);
                        dot[j] = fmaf(gi, to_f32(v[j].v[i]), dot[j]);
                        o.v[i] = from_f32<TY>(wj[j] * gi);
                    }
                    store_row(dst + (int64_t)pos[j] * sp.pieces + c, o);
                }
        }
    }
    if (lanes > 64) {
        const int wave = threadIdx.x >> 6, per = lanes >> 6;  // waves of one token
        // each of the first three steps gives half of the sums to the partner lane: ten exchanges, not 48
        // (517 tokens of 1001 fp32 values 9.7 -> 7.7 us; 16384 of 4096 bf16 values in eight slots 478 -> 472 us)
#pragma unroll
        for (int half = 4, off = 32; half > 0; half >>= 1, off >>= 1) {
            const bool upper = threadIdx.x & off;
#pragma unroll
            for (int j = 0; j < half; ++j) {
                const float give = upper ? dot[j] : dot[j + half];
                dot[j] = (upper ? dot[j + half] : dot[j]) + __shfl_xor(give, off);
            }
        }
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) dot[0] += __shfl_xor(dot[0], off);
        // lane bits 5, 4, 3 are the sum's number, highest first
        if ((threadIdx.x & 7) == 0) part[wave][(threadIdx.x & 63) >> 3] = dot[0];
        __syncthreads();
        if (lane < 8 && lane < k && valid) {
            const int first = wave;  // the token's first wave: lane < 8 lies in it
            float sum = 0.0f;
            for (int i = 0; i < per; ++i) sum += part[first + i][lane];
            d_w[t * k + lane] = sum;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            for (int off = lanes >> 1; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off);
        if (lane == 0 && valid) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < k) d_w[t * k + j] = dot[j];
        }
    }
}

// Threads per token: as many as a row has pieces, up to the workgroup. Where there are few
// tokens, a row's pieces go to several workgroups (grid.y) so that one token fills more
// than one CU.
Span make_span(int32_t T, int32_t pieces, bool whole_rows, dim3 &grid) {
    Span sp{};
    while (sp.log_lanes < 8 && (1 << sp.log_lanes) < pieces) ++sp.log_lanes;
    sp.pieces = pieces;
    sp.per_block = pieces;
    const int tokens = kThreads >> sp.log_lanes;  // per workgroup
    grid.x = (unsigned)((T + tokens - 1) / tokens);
    if (!whole_rows && grid.x < 1024) {  // a grid has at most 65535 in y
        const int lanes = 1 << sp.log_lanes;
        sp.per_block = ((pieces - 1) / (65535 * lanes) + 1) * lanes;
    }
    grid.y = (unsigned)((pieces + sp.per_block - 1) / sp.per_block);
    return sp;
}

template <typename T>
hipError_t gather(const moe_groups &g, int32_t D, const void *x, void *rows, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    dim3 grid(1, 1, 1);
    if (D % V == 0) {
        const Span sp = make_span(g.T, D / V, false, grid);
        hipLaunchKernelGGL((gather_kernel<T, V>), grid, dim3(kThreads), 0, s, g.T, g.top_k, sp, g.slot_pos,
                           static_cast<const T *>(x), static_cast<T *>(rows));
    } else {
        const Span sp = make_span(g.T, D, false, grid);
        hipLaunchKernelGGL((gather_kernel<T, 1>), grid, dim3(kThreads), 0, s, g.T, g.top_k, sp, g.slot_pos,
                           static_cast<const T *>(x), static_cast<T *>(rows));
    }
    return hipGetLastError();
}

template <typename TY, typename TO, int V>
hipError_t join(const moe_groups &g, int32_t D, const void *y, const float *w, void *out, hipStream_t s) {
    dim3 grid(1, 1, 1);
    const Span sp = make_span(g.T, D / V, false, grid);
    const TY *py = static_cast<const TY *>(y);
    TO *po = static_cast<TO *>(out);
    if (w)
        hipLaunchKernelGGL((join_kernel<TY, TO, V, true>), grid, dim3(kThreads), 0, s, g.T, g.top_k, sp, g.slot_pos, w,
                           py, po);
    else
        hipLaunchKernelGGL((join_kernel<TY, TO, V, false>), grid, dim3(kThreads), 0, s, g.T, g.top_k, sp, g.slot_pos, w,
                           py, po);
    return hipGetLastError();
}

template <typename TY, typename TO, int V>
hipError_t spread_back(const moe_groups &g, int32_t D, const void *d_out, const void *y, const float *w, void *d_y,
                       float *d_w, hipStream_t s) {
    dim3 grid(1, 1, 1);
    const Span sp = make_span(g.T, D / V, true, grid);
    hipLaunchKernelGGL((combine_backward_kernel<TY, TO, V>), grid, dim3(kThreads), 0, s, g.T, g.top_k, sp, g.slot_pos,
                       w, static_cast<const TO *>(d_out), static_cast<const TY *>(y), static_cast<TY *>(d_y), d_w);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gather(const moe_groups &g, int32_t dtype, int32_t D, const void *x, void *rows, hipStream_t s) {
    return dtype == MOE_DT_BF16 ? gather<Bf16>(g, D, x, rows, s) : gather<float>(g, D, x, rows, s);
}

// A piece holds as many elements as 16 bytes of the narrower type that is involved, so that
// bf16 rows move 16 bytes at a time; fp32 rows beside them move two such loads or stores.
#define MOE_BY_TYPES(FN, ...)                                                                            \
    do {                                                                                                 \
        if (y_dtype == MOE_DT_BF16 && out_dtype == MOE_DT_BF16)                                          \
            return D % 8 ? FN<Bf16, Bf16, 1>(__VA_ARGS__) : FN<Bf16, Bf16, 8>(__VA_ARGS__);              \
        if (y_dtype == MOE_DT_BF16) return D % 8 ? FN<Bf16, float, 1>(__VA_ARGS__) : FN<Bf16, float, 8>(__VA_ARGS__); \
        if (out_dtype == MOE_DT_BF16) return D % 8 ? FN<float, Bf16, 1>(__VA_ARGS__) : FN<float, Bf16, 8>(__VA_ARGS__); \
        return D % 4 ? FN<float, float, 1>(__VA_ARGS__) : FN<float, float, 4>(__VA_ARGS__);              \
    } while (0)

hipError_t launch_combine_rows(const moe_groups &g, int32_t y_dtype, int32_t out_dtype, int32_t D, const void *y,
                               const float *w, void *out, hipStream_t s) {
    MOE_BY_TYPES(join, g, D, y, w, out, s);
}

hipError_t launch_combine_backward(const moe_groups &g, int32_t y_dtype, int32_t out_dtype, int32_t D,
                                   const void *d_out, const void *y, const float *w, void *d_y, float *d_w,
                                   hipStream_t s) {
    MOE_BY_TYPES(spread_back, g, D, d_out, y, w, d_y, d_w, s);
}

}  // namespace moe
