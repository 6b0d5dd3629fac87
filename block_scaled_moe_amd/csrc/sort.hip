// sort.hip - the stable counting sort behind moe_sort (include/moe_ops.h): slots by expert and
// by slot, each expert's first row, and the work lists of the grouped products.
//
// Bound by latency, not by bytes (65536 slots are 0.8 MB): so it has as few dependent steps as it
// can. Up to kSingle slots one workgroup of 16 waves does it all; beyond, a first launch counts
// each chunk of slots by expert, and in a second each chunk's workgroup adds up the counts of all
// chunks for itself (which gives it the experts' first rows and its own places in them) and places
// its slots, 1024 at a time: a lane's rank among the 64 slots of its wave comes from one ballot per
// bit of the expert number, its wave's place from the 16 waves' counts in LDS. The order of the
// slots alone decides every position. Up to 1024 local experts; permute.hip takes more. Kernel times with
// 384 experts: 8 slots 4.5 us, 4096 11 us (one launch), 65536 15 us, 131072 20 us (two); permute.hip's with
// 4096 experts and 16384 slots 160 us.
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kCountThreads = 256;
constexpr int32_t kSingle = 4096;    // slots of the one-workgroup sort
constexpr int32_t kMaxChunks = 256;  // each chunk's workgroup reads every chunk's counts

__device__ __forceinline__ int local_expert(const PermuteArgs &a, int64_t s, int64_t end) {
    if (s >= end) return -1;
    const uint32_t e = (uint32_t)a.idx[s] - (uint32_t)a.e_begin;  // wraps past n_loc for any other value
    return e < (uint32_t)a.n_loc ? (int)e : -1;
}

__global__ void __launch_bounds__(kCountThreads) sort_count_kernel(const PermuteArgs a, int32_t n_slots, int32_t chunk) {
    extern __shared__ int32_t cnt[];
    for (int i = threadIdx.x; i < a.n_loc; i += kCountThreads) cnt[i] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * chunk, s1 = min<int64_t>(s0 + chunk, n_slots);
    for (int64_t s = s0 + threadIdx.x; s < s1; s += kCountThreads) {
        const int e = local_expert(a, s, s1);
        if (e >= 0) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    int32_t *dst = a.chunk_counts + (int64_t)blockIdx.x * a.n_loc;
    for (int i = threadIdx.x; i < a.n_loc; i += kCountThreads) dst[i] = cnt[i];
}

// Inclusive sum of v over the lanes of a wave.
__device__ __forceinline__ int wave_sum(int v, int lane) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int other = __shfl_up(v, off);
        v += lane >= off ? other : 0;
    }
    return v;
}

__global__ void __launch_bounds__(kThreads) sort_place_kernel(const PermuteArgs a, int32_t n_slots, int32_t chunk) {
    extern __shared__ int32_t lds[];
    const int n = a.n_loc, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int32_t *tot = lds, *base = lds + n;                          // [n] slots of each expert; next place in it
    uint16_t *hist = reinterpret_cast<uint16_t *>(lds + 2 * n);  // [16][n] slots of each wave of 1024
    __shared__ int32_t part[2][kWaves];
    const int64_t s0 = (int64_t)blockIdx.x * chunk, s1 = min<int64_t>(s0 + chunk, n_slots);
    if (tid < n) {
        tot[tid] = 0;
        base[tid] = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) hist[w * n + tid] = 0;
    }
    __syncthreads();
    if (gridDim.x == 1) {
        for (int64_t s = tid; s < s1; s += kThreads) {
            const int e = local_expert(a, s, s1);
            if (e >= 0) atomicAdd(&tot[e], 1);
        }
    } else {  // runs of chunks, each summed by one thread per expert
        const int segs = kThreads / n, chunks = gridDim.x, len = (chunks + segs - 1) / segs;
        if (tid < n * segs) {
            const int e = tid % n, c0 = tid / n * len, c1 = min(c0 + len, chunks);
            int all = 0, before = 0;
#pragma unroll 16
            for (int c = c0; c < c1; ++c) {
                const int v = a.chunk_counts[(int64_t)c * n + e];
                all += v;
                before += c < (int)blockIdx.x ? v : 0;
            }
            if (c0 < c1) {
                atomicAdd(&tot[e], all);
                atomicAdd(&base[e], before);
            }
        }
    }
    __syncthreads();
    // exclusive sums over the experts: first rows, and first tiles of the work list
    const int mine = tid < n ? tot[tid] : 0, my_tiles = (mine + a.bm - 1) / a.bm;
    const int sum = wave_sum(mine, lane), tiles = wave_sum(my_tiles, lane);
    if (lane == 63) {
        part[0][wave] = sum;
        part[1][wave] = tiles;
    }
    __syncthreads();
    int before = 0, tiles_before = 0, S = 0, n_tiles = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) {
            before += part[0][w];
            tiles_before += part[1][w];
        }
        S += part[0][w];
        n_tiles += part[1][w];
    }
    const int first = before + sum - mine, t0 = tiles_before + tiles - my_tiles;
    if (tid < n) {
        base[tid] += first;
        if (blockIdx.x == 0) {
            a.counts[tid] = mine;
            a.offsets[tid] = first;
            for (int i = 0; i < my_tiles; ++i) {
                a.tile_expert[t0 + i] = tid;
                a.tile_row0[t0 + i] = first + i * a.bm;
            }
        }
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.offsets[n] = S;
        a.ctrl->S = S;
        a.ctrl->n_tiles = n_tiles;
    }
    const int bits = n > 1 ? 32 - __clz(n - 1) : 0;
    for (int64_t p = s0; p < s1; p += kThreads) {
        const int64_t s = p + tid;
        const int e = local_expert(a, s, s1);
        // the lanes of this wave with the same expert
        uint64_t same = __ballot(e >= 0);
        for (int b = 0; b < bits; ++b) {
            const bool set = (e >> b) & 1;
            const uint64_t m = __ballot(set);
            same &= set ? m : ~m;
        }
        const int rank = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0u));
        if (e >= 0 && rank == 0) hist[wave * n + e] = (uint16_t)__popcll(same);
        __syncthreads();
        int run = 0;
        if (tid < n) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const int c = hist[w * n + tid];
                hist[w * n + tid] = (uint16_t)run;
                run += c;
            }
        }
        __syncthreads();
        if (e >= 0) {
            const int pos = base[e] + hist[wave * n + e] + rank;
            a.sorted_slot[pos] = (int32_t)s;
            a.slot_pos[s] = pos;
        } else if (s < s1) {
            a.slot_pos[s] = -1;
        }
        if (p + kThreads < s1) {
            __syncthreads();
            if (tid < n) {
                base[tid] += run;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) hist[w * n + tid] = 0;
            }
            __syncthreads();
        }
    }
    // this chunk's share of the places behind the last local slot
    for (int64_t p = max<int64_t>(s0, S) + tid; p < s1; p += kThreads) a.sorted_slot[p] = -1;
}

}  // namespace

int32_t sort_chunk_slots(int64_t n_slots) {
    if (n_slots <= kSingle) return kSingle;
    const int64_t per = (n_slots + kMaxChunks - 1) / kMaxChunks;
    return (int32_t)((per + kThreads - 1) / kThreads * kThreads);
}

hipError_t launch_sort(const PermuteArgs &a, int32_t n_slots, hipStream_t s) {
    const int32_t chunk = sort_chunk_slots(n_slots);
    const int chunks = n_slots > 0 ? (int)(((int64_t)n_slots + chunk - 1) / chunk) : 1;
    if (chunks > 1) {
        hipLaunchKernelGGL(sort_count_kernel, dim3(chunks), dim3(kCountThreads), sizeof(int32_t) * (size_t)a.n_loc, s, a,
                           n_slots, chunk);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    const size_t lds = (size_t)a.n_loc * (2 * sizeof(int32_t) + kWaves * sizeof(uint16_t));
    hipLaunchKernelGGL(sort_place_kernel, dim3(chunks), dim3(kThreads), lds, s, a, n_slots, chunk);
    return hipGetLastError();
}

}  // namespace moe
