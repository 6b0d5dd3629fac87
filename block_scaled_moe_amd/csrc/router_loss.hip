// router_loss.hip - losses of the router and the gradient of its logits (include/moe_router.h,
// moe_router_losses, moe_logits_grad).
//
//   p[t][e] = exp(l[t][e] - m[t]) / sum over e of the same,  m[t] = max over e (in both: none goes by the rounded lse)
//   P[e] = sum over t of p, N[e] = slots of e;  balance = E / (k n^2) sum of N P,  z = mean of (m + log sum)^2
//   d_l = p (a - <a, p>) + b lse p + gate,  a[e] = d_balance E / (k n^2) N[e],  b = 2 d_z / n
//
// Both are bound by memory: every logit is read once (the gradient writes one fp32 for it), with about ten
// operations each. A token's row stays in the registers of 16, 32 or 64 lanes, four consecutive values a piece,
// so that its maximum and sums are exchanges among them and no value is read twice; the sums over tokens are kept by
// those lanes too, one accumulator per value of a row, over a run of tokens of one sequence. Runs are what
// workgroups take: the losses' leave one line of partial sums each, which a second launch adds in the order of
// the runs; there are no atomics on values.
//
// Medians: 131072 x 384 fp32 logits, one sequence, losses 59 us (201 MB; 45 where they lie in the last-level cache) and 7.4 us to join
// the runs, gradient 75 us (403 MB, 5.4 TB/s of reads and writes). 16384 x 384, eight sequences: 11.8, 6.3 and 16.4 us. Small
// batches: 4 us a kernel, of which a launch is most.
#include "router_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kGradThreads = 256;
constexpr float kNegInf = -__builtin_inff();

// exp(x) within about two units of the last place, x <= 0: 2^(x log2 e), the product's rounding error put back
__device__ __forceinline__ float exp_neg(float x) {
    constexpr float kLog2e = 1.44269504088896341f, kLog2eLow = 1.92596299112661746e-8f, kLn2 = 0.693147180559945309f;
    const float t = x * kLog2e;
    // where 2^t is 0 the error may be an infinity or a NaN
    const float r = fminf(fmaxf(fmaf(x, kLog2e, -t) + x * kLog2eLow, -1.0f), 1.0f);
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, r * kLn2, e);
}

// m + log(sum), rounded once: a logarithm of several units would add a rounding of its own
__device__ __forceinline__ float log_sum_exp(float m, float sum) {
    constexpr double kLn2 = 0.693147180559945309;
    int k;
    const float f = frexpf(sum, &k);
    return (float)((double)m + fma((double)k, kLn2, (double)logf(f)));
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
    return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
    return v;
}

// Piece of four consecutive values of a row, fp32 whatever the type; `whole`: E % 4 == 0 (rows then start on 8 or 16 bytes)
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint16_t h4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ float wide(float v) { return v; }
__device__ __forceinline__ float wide(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
template <typename T>
__device__ __forceinline__ f4 load_piece(const T *row, int e, int E, bool whole) {
    f4 v = {kNegInf, kNegInf, kNegInf, kNegInf};
    if (whole) {
        if (e < E) {
            if constexpr (sizeof(T) == 4) {
                v = *reinterpret_cast<const f4 *>(row + e);
            } else {
                const h4 u = *reinterpret_cast<const h4 *>(row + e);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = wide(u[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e + i < E) v[i] = wide(row[e + i]);
    }
    return v;
}

// Tokens row0 .. row1 - 1 of sequence s, or (s = -1 or B) of those before the first one or behind the last: run `run` of the batch.
// false: there is no such run.
struct Run {
    int32_t s, row0, row1;
};
// First token of sequence s of -1 .. B + 1, the outer ones being the tokens in none and the end.
__device__ __forceinline__ int32_t start_of(const int32_t *seq, int32_t s, int32_t T, int32_t B) {
    return s < 0 ? 0 : s > B ? T : min(max(seq[s], 0), T);
}
__device__ __forceinline__ bool find_run(const int32_t *seq, int32_t T, int32_t B, int32_t log_rows, int64_t run, Run &r) {
    int32_t lo = 0, hi = T;
    r.s = 0;
    if (seq) {
        // the last sequence whose first run is not behind `run`: a wave's lanes look at 64 of them at a time
        int32_t a = 0, n = B + 2;  // numbered from -1 on
        for (;;) {
            const int32_t step = (n + 63) / 64, at = a + (threadIdx.x & 63) * step;
            const bool before = at < a + n && (int64_t)(start_of(seq, min(at, B + 1) - 1, T, B) >> log_rows) + at <= run;
            const int32_t last = max(__popcll(__ballot(before)), 1) - 1;
            a += last * step;
            if (step == 1) break;
            n = min(step, n - last * step);
        }
        a = __builtin_amdgcn_readfirstlane(a);
        r.s = a - 1;
        lo = start_of(seq, r.s, T, B);
        hi = start_of(seq, r.s + 1, T, B);
        run -= a;
    }
    const int64_t first = (int64_t)lo + ((run - (lo >> log_rows)) << log_rows);
    if (first < lo || first >= hi) return false;
    r.row0 = (int32_t)first;
    r.row1 = (int32_t)min((int64_t)hi, first + (1 << log_rows));
    return true;
}

struct LossArgs {
    moe_losses l;
    int32_t log_rows, whole;
    const void *logits;
    const int32_t *topk_idx;
    const uint8_t *valid;
    float *sums;        // [run][E]
    int32_t *counts;    // [run][E]
    double *squares;    // [run]
    int32_t *tokens;    // [run]
    double *parts;      // [B][workgroups] of the balance loss
    uint32_t *arrived;  // [B] workgroups that have left their part
};

// L lanes a token, NP pieces of four values a lane. ONE: the only run there is; it leaves the losses themselves.
template <typename T, int L, int NP, bool ONE>
__global__ void __launch_bounds__(kThreads) loss_kernel(const LossArgs a) {
    constexpr int kRow = L * NP * 4;
    __shared__ float sums[kWaves][kRow];
    __shared__ int32_t hist[kRow];
    __shared__ double squares[kThreads / L];
    __shared__ int32_t tokens[kThreads / L];
    __shared__ double total[kWaves];
    const int t = threadIdx.x, lane = t % L, group = t / L;
    const int E = a.l.E, k = a.l.top_k;
    if (!ONE && t == 0 && (int)blockIdx.x < a.l.B) a.arrived[blockIdx.x] = 0;
    Run r = {0, 0, a.l.T};
    if constexpr (ONE) {
        if (a.l.seq) r = {0, start_of(a.l.seq, 0, a.l.T, 1), start_of(a.l.seq, 1, a.l.T, 1)};
        for (int row = t; row < a.l.T; row += kThreads)
            if (row < r.row0 || row >= r.row1) a.l.lse[row] = kNegInf;
    } else {
        if (!find_run(a.l.seq, a.l.T, a.l.B, a.log_rows, blockIdx.x, r)) return;
        if (r.s < 0 || r.s == a.l.B) {  // in no sequence
            for (int row = r.row0 + t; row < r.row1; row += kThreads) a.l.lse[row] = kNegInf;
            return;
        }
    }
    f4 acc[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) acc[p] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
    double square = 0.0;
    int32_t n = 0;
    const T *logits = static_cast<const T *>(a.logits);
    struct Row {
        f4 v[NP];
        int32_t idx;
        bool valid;
    };
    auto load = [&](int row, Row &x) __attribute__((always_inline)) {
        if (row >= r.row1) return;
        x.valid = !a.valid || a.valid[row] != 0;
        x.idx = lane < k ? a.topk_idx[(int64_t)row * k + lane] : -1;
#pragma unroll
        for (int p = 0; p < NP; ++p) x.v[p] = load_piece(logits + (int64_t)row * E, 4 * (p * L + lane), E, a.whole);
    };
    Row next;
    load(r.row0 + group, next);
    for (int e = t; e < kRow; e += kThreads) hist[e] = 0;
    __syncthreads();
    for (int row = r.row0 + group; row < r.row1; row += kThreads / L) {
        const Row x = next;
        load(row + kThreads / L, next);
        float m = kNegInf;
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, x.v[p][i]);
        m = lanes_max<L>(m);
        if (m == kNegInf) m = 0.0f;  // nothing above -inf: the sum is 0, or a NaN
        f4 ex[NP];
        f4 four = {0.0f, 0.0f, 0.0f, 0.0f};  // four chains: shorter ones round less
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i) four[i] += ex[p][i] = exp_neg(x.v[p][i] - m);
        const float sum = lanes_sum<L>((four[0] + four[1]) + (four[2] + four[3]));
        const bool counted = x.valid && sum != 0.0f;
        const float lse = counted ? log_sum_exp(m, sum) : kNegInf;
        if (lane == 0) a.l.lse[row] = lse;
        if (counted) {
            const float inv = 1.0f / sum;
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[p][i] = fmaf(ex[p][i], inv, acc[p][i]);
            square = fma((double)lse, (double)lse, square);
            ++n;
            if ((uint32_t)x.idx < (uint32_t)E) atomicAdd(&hist[x.idx], 1);
        }
    }
    // the tokens of a wave, then its place in LDS
#pragma unroll
    for (int p = 0; p < NP; ++p) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int off = L; off < 64; off <<= 1) acc[p][i] += __shfl_xor(acc[p][i], off);
        if (t % 64 < L) *reinterpret_cast<f4 *>(&sums[t / 64][4 * (p * L + lane)]) = acc[p];
    }
    if (lane == 0) {
        squares[group] = square;
        tokens[group] = n;
    }
    __syncthreads();
    double part = 0.0;
    for (int e = t; e < E; e += kThreads) {
        float s = sums[0][e];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += sums[w][e];
        if constexpr (ONE) {
            a.l.prob_sums[e] = s;
            a.l.counts[e] = hist[e];
            part += (double)s * hist[e];
        } else {
            a.sums[(int64_t)blockIdx.x * E + e] = s;
            a.counts[(int64_t)blockIdx.x * E + e] = hist[e];
        }
    }
    if constexpr (ONE) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) part += __shfl_xor(part, off);
        if (t % 64 == 0) total[t / 64] = part;
        __syncthreads();
    }
    if (t == 0) {
        double s = 0.0;
        int32_t c = 0;
        for (int g = 0; g < kThreads / L; ++g) {
            s += squares[g];
            c += tokens[g];
        }
        if constexpr (ONE) {
            double b = 0.0;
            for (int w = 0; w < kWaves; ++w) b += total[w];
            a.l.tokens[0] = c;
            a.l.z[0] = c ? (float)(s / c) : 0.0f;
            a.l.balance[0] = c ? (float)(b * E / ((double)k * c * c)) : 0.0f;
        } else {
            a.squares[blockIdx.x] = s;
            a.tokens[blockIdx.x] = c;
        }
    }
}

// The sums of 64 experts of one sequence over its runs, a run a wave. Where that is not all of them, the workgroup that comes last
// for a sequence adds the parts of its balance loss, in the order of the experts. (16 experts a workgroup, four runs a wave, read the
// runs in fewer turns, but more of them meet: 16384 x 384 in eight sequences 17.9 us for the losses, so 15.5; 5003 x 61 in 17 11.0
// and 8.8; 131072 x 384 in one 40.9 and 41.4; 2000 x 16 in one 7.9 and 8.2.)
constexpr int kJoinThreads = 1024, kJoinWaves = kJoinThreads / 64, kJoinExperts = 64;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const LossArgs a) {
    __shared__ double sum[kJoinWaves][kJoinExperts];
    __shared__ int32_t count[kJoinWaves][kJoinExperts];
    __shared__ double squares[kJoinWaves];
    __shared__ int32_t tokens[kJoinWaves];
    const int E = a.l.E, ne = (E + kJoinExperts - 1) / kJoinExperts;
    const int s = blockIdx.x / ne, eb = blockIdx.x % ne, t = threadIdx.x;
    const int e = eb * kJoinExperts + t % 64;
    int32_t lo = 0, hi = a.l.T;
    int64_t first = 0;
    if (a.l.seq) {
        lo = start_of(a.l.seq, s, a.l.T, a.l.B);
        hi = start_of(a.l.seq, s + 1, a.l.T, a.l.B);
        first = (lo >> a.log_rows) + s + 1;
    }
    const int n = hi > lo ? (hi - lo + (1 << a.log_rows) - 1) >> a.log_rows : 0;
    double p = 0.0, z = 0.0;
    int32_t c = 0, m = 0;
    if (e < E) {
#pragma unroll 8
        for (int i = t / 64; i < n; i += kJoinWaves) {
            p += a.sums[(first + i) * E + e];
            c += a.counts[(first + i) * E + e];
        }
    }
    for (int i = t; i < n; i += kJoinThreads) {
        z += a.squares[first + i];
        m += a.tokens[first + i];
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        z += __shfl_xor(z, off);
        m += __shfl_xor(m, off);
    }
    sum[t / 64][t % 64] = p;
    count[t / 64][t % 64] = c;
    if (t % 64 == 0) {
        squares[t / 64] = z;
        tokens[t / 64] = m;
    }
    __syncthreads();
    if (t >= 64) return;
    double part = 0.0;
    if (e < E) {
        p = sum[0][t];
        c = count[0][t];
#pragma unroll
        for (int i = 1; i < kJoinWaves; ++i) {
            p += sum[i][t];
            c += count[i][t];
        }
        a.l.prob_sums[(int64_t)s * E + e] = (float)p;
        a.l.counts[(int64_t)s * E + e] = c;
        part = p * c;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) part += __shfl_xor(part, off);
    if (t != 0) return;
    for (int i = 1; i < kJoinWaves; ++i) {
        z += squares[i];
        m += tokens[i];
    }
    if (eb == 0) {
        a.l.tokens[s] = m;
        a.l.z[s] = m ? (float)(z / m) : 0.0f;
    }
    if (ne > 1) {
        double *parts = a.parts + (int64_t)s * ne;
        __hip_atomic_store(parts + eb, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint32_t before = __hip_atomic_fetch_add(a.arrived + s, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        if (before + 1 != (uint32_t)ne) return;
        part = 0.0;
#pragma unroll 8
        for (int i = 0; i < ne; ++i) part += __hip_atomic_load(parts + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    a.l.balance[s] = m ? (float)(part * E / ((double)a.l.top_k * m * m)) : 0.0f;
}

// ---------------------------------------------------------------- gradient of the logits

struct GradArgs {
    moe_logits_grad_args a;
    moe_losses l;
    int32_t log_rows, whole;
    int32_t all;  // rows of tokens in no sequence too
};

// LOSS: the gradients of the losses; GATE: those of the gate's weights, put into their places of a row in LDS, from where the
// row's lanes add them: the places are written anew for each token and cleared behind it.
template <typename T, int L, int NP, bool LOSS, bool GATE>
__global__ void __launch_bounds__(kGradThreads) logits_grad_kernel(const GradArgs g) {
    constexpr int kRow = L * NP * 4, kGroups = kGradThreads / L;
    __shared__ __attribute__((aligned(16))) float gate[GATE ? kGroups : 1][GATE ? kRow : 4];
    const int t = threadIdx.x, lane = t % L, group = t / L;
    const int E = g.a.E, k = g.a.top_k;
    Run r;
    if (!find_run(LOSS ? g.l.seq : nullptr, g.a.T, LOSS ? g.l.B : 1, g.log_rows, blockIdx.x, r)) return;
    const bool outside = LOSS && (r.s < 0 || r.s == g.l.B);  // in no sequence
    if (outside && !g.all) return;
    if constexpr (GATE) {
#pragma unroll
        for (int p = 0; p < NP; ++p) *reinterpret_cast<f4 *>(&gate[group][4 * (p * L + lane)]) = (f4){0.0f, 0.0f, 0.0f, 0.0f};
    }
    const T *logits = static_cast<const T *>(g.a.logits);
    struct Row {
        f4 v[NP];
        float lse, w, dw;
        int32_t idx;
    };
    auto load = [&](int row, Row &x) __attribute__((always_inline)) {
        if (row >= r.row1) return;
        if constexpr (GATE) {
            const bool slot = lane < k;
            x.idx = slot ? g.a.topk_idx[(int64_t)row * k + lane] : -1;
            x.w = slot ? g.a.topk_w[(int64_t)row * k + lane] : 0.0f;
            x.dw = slot ? g.a.d_topk_w[(int64_t)row * k + lane] : 0.0f;
        }
        if constexpr (LOSS) {
            x.lse = outside ? kNegInf : g.l.lse[row];
#pragma unroll
            for (int p = 0; p < NP; ++p) x.v[p] = load_piece(logits + (int64_t)row * E, 4 * (p * L + lane), E, g.whole);
        }
    };
    Row next;
    load(r.row0 + group, next);
    f4 f[NP];
    float b = 0.0f;
    if constexpr (LOSS) {
        const int32_t n = outside ? 0 : g.l.tokens[r.s];
        float a = 0.0f;
        if (n != 0) {
            if (g.a.d_balance) a = (float)((double)g.a.d_balance[r.s] * E / ((double)k * n * n));
            if (g.a.d_z) b = (float)(2.0 * (double)g.a.d_z[r.s] / n);
        }
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = 4 * (p * L + lane) + i;
                f[p][i] = e < E && g.a.d_balance && !outside ? a * (float)g.l.counts[(int64_t)r.s * E + e] : 0.0f;
            }
    }
    for (int row = r.row0 + group; row < r.row1; row += kGroups) {
        const Row x = next;
        load(row + kGroups, next);
        f4 d[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) d[p] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
        const bool here = GATE && (uint32_t)x.idx < (uint32_t)E;
        if constexpr (GATE) {
            const float w = here ? x.w : 0.0f;
            // the lanes behind top_k (at most eight) add nothing
            const float dot = lanes_sum<8>(here ? w * x.dw : 0.0f);
            const float mine = here ? w * (x.dw - dot) : 0.0f;
            float all = 0.0f;  // over the token's slots of this expert, in their order
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = __shfl(mine, j, L);
                if (__shfl(x.idx, j, L) == x.idx) all += v;
            }
            if (here) gate[group][x.idx] = all;
        }
        if constexpr (LOSS) {
            if (x.lse != kNegInf) {
                // by the row's own maximum and sum, as the losses have them: beside a maximum far from zero, lse has few bits left
                // of the sum's logarithm, or none
                float m = kNegInf;
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int i = 0; i < 4; ++i) m = fmaxf(m, x.v[p][i]);
                m = lanes_max<L>(m);
                float dot = 0.0f;
                f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};  // four chains: shorter ones round less
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d[p][i] = exp_neg(x.v[p][i] - m);
                        sum[i] += d[p][i];
                        dot = fmaf(d[p][i], f[p][i], dot);
                    }
                const float inv = 1.0f / lanes_sum<L>((sum[0] + sum[1]) + (sum[2] + sum[3]));
                dot = lanes_sum<L>(dot) * inv - (g.a.d_z ? b * x.lse : 0.0f);
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[p][i] *= inv * (f[p][i] - dot);
            }
        }
        float *out = g.a.d_logits + (int64_t)row * E;
        if constexpr (GATE) __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int e = 4 * (p * L + lane);
            if constexpr (GATE) d[p] += *reinterpret_cast<const f4 *>(&gate[group][e]);
            if (g.whole) {
                if (e < E) *reinterpret_cast<f4 *>(out + e) = d[p];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (e + i < E) out[e + i] = d[p][i];
            }
        }
        if constexpr (GATE) {
            __builtin_amdgcn_wave_barrier();
            if (here) gate[group][x.idx] = 0.0f;
        }
    }
}

// f is called with the lanes a token and pieces a lane for rows of E values: the fewest lanes that hold a row in at most
// four pieces each, more pieces only where a wave is not enough. Three pieces, so that no quarter of the places is empty, stand only
// at 257 to 384 values.
template <typename F>
void by_row(int32_t E, F &&f) {
    using std::integral_constant;
#define MOE_ROW(L, NP) f(integral_constant<int, L>{}, integral_constant<int, NP>{})
    if (E <= 64) MOE_ROW(16, 1);
    else if (E <= 128) MOE_ROW(16, 2);
    else if (E <= 256) MOE_ROW(16, 4);
    else if (E <= 384) MOE_ROW(32, 3);
    else if (E <= 512) MOE_ROW(32, 4);
    else if (E <= 1024) MOE_ROW(64, 4);
    else if (E <= 2048) MOE_ROW(64, 8);
    else MOE_ROW(64, 16);
#undef MOE_ROW
}
int32_t row_lanes(int32_t E) { return E <= 256 ? 16 : E <= 512 ? 32 : 64; }

}  // namespace

RunSplit run_split(int32_t T, int32_t B, bool seq, int32_t rows_at_least, int32_t runs_at_most) {
    RunSplit r{};
    while ((1 << r.log_rows) < rows_at_least) ++r.log_rows;
    while ((T >> r.log_rows) > runs_at_most) ++r.log_rows;
    r.n = seq ? ((int64_t)T >> r.log_rows) + B + 2 : ((int64_t)T + (1 << r.log_rows) - 1) >> r.log_rows;
    return r;
}

LossPlan loss_plan(int32_t T, int32_t E, int32_t B, bool seq) {
    LossPlan p{};
    p.runs = run_split(T, B, seq, 2 * kThreads / row_lanes(E), 512);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~(size_t)255;
        return at;
    };
    const size_t lines = (size_t)run_split(T, B, true, 1 << p.runs.log_rows, INT32_MAX).n;  // the same with and without seq
    p.sums = take(4 * lines * E);
    p.counts = take(4 * lines * E);
    p.squares = take(8 * lines);
    p.tokens = take(4 * lines);
    p.parts = take(8 * (size_t)B * ((E + kJoinExperts - 1) / kJoinExperts));
    p.arrived = take(4 * (size_t)B);
    p.total = off > 0 ? off : 256;
    return p;
}

hipError_t launch_router_losses(const moe_losses &l, int32_t dtype, const void *logits, const int32_t *topk_idx,
                                const uint8_t *valid, uint8_t *workspace, hipStream_t s) {
    const LossPlan p = loss_plan(l.T, l.E, l.B, l.seq);
    LossArgs a{};
    a.l = l;
    a.log_rows = p.runs.log_rows;
    a.whole = l.E % 4 == 0;
    a.logits = logits;
    a.topk_idx = topk_idx;
    a.valid = valid;
    a.sums = reinterpret_cast<float *>(workspace + p.sums);
    a.counts = reinterpret_cast<int32_t *>(workspace + p.counts);
    a.squares = reinterpret_cast<double *>(workspace + p.squares);
    a.tokens = reinterpret_cast<int32_t *>(workspace + p.tokens);
    a.parts = reinterpret_cast<double *>(workspace + p.parts);
    a.arrived = reinterpret_cast<uint32_t *>(workspace + p.arrived);
    const bool one = l.B == 1 && l.T <= 1 << p.runs.log_rows;
    by_row(l.E, [&](auto L, auto NP) {
        constexpr int kL = decltype(L)::value, kNP = decltype(NP)::value;
        auto go = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)(one ? 1 : p.runs.n)), dim3(kThreads), 0, s, a);
        };
        if (dtype == MOE_DT_BF16) {
            if (one) go(loss_kernel<uint16_t, kL, kNP, true>);
            else go(loss_kernel<uint16_t, kL, kNP, false>);
        } else {
            if (one) go(loss_kernel<float, kL, kNP, true>);
            else go(loss_kernel<float, kL, kNP, false>);
        }
    });
    if (!one) {
        const unsigned groups = (unsigned)(l.B * ((l.E + kJoinExperts - 1) / kJoinExperts));
        hipLaunchKernelGGL(join_kernel, dim3(groups), dim3(kJoinThreads), 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_logits_grad(const moe_logits_grad_args &args, bool all, hipStream_t s) {
    const int32_t B = args.l ? args.l->B : 1;
    const RunSplit runs = run_split(args.T, B, args.l && args.l->seq, kGradThreads / row_lanes(args.E), 1024);
    GradArgs g{};
    g.a = args;
    if (args.l) g.l = *args.l;
    g.all = all;
    g.log_rows = runs.log_rows;
    g.whole = args.E % 4 == 0;
    by_row(args.E, [&](auto L, auto NP) {
        constexpr int kL = decltype(L)::value, kNP = decltype(NP)::value;
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)runs.n), dim3(kGradThreads), 0, s, g); };
        auto typed = [&](auto zero) {
            using T = decltype(zero);
            if (args.topk_w) go(logits_grad_kernel<T, kL, kNP, true, true>);
            else go(logits_grad_kernel<T, kL, kNP, true, false>);
        };
        if (!args.l) go(logits_grad_kernel<float, kL, kNP, false, true>);
        else if (args.dtype == MOE_DT_BF16) typed((uint16_t)0);
        else typed(0.0f);
    });
    return hipGetLastError();
}

}  // namespace moe
