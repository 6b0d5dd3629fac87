// router_grad.hip - gradients of the router's product (include/moe_router.h, moe_route_backward).
//
//   dh[t][d] = sum over e of g[t][e] wr[e][d],  dwr[e][d] = sum over t of g[t][e] h[t][d],  dbias[e] = sum over t of g
//
// Both are products of a fp32 matrix with a bf16 one whose rows run along the reduction, so one kernel does both. The
// fp32 one, which is the smaller, goes through the bf16 MFMA in pieces: its value is the sum of its upper 8 bits, the next 8
// and the last 8, each a bf16 exactly. All three are needed for bf16 results too: a row of g sums to nearly nothing, so what
// the experts' weights have in common cancels, and the leading bits with it. Where many column tiles share it, split_kernel cuts
// it once into the order in which the MFMA takes it, for either product: tiles of 128 rows, steps of 32 of the reduction,
// pieces, 16 rows, lanes; a tile's step is one contiguous copy. Where few do, a launch costs more than cutting it in every workgroup.
//
// product_kernel: BM rows x 256 columns a workgroup of 4 waves, two workgroups a CU, a step of 32 of the reduction in one LDS
// buffer while the next one arrives in the other. The bf16 matrix comes as it is and is turned over by the transposing
// LDS read (4 rows x 16 columns per 16 lanes), the same operand for all pieces.
//
// Bound by the MFMAs where they are many: 16384 x 384, 4096 columns, bf16 results: split 23 us, both products 268 (309 GFLOP of
// pieces, 1.15 PFLOP/s; 231 and 1.34 at best, the matrix cores then busy 62% of the cycles), joining dwr's parts 7.8; two pieces took 190
// for results up to 2^-15 of each value of g off. 5003 x 61, 1088 columns, fp32 results with the bias's: 19.1 and 4.0 us. 300 x 64,
// 256 columns: 13.3 us, ten steps' latency one behind the other and the launch.
#include "block_mma.h"
#include "router_internal.h"

#include <type_traits>

namespace moe {
namespace {

using namespace block;

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kBM = 128, kFusedBM = 64, kBN = 256, kStep = 32;

// v in pieces of bf16: cut off at 8 bits each, which nothing can overflow
constexpr int kPieces = 3;
__device__ __forceinline__ void split(float v, uint16_t (&out)[kPieces]) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const uint32_t u = __float_as_uint(v) & 0xFFFF0000u;
        out[p] = (uint16_t)(u >> 16);
        v -= __uint_as_float(u);
    }
}

// One lane's operand of a 16 x 32 piece: row r of 16, values k = 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3; the pieces lie
// `stride` operands apart.
__device__ __forceinline__ void write_operand(const float (&v)[8], u32x4 *dst, int lane, int stride = 8) {
    uint16_t x[8][kPieces];
#pragma unroll
    for (int i = 0; i < 8; ++i) split(v[i], x[i]);
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = (uint32_t)x[2 * i][p] | (uint32_t)x[2 * i + 1][p] << 16;
        dst[p * stride * 64 + lane] = o;
    }
}

// A block of 128 tokens x 32 experts of g: its operands with tokens as rows (dh), and with experts as rows (dwr).
// Both forms are filled up with zeros to whole tiles and steps.
template <bool H, bool W>
__global__ void __launch_bounds__(kThreads) split_kernel(const float *__restrict__ g, int32_t T, int32_t E, int32_t e_steps,
                                                         int32_t t_steps, u32x4 *__restrict__ a_h, u32x4 *__restrict__ a_w) {
    __shared__ float v[128][33];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, i16 = lane & 15, q = lane >> 4;
    const int t0 = blockIdx.x * 128, e0 = blockIdx.y * 32;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = (t >> 5) + 8 * i, c = t & 31;
        v[r][c] = t0 + r < T && e0 + c < E ? g[(int64_t)(t0 + r) * E + e0 + c] : 0.0f;
    }
    __syncthreads();
    if constexpr (H) {
        if (e0 / 32 < e_steps) {
            u32x4 *tile = a_h + ((int64_t)blockIdx.x * e_steps + blockIdx.y) * (kPieces * 512);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int m = wave + 4 * j;  // 16 tokens
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = v[16 * m + i16][(i >> 2) * 16 + 4 * q + (i & 3)];
                write_operand(x, tile + m * 64, lane);
            }
        }
    }
    if constexpr (W) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int m = 2 * (blockIdx.y & 3) + j;            // 16 experts of the tile
            const int step = blockIdx.x * 4 + wave;            // 32 tokens
            if (step < t_steps) {
                u32x4 *tile = a_w + ((int64_t)(blockIdx.y >> 2) * t_steps + step) * (kPieces * 512);
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = v[32 * wave + (i >> 2) * 16 + 4 * q + (i & 3)][16 * j + i16];
                write_operand(x, tile + m * 64, lane);
            }
        }
    }
}

// One product: out[m][n] = sum over k of a[m][k] b[k][n], M x D, K of the reduction.
struct Product {
    const u32x4 *a;         // operands, tiles x steps; or (not cut beforehand) NULL
    const uint16_t *b;      // bf16 [K][D]
    void *out;              // [M][D] of out_dtype, or fp32 [splits][M][D]
    float *bias;            // fp32 [splits][M] sums of a's rows, or NULL
    int32_t M, K, out_dtype;
    int32_t m_tiles, steps, splits, steps_per_split;
};
struct ProductArgs {
    Product w, h;
    const float *g;
    int32_t T, E, D, n_tiles;
    int32_t w_items, h_items;
};

// OUTER: a's rows run along g's columns (dwr); CUT: a was cut beforehand
template <int BM, bool OUTER, bool CUT>
__device__ __forceinline__ void product(const ProductArgs &args, const Product &p, int item, uint8_t *lds) {
    constexpr int kSub = BM / 16;                        // pieces of 16 rows
    constexpr int kWM = BM / 64, kJ = 16 / (4 / kWM);    // row waves; column tiles of 16 a wave
    constexpr int kA = kPieces * kSub * 1024, kB = kStep * kBN * 2, kBuffer = kA + kB;
    static_assert(!CUT || BM == kBM, "tiles of split_kernel");
    const int D = args.D, n_tiles = args.n_tiles, T = args.T, E = args.E;
    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const int i16 = lane & 15, g = lane >> 4, wm = wave / (4 / kWM), wn = wave % (4 / kWM);
    // items of one part of the reduction together, its row tiles innermost: they share b's columns
    const int part = item / (p.m_tiles * n_tiles), rest = item % (p.m_tiles * n_tiles);
    int mt, nt;
    if (p.splits > 1 || p.m_tiles < n_tiles) {
        mt = rest % p.m_tiles;
        nt = rest / p.m_tiles;
    } else {
        mt = rest / n_tiles;
        nt = rest % n_tiles;
    }
    const int s0 = part * p.steps_per_split, s1 = min(s0 + p.steps_per_split, p.steps);
    const int n0 = nt * kBN;
    const u32x4 *a = CUT ? p.a + (int64_t)mt * p.steps * (kA / 16) : nullptr;
    const uint32_t base = lds_address(lds) + wave * 1024;

    // copy c of 16 of b's step: rows 2 c and 2 c + 1 of 512 bytes; the 32-byte pieces of a row are swapped by the row's
    // last three bits, so that eight rows' pieces of one column lie in different banks
    uint32_t b_col;
    {
        const int q = lane & 31, r = (2 * wave + (lane >> 5)) & 7;  // of copies wave + 4 j: the same r for all
        const int col = ((((q >> 1) ^ r) << 1) | (q & 1)) * 8;
        b_col = (uint32_t)min(n0 + col, D - 8) * 2;
    }
    auto copy = [&](int s) __attribute__((always_inline)) {
        const uint32_t dst = base + (s & 1) * kBuffer;
        if constexpr (CUT) {
            const uint8_t *src = reinterpret_cast<const uint8_t *>(a + (int64_t)s * (kA / 16));
#pragma unroll
            for (int j = 0; j < kPieces * kSub / 4; ++j) copy_to_lds(src + (wave + 4 * j) * 1024, lane * 16, dst + j * 4096);
        }
        const uint8_t *rows = reinterpret_cast<const uint8_t *>(p.b) + (int64_t)s * kStep * D * 2;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = min(2 * (wave + 4 * j) + (lane >> 5), p.K - 1 - s * kStep);  // rows past the end meet zeros
            copy_to_lds(rows, (uint32_t)r * (uint32_t)D * 2 + b_col, dst + kA + j * 4096);
        }
    };
    // not cut beforehand: the operands that this lane writes, of rows 16 (wave + 4 i) + i16
    constexpr int kOwn = CUT ? 1 : kSub / 4;
    float v[kOwn][8];
    auto load = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int m = mt * BM + 16 * (wave + 4 * i) + i16;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = s * kStep + (j >> 2) * 16 + 4 * g + (j & 3);
                const int row = OUTER ? k : m, col = OUTER ? m : k;
                v[i][j] = row < T && col < E ? args.g[(int64_t)row * E + col] : 0.0f;
            }
        }
    };

    f4 acc[4][kJ];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j) acc[i][j] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
    f4 bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
    const bool want_bias = OUTER && p.bias && nt == 0 && wn == 0;

    if (s0 < s1) {
        copy(s0);
        if constexpr (!CUT) load(s0);
    }
    for (int s = s0; s < s1; ++s) {
        uint8_t *buf = lds + (s & 1) * kBuffer;
        if constexpr (!CUT) {
#pragma unroll
            for (int i = 0; i < kOwn; ++i) write_operand(v[i], reinterpret_cast<u32x4 *>(buf) + (wave + 4 * i) * 64, lane, kSub);
        }
        wait_copies<0>();
        lds_barrier();
        if (s + 1 < s1) {
            copy(s + 1);
            if constexpr (!CUT) load(s + 1);
        }
        bf8 x[kPieces][4];
#pragma unroll
        for (int q = 0; q < kPieces; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[q][i] = __builtin_bit_cast(bf8, *reinterpret_cast<const u32x4 *>(buf + (q * kSub + 4 * wm + i) * 1024 + lane * 16));
        const int r = 4 * g + (i16 >> 2);
        const uint8_t *row = buf + kA + r * 512 + (i16 & 3) * 8;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const uint8_t *at = row + ((kJ * wn + j) ^ (r & 7)) * 32;
            const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4 *)at);
            const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4 *)(at + 16 * 512));
            const bf8 y = __builtin_bit_cast(bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
            for (int q = 0; q < kPieces; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y, x[q][i], acc[i][j], 0, 0, 0);
        }
        if (want_bias) {
            const bf8 one = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
#pragma unroll
            for (int q = 0; q < kPieces; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) bias[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(one, x[q][i], bias[i], 0, 0, 0);
        }
    }

    // accumulator v of (i, j): row 16 i + i16, column 16 j + 4 g + v of the wave's
    const bool narrow = p.splits == 1 && p.out_dtype == MOE_DT_BF16;
    const int c0 = n0 + 16 * kJ * wn;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = mt * BM + 64 * wm + 16 * i + i16;
        if (want_bias && g == 0 && m < p.M) p.bias[(int64_t)part * p.M + m] = bias[i][0];
        const int64_t at = ((int64_t)part * p.M + m) * D + c0;
        if (narrow) {
            uint16_t *o = static_cast<uint16_t *>(p.out) + at;
#pragma unroll
            for (int j = 0; j < kJ; j += 2) {
                const uint2 c = make_uint2(bf16_pair(acc[i][j][0], acc[i][j][1]), bf16_pair(acc[i][j][2], acc[i][j][3]));
                const uint2 d = make_uint2(bf16_pair(acc[i][j + 1][0], acc[i][j + 1][1]), bf16_pair(acc[i][j + 1][2], acc[i][j + 1][3]));
                const u32x4 v = swap_groups(c, d);
                const int col = 16 * (j + (g & 1)) + 8 * (g >> 1);
                if (m < p.M && c0 + col < D) *reinterpret_cast<u32x4 *>(o + col) = v;
            }
        } else {
            float *o = static_cast<float *>(p.out) + at;
#pragma unroll
            for (int j = 0; j < kJ; ++j)
                if (m < p.M && c0 + 16 * j < D) *reinterpret_cast<f4 *>(o + 16 * j + 4 * g) = acc[i][j];
        }
    }
}

template <bool H, bool W, bool CUT>
__global__ void __launch_bounds__(kThreads, 2) product_kernel(const ProductArgs a) {
    constexpr int BM = CUT ? kBM : kFusedBM;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * (kPieces * BM * 64 + kStep * kBN * 2)];
    // each XCD (workgroups 8 apart) takes a range of either product's items
    auto mine = [](int b, int items) __attribute__((always_inline)) {
        const int per = (items + 7) / 8, x = b & 7, i = b >> 3;
        const int at = x * per + i;
        return i < per && at < items ? at : -1;
    };
    const int w_groups = (a.w_items + 7) / 8 * 8;
    if ((int)blockIdx.x < w_groups) {
        if constexpr (W) {
            const int item = mine(blockIdx.x, a.w_items);
            if (item >= 0) product<BM, true, CUT>(a, a.w, item, lds);
        }
    } else {
        if constexpr (H) {
            const int item = mine(blockIdx.x - w_groups, a.h_items);
            if (item >= 0) product<BM, false, CUT>(a, a.h, item, lds);
        }
    }
}

// Sums of the parts of dwr's and dbias's reduction, in their order; no parts: zeros (no tokens).
__global__ void __launch_bounds__(256) parts_kernel(const float *__restrict__ parts, const float *__restrict__ bias_parts,
                                                    int32_t splits, int32_t E, int64_t n, void *out, int32_t dtype, float *dbias) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 2;
    if (out && i < n) {
        float s[2] = {0.0f, 0.0f};
#pragma unroll 8
        for (int k = 0; k < splits; ++k) {
            const f2 v = *reinterpret_cast<const f2 *>(parts + k * n + i);
            s[0] += v[0];
            s[1] += v[1];
        }
        if (dtype == MOE_DT_BF16) *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(out) + i) = bf16_pair(s[0], s[1]);
        else *reinterpret_cast<f2 *>(static_cast<float *>(out) + i) = (f2){s[0], s[1]};
    }
    if (dbias) {
        const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (e < E) {
            float s = 0.0f;
#pragma unroll 8
            for (int k = 0; k < splits; ++k) s += bias_parts[(int64_t)k * E + e];
            dbias[e] = s;
        }
    }
}

// Values of g times column tiles from which on g is cut beforehand, which takes a launch and a pass over g, instead of anew
// for every column tile. us cut in the workgroups and beforehand (bf16 dh, fp32 dwr): 2^19 (2000 x 64, 1024 columns) 19, 25;
// 2^21.6 (1024 x 384, 2048) 29, 33; 2^23 (4096 x 256, 2048) 39, 41; 2^23.6 (4096 x 384, 2048) 52, 50; 2^25 (8192 x 256, 4096)
// 120, 97; 2^26.6 (16384 x 384, 4096) 349, 263.
constexpr int64_t kCutFrom = 1 << 23;

}  // namespace

RouteBackwardPlan route_backward_plan(const moe_route_backward_args &a) {
    RouteBackwardPlan p{};
    const int64_t n_tiles = (a.D + kBN - 1) / kBN;
    p.cut = (int64_t)a.T * a.E * n_tiles >= kCutFrom;
    const int32_t bm = p.cut ? kBM : kFusedBM;
    p.t_tiles = (a.T + bm - 1) / bm;
    p.e_tiles = (a.E + bm - 1) / bm;
    p.t_steps = (a.T + kStep - 1) / kStep;
    p.e_steps = (a.E + kStep - 1) / kStep;
    // dwr has few tiles: its reduction is cut so that they fill the CUs once, in parts of 256 tokens at least
    const int64_t tiles = p.e_tiles * n_tiles;
    p.splits = 1;
    if (a.dwr && tiles < 256) {
        const int64_t most = p.t_steps / 8;
        p.splits = (int32_t)(256 / tiles < most ? 256 / tiles : most);
        if (p.splits < 1) p.splits = 1;
    }
    p.steps_per_split = (p.t_steps + p.splits - 1) / p.splits;
    if (p.steps_per_split > 0) p.splits = (p.t_steps + p.steps_per_split - 1) / p.steps_per_split;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~(size_t)255;
        return at;
    };
    p.a_h = take(p.cut && a.dh ? (size_t)kPieces * 8192 * (size_t)p.t_tiles * p.e_steps : 0);
    p.a_w = take(p.cut && a.dwr ? (size_t)kPieces * 8192 * (size_t)p.e_tiles * p.t_steps : 0);
    p.parts = take(p.splits > 1 && a.dwr ? 4 * (size_t)p.splits * a.E * (size_t)a.D : 0);
    p.bias_parts = take(p.splits > 1 && a.dbias ? 4 * (size_t)p.splits * a.E : 0);
    p.total = off > 0 ? off : 256;
    return p;
}

hipError_t launch_route_backward(const moe_route_backward_args &a, const RouteBackwardPlan &p, hipStream_t s) {
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    u32x4 *a_h = reinterpret_cast<u32x4 *>(ws + p.a_h), *a_w = reinterpret_cast<u32x4 *>(ws + p.a_w);
    float *parts = reinterpret_cast<float *>(ws + p.parts), *bias_parts = reinterpret_cast<float *>(ws + p.bias_parts);
    const bool parted = p.splits > 1 || a.T == 0;
    ProductArgs q{};
    q.g = a.d_logits;
    q.T = a.T;
    q.E = a.E;
    q.D = a.D;
    q.n_tiles = (a.D + kBN - 1) / kBN;
    if (a.dwr) {
        q.w = {a_w, a.h, parted ? parts : a.dwr, a.dbias && parted ? bias_parts : a.dbias, a.E, a.T, a.dwr_dtype,
               p.e_tiles, p.t_steps, p.splits, p.steps_per_split};
        q.w_items = p.e_tiles * q.n_tiles * p.splits;
    }
    if (a.dh) {
        q.h = {a_h, a.wr, a.dh, nullptr, a.T, a.E, a.dh_dtype, p.t_tiles, p.e_steps, 1, p.e_steps};
        q.h_items = p.t_tiles * q.n_tiles;
    }
    auto run = [&](auto h, auto w) {
        constexpr bool H = decltype(h)::value, W = decltype(w)::value;
        const unsigned grid = (unsigned)((q.w_items + 7) / 8 * 8 + (q.h_items + 7) / 8 * 8);
        if (p.cut) {
            // with experts as rows the last tile is filled up to 128
            const unsigned e_blocks = (unsigned)(W ? 4 * p.e_tiles : p.e_steps);
            hipLaunchKernelGGL((split_kernel<H, W>), dim3((unsigned)p.t_tiles, e_blocks), dim3(kThreads), 0, s, a.d_logits,
                               a.T, a.E, p.e_steps, p.t_steps, a_h, a_w);
            hipLaunchKernelGGL((product_kernel<H, W, true>), dim3(grid), dim3(kThreads), 0, s, q);
        } else {
            hipLaunchKernelGGL((product_kernel<H, W, false>), dim3(grid), dim3(kThreads), 0, s, q);
        }
    };
    using std::integral_constant;
    if (a.T > 0) {
        if (a.dh && a.dwr) run(integral_constant<bool, true>{}, integral_constant<bool, true>{});
        else if (a.dh) run(integral_constant<bool, true>{}, integral_constant<bool, false>{});
        else run(integral_constant<bool, false>{}, integral_constant<bool, true>{});
    }
    if (parted && a.dwr) {
        const int64_t n = (int64_t)a.E * a.D, threads = n / 2;  // D >= 64: more than dbias has
        hipLaunchKernelGGL(parts_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, parts, bias_parts,
                           a.T == 0 ? 0 : p.splits, a.E, n, a.dwr, a.dwr_dtype, a.dbias);
    }
    return hipGetLastError();
}

}  // namespace moe
