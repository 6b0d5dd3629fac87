// ops_api.hip - host side of the C ABI declared in include/moe_ops.h: argument validation
// (pure host code, no HIP call), the groups' plan layout and the launches on the caller's
// stream.
#include "ops_internal.h"

#include "api_common.h"

using namespace moe;

namespace moe {

GroupsPlan groups_plan(int32_t T, int32_t top_k, int32_t n) {
    GroupsPlan p{};
    const int64_t TK = (int64_t)T * top_k;
    p.n = n;
    p.max_tiles = (int32_t)((TK < n ? TK : n) + TK / kGroupTile);  // a last partial tile per non-empty group
    if (n <= kSortMaxLocal) {
        p.n_chunks = (int32_t)((TK + sort_chunk_slots(TK) - 1) / sort_chunk_slots(TK));
    } else {
        const int32_t ct = T / 256;
        p.chunk_tokens = ct < 8 ? 8 : (ct > 64 ? 64 : ct);
        p.n_chunks = (T + p.chunk_tokens - 1) / p.chunk_tokens;
    }
    if (p.n_chunks < 1) p.n_chunks = 1;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~(size_t)255;
        return at;
    };
    p.ctrl = take(sizeof(Ctrl));
    p.counts = take(sizeof(int32_t) * (size_t)n);
    p.tile_expert = take(sizeof(int32_t) * (size_t)p.max_tiles);
    p.tile_row0 = take(sizeof(int32_t) * (size_t)p.max_tiles);
    p.chunk_counts = take(sizeof(int32_t) * (size_t)p.n_chunks * n);
    p.total = off;
    return p;
}

}  // namespace moe

namespace {

constexpr int32_t kMaxRows = INT32_MAX / 2;  // slots, or rows of one group: rounded up to runs they stay in 32 bits

// The size fields of g.
int32_t check_sizes(const moe_groups *g) {
    if (!g || g->T < 0 || g->top_k < 1 || g->top_k > 8 || g->E < 1 || g->E > 4096) return MOE_ERR_INVALID_ARG;
    if (g->e_begin < 0 || g->e_end <= g->e_begin || g->e_end > g->E) return MOE_ERR_INVALID_ARG;
    if ((int64_t)g->T * g->top_k > kMaxRows) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// Everything of g that moe_sort filled.
int32_t check_groups(const moe_groups *g) {
    const int32_t rc = check_sizes(g);
    if (rc != MOE_OK) return rc;
    if (!g->offsets || (g->T > 0 && (!g->sorted_slot || !g->slot_pos))) return MOE_ERR_INVALID_ARG;
    if (!g->plan || g->plan_bytes < groups_plan(g->T, g->top_k, g->e_end - g->e_begin).total) return MOE_ERR_WORKSPACE;
    if (!aligned(g->offsets, 16) || !aligned(g->sorted_slot, 16) || !aligned(g->slot_pos, 16) || ((uintptr_t)g->plan & 255u))
        return MOE_ERR_ALIGNMENT;
    return MOE_OK;
}

// The row operators' arguments beside their groups: tokens below 2^24 (workgroups of a grid), rows of
// up to 2^30 elements.
int32_t check_rows(const moe_groups *g, int32_t D) {
    if (D < 1) return MOE_ERR_INVALID_ARG;
    return g->T < (1 << 24) && D <= (1 << 30) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

// The output meets one of the buffers; a call refuses that (buffers not given are NULL).
bool overlaps_any(const Extent &out, std::initializer_list<Extent> others) {
    for (const Extent &b : others)
        if (meet(out, b)) return true;
    return false;
}

int64_t row_bytes(int32_t dtype, int32_t D) { return D * type_bytes(dtype); }

// Blocks of a column form that a call touches at most: of g's slots, or of the one group of `rows` rows.
int64_t column_blocks(const moe_groups *g, int32_t rows) {
    return g ? moe_block_column_blocks(g->T * g->top_k, g->e_end - g->e_begin) : ((int64_t)rows + 127) / 128;
}

}  // namespace

namespace moe {

int32_t check_filled_groups(const moe_groups *g) { return check_groups(g); }

GroupView group_view(const moe_groups *g, int32_t rows) {
    GroupView v{};
    if (!g) {
        v.rows = rows;
        v.top_k = 1;
        v.n = 1;
        v.max_tiles = (int32_t)(((int64_t)rows + kGroupTile - 1) / kGroupTile);
        v.mean_rows = rows;
        return v;
    }
    const int32_t n = g->e_end - g->e_begin;
    const GroupsPlan p = groups_plan(g->T, g->top_k, n);
    uint8_t *at = static_cast<uint8_t *>(g->plan);
    v.ctrl = reinterpret_cast<const Ctrl *>(at + p.ctrl);
    v.tile_expert = reinterpret_cast<const int32_t *>(at + p.tile_expert);
    v.tile_row0 = reinterpret_cast<const int32_t *>(at + p.tile_row0);
    v.offsets = g->offsets;
    v.sorted_slot = g->sorted_slot;
    v.rows = g->T * g->top_k;
    v.top_k = g->top_k;
    v.n = n;
    v.max_tiles = p.max_tiles;
    v.mean_rows = (int32_t)((int64_t)g->T * g->top_k / g->E);
    return v;
}

}  // namespace moe

extern "C" {

int32_t moe_ops_abi_version(void) { return MOE_OPS_ABI_VERSION; }

size_t moe_groups_plan_bytes(const moe_groups *g) {
    if (check_sizes(g) != MOE_OK) return 0;
    return groups_plan(g->T, g->top_k, g->e_end - g->e_begin).total;
}

int32_t moe_sort(const moe_groups *g, const int32_t *topk_idx, void *stream) {
    const int32_t rc = check_groups(g);
    if (rc != MOE_OK) return rc;
    if (g->T > 0 && !topk_idx) return MOE_ERR_INVALID_ARG;
    if (!aligned(topk_idx, 16)) return MOE_ERR_ALIGNMENT;
    const int32_t n = g->e_end - g->e_begin;
    const GroupsPlan p = groups_plan(g->T, g->top_k, n);
    uint8_t *at = static_cast<uint8_t *>(g->plan);
    PermuteArgs a{};
    a.T = g->T;
    a.k = g->top_k;
    a.e_begin = g->e_begin;
    a.n_loc = n;
    a.chunk_tokens = p.chunk_tokens;
    a.n_chunks = p.n_chunks;
    a.bm = kGroupTile;
    a.max_tiles = p.max_tiles;
    a.idx = topk_idx;
    a.chunk_counts = reinterpret_cast<int32_t *>(at + p.chunk_counts);
    a.counts = reinterpret_cast<int32_t *>(at + p.counts);
    a.offsets = g->offsets;
    a.tile_expert = reinterpret_cast<int32_t *>(at + p.tile_expert);
    a.tile_row0 = reinterpret_cast<int32_t *>(at + p.tile_row0);
    a.sorted_slot = g->sorted_slot;
    a.slot_pos = g->slot_pos;
    a.ctrl = reinterpret_cast<Ctrl *>(at + p.ctrl);
    a.fill_tail = 1;
    hipStream_t s = (hipStream_t)stream;
    return status_of(n <= kSortMaxLocal ? launch_sort(a, g->T * g->top_k, s) : launch_permute(a, s));
}

int32_t moe_gather(const moe_groups *g, int32_t dtype, int32_t D, const void *x, void *rows, void *stream) {
    const int32_t rc = check_groups(g);
    if (rc != MOE_OK) return rc;
    if (!type_ok(dtype)) return MOE_ERR_INVALID_ARG;
    const int32_t rr = check_rows(g, D);
    if (rr != MOE_OK) return rr;
    if (g->T == 0) return MOE_OK;
    if (!x || !rows) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(rows, 16)) return MOE_ERR_ALIGNMENT;
    const int64_t bytes = row_bytes(dtype, D);
    if (overlaps_any({rows, (int64_t)g->T * g->top_k, bytes}, {{x, g->T, bytes}})) return MOE_ERR_INVALID_ARG;
    return status_of(launch_gather(*g, dtype, D, x, rows, (hipStream_t)stream));
}

int32_t moe_gather_backward(const moe_groups *g, int32_t dtype, int32_t D, const void *d_rows, void *dx, void *stream) {
    const int32_t rc = check_groups(g);
    if (rc != MOE_OK) return rc;
    if (!type_ok(dtype)) return MOE_ERR_INVALID_ARG;
    const int32_t rr = check_rows(g, D);
    if (rr != MOE_OK) return rr;
    if (g->T == 0) return MOE_OK;
    if (!d_rows || !dx) return MOE_ERR_INVALID_ARG;
    if (!aligned(d_rows, 16) || !aligned(dx, 16)) return MOE_ERR_ALIGNMENT;
    const int64_t bytes = row_bytes(dtype, D);
    if (overlaps_any({dx, g->T, bytes}, {{d_rows, (int64_t)g->T * g->top_k, bytes}})) return MOE_ERR_INVALID_ARG;
    return status_of(launch_combine_rows(*g, dtype, dtype, D, d_rows, nullptr, dx, (hipStream_t)stream));
}

int32_t moe_combine(const moe_groups *g, int32_t y_dtype, int32_t out_dtype, int32_t D, const void *y, const float *w,
                    void *out, void *stream) {
    const int32_t rc = check_groups(g);
    if (rc != MOE_OK) return rc;
    if (!type_ok(y_dtype) || !type_ok(out_dtype)) return MOE_ERR_INVALID_ARG;
    const int32_t rr = check_rows(g, D);
    if (rr != MOE_OK) return rr;
    if (g->T == 0) return MOE_OK;
    if (!y || !w || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(w, 16) || !aligned(out, 16)) return MOE_ERR_ALIGNMENT;
    const int64_t slots = (int64_t)g->T * g->top_k;
    if (overlaps_any({out, g->T, row_bytes(out_dtype, D)}, {{y, slots, row_bytes(y_dtype, D)}, {w, slots, 4}}))
        return MOE_ERR_INVALID_ARG;
    return status_of(launch_combine_rows(*g, y_dtype, out_dtype, D, y, w, out, (hipStream_t)stream));
}

int32_t moe_combine_backward(const moe_groups *g, int32_t y_dtype, int32_t out_dtype, int32_t D, const void *d_out,
                             const void *y, const float *w, void *d_y, float *d_w, void *stream) {
    const int32_t rc = check_groups(g);
    if (rc != MOE_OK) return rc;
    if (!type_ok(y_dtype) || !type_ok(out_dtype)) return MOE_ERR_INVALID_ARG;
    const int32_t rr = check_rows(g, D);
    if (rr != MOE_OK) return rr;
    if (g->T == 0) return MOE_OK;
    if (!d_out || !y || !w || !d_y || !d_w) return MOE_ERR_INVALID_ARG;
    if (!aligned(d_out, 16) || !aligned(y, 16) || !aligned(w, 16) || !aligned(d_y, 16) || !aligned(d_w, 16))
        return MOE_ERR_ALIGNMENT;
    const int64_t slots = (int64_t)g->T * g->top_k;
    const Extent bo = {d_out, g->T, row_bytes(out_dtype, D)}, by = {y, slots, row_bytes(y_dtype, D)}, bw = {w, slots, 4};
    const Extent bdy = {d_y, slots, by.item}, bdw = {d_w, slots, 4};
    if (overlaps_any(bdy, {bo, by, bw, bdw}) || overlaps_any(bdw, {bo, by}) || (d_w != w && meet(bdw, bw)))
        return MOE_ERR_INVALID_ARG;
    return status_of(launch_combine_backward(*g, y_dtype, out_dtype, D, d_out, y, w, d_y, d_w, (hipStream_t)stream));
}

int64_t moe_block_column_blocks(int32_t rows, int32_t n) {
    if (rows < 0 || n < 1) return 0;
    return (int64_t)rows / 128 + n;
}

int32_t moe_block_quantize(const moe_block_quantize_args *q, void *stream) {
    if (!q || q->rows < 0 || q->C < 1) return MOE_ERR_INVALID_ARG;
    if (q->C % 128 || q->C > kMaxBlockDim) return MOE_ERR_UNSUPPORTED;
    const bool by_rows = q->codes || q->scales, by_columns = q->col_codes || q->col_scales;
    if (!by_rows && !by_columns) return MOE_ERR_INVALID_ARG;
    if (by_rows && (!q->codes || !q->scales)) return MOE_ERR_INVALID_ARG;
    if (by_columns && (!q->col_codes || !q->col_scales)) return MOE_ERR_INVALID_ARG;
    if (q->by_token && (!q->g || by_rows)) return MOE_ERR_INVALID_ARG;
    if (q->g) {
        const int32_t rc = check_groups(q->g);
        if (rc != MOE_OK) return rc;
        if (q->rows != (q->by_token ? q->g->T : q->g->T * q->g->top_k)) return MOE_ERR_INVALID_ARG;
    }
    if ((by_rows && !rows_form_fits(q->rows, q->C)) || q->rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (q->rows == 0) return MOE_OK;
    if (!q->x) return MOE_ERR_INVALID_ARG;
    if (!aligned(q->x, 16) || !aligned(q->codes, 16) || !aligned(q->scales, 16) || !aligned(q->col_codes, 16) ||
        !aligned(q->col_scales, 16))
        return MOE_ERR_ALIGNMENT;
    const Extent x = {q->x, q->rows, (int64_t)q->C * 2};
    const Extent c = {q->codes, q->rows, q->C}, s = {q->scales, q->rows, (int64_t)scale_stride(q->C) * 4};
    const int64_t blocks = column_blocks(q->g, q->rows);
    const Extent cc = {q->col_codes, blocks, (int64_t)q->C * 128}, cs = {q->col_scales, blocks, (int64_t)q->C * 4};
    if (overlaps_any(x, {c, s, cc, cs}) || overlaps_any(c, {s, cc, cs}) || overlaps_any(s, {cc, cs}) || overlaps_any(cc, {cs}))
        return MOE_ERR_INVALID_ARG;
    BlockQuantArgs a{};
    a.offsets = q->g ? q->g->offsets : nullptr;
    a.sorted_slot = q->by_token ? q->g->sorted_slot : nullptr;
    a.rows = q->g ? q->g->T * q->g->top_k : q->rows;
    a.n = q->g ? q->g->e_end - q->g->e_begin : 1;
    a.top_k = q->g ? q->g->top_k : 1;
    a.C = q->C;
    a.x = q->x;
    a.codes = q->codes;
    a.scales = q->scales;
    a.col_codes = q->col_codes;
    a.col_scales = q->col_scales;
    hipStream_t hs = (hipStream_t)stream;
    return status_of(by_columns ? launch_block_quant_columns(a, hs) : launch_block_quant_rows(a, hs));
}

// Codes and scales of weights [E][N][K].
static Extent weight_codes(const void *p, int32_t E, int32_t N, int32_t K) { return {p, E, (int64_t)N * K}; }
static Extent weight_scales(const void *p, int32_t E, int32_t N, int32_t K) { return {p, E, (int64_t)(N / 128) * (K / 128) * 4}; }

// Sizes and buffers of weights [E][N][K].
static int32_t check_weights(int32_t E, int32_t N, int32_t K, const void *codes, const void *scales) {
    if (E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
    if (N % 128 || K % 128 || N > kMaxBlockDim || K > kMaxBlockDim) return MOE_ERR_UNSUPPORTED;
    if (!codes || !scales) return MOE_ERR_INVALID_ARG;
    // the scales are read one at a time: those of an expert in the middle are as good as the first's
    if (!aligned(codes, 16) || ((uintptr_t)scales & 3u)) return MOE_ERR_ALIGNMENT;
    return MOE_OK;
}

int32_t moe_block_quantize_weights(const uint16_t *w, int32_t E, int32_t N, int32_t K, uint8_t *codes, float *scales,
                                   void *stream) {
    const int32_t rc = check_weights(E, N, K, codes, scales);
    if (rc != MOE_OK) return rc;
    if (!w) return MOE_ERR_INVALID_ARG;
    if (!aligned(w, 16)) return MOE_ERR_ALIGNMENT;
    const Extent c = weight_codes(codes, E, N, K), s = weight_scales(scales, E, N, K), x = {w, E, (int64_t)N * K * 2};
    if (overlaps_any(x, {c, s}) || overlaps_any(c, {s})) return MOE_ERR_INVALID_ARG;
    return status_of(launch_block_quant_weights(w, E, N, K, codes, scales, (hipStream_t)stream));
}

int32_t moe_block_pack_weights(const uint8_t *rowmajor, int32_t E, int32_t N, int32_t K, uint8_t *codes, void *stream) {
    const int32_t rc = check_weights(E, N, K, codes, codes);
    if (rc != MOE_OK) return rc;
    if (!rowmajor) return MOE_ERR_INVALID_ARG;
    if (!aligned(rowmajor, 16)) return MOE_ERR_ALIGNMENT;
    if (overlaps_any(weight_codes(codes, E, N, K), {weight_codes(rowmajor, E, N, K)})) return MOE_ERR_INVALID_ARG;
    return status_of(launch_pack_rowmajor(MOE_FMT_FP8, rowmajor, nullptr, E, N, K, codes, nullptr, (hipStream_t)stream));
}

int32_t moe_block_gemm(const moe_block_gemm_args *a, void *stream) {
    if (!a || a->rows < 0) return MOE_ERR_INVALID_ARG;
    int32_t rc = check_weights(a->w.E, a->w.N, a->w.K, a->w.codes, a->w.scales);
    if (rc != MOE_OK) return rc;
    if (a->g) {
        rc = check_groups(a->g);
        if (rc != MOE_OK) return rc;
        if (a->w.E != a->g->e_end - a->g->e_begin) return MOE_ERR_INVALID_ARG;
        if (a->rows != (a->by_token ? a->g->T : a->g->T * a->g->top_k)) return MOE_ERR_INVALID_ARG;
    } else if (a->by_token || a->w.E != 1) {
        return MOE_ERR_INVALID_ARG;
    }
    if (a->by_token && a->transposed) return MOE_ERR_INVALID_ARG;  // gradients come in sorted rows
    if (!rows_form_fits(a->rows, a->transposed ? a->w.N : a->w.K)) return MOE_ERR_UNSUPPORTED;
    if (a->rows == 0) return MOE_OK;
    if (!a->x_codes || !a->x_scales || !a->out) return MOE_ERR_INVALID_ARG;
    if (!aligned(a->x_codes, 16) || !aligned(a->x_scales, 16) || !aligned(a->out, 16)) return MOE_ERR_ALIGNMENT;
    BlockGemmArgs p{};
    p.v = group_view(a->g, a->rows);
    p.by_token = a->by_token ? 1 : 0;
    p.x_rows = a->rows;
    p.R = a->transposed ? a->w.N : a->w.K;
    p.C = a->transposed ? a->w.K : a->w.N;
    p.x_codes = a->x_codes;
    p.x_scales = a->x_scales;
    p.w_codes = a->w.codes;
    p.w_scales = a->w.scales;
    p.w_expert_bytes = (int64_t)a->w.N * a->w.K;
    p.w_expert_scales = (a->w.N / 128) * (a->w.K / 128);
    p.w_kb = a->w.K / 128;
    p.out = a->out;
    const int64_t out_rows = a->g ? a->g->T * a->g->top_k : a->rows;
    if (overlaps_any({a->out, out_rows, (int64_t)p.C * 2},
                     {{a->x_codes, a->rows, p.R}, {a->x_scales, a->rows, (int64_t)scale_stride(p.R) * 4},
                      weight_codes(a->w.codes, a->w.E, a->w.N, a->w.K), weight_scales(a->w.scales, a->w.E, a->w.N, a->w.K)}))
        return MOE_ERR_INVALID_ARG;
    return status_of(launch_block_gemm(p, a->transposed != 0, (hipStream_t)stream));
}

int32_t moe_block_wgrad(const moe_block_wgrad_args *a, void *stream) {
    if (!a || a->rows < 0 || a->N < 1 || a->K < 1) return MOE_ERR_INVALID_ARG;
    if (a->N % 128 || a->K % 128 || a->N > kMaxBlockDim || a->K > kMaxBlockDim || a->rows > kMaxRows)
        return MOE_ERR_UNSUPPORTED;
    if (a->g) {
        const int32_t rc = check_groups(a->g);
        if (rc != MOE_OK) return rc;
        if (a->rows != a->g->T * a->g->top_k) return MOE_ERR_INVALID_ARG;
    }
    if (!a->dw || (a->rows > 0 && (!a->g_codes || !a->g_scales || !a->x_codes || !a->x_scales)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(a->dw, 16) || !aligned(a->g_codes, 16) || !aligned(a->g_scales, 16) || !aligned(a->x_codes, 16) ||
        !aligned(a->x_scales, 16))
        return MOE_ERR_ALIGNMENT;
    const int64_t blocks = column_blocks(a->g, a->rows);
    if (overlaps_any({a->dw, a->g ? a->g->e_end - a->g->e_begin : 1, (int64_t)a->N * a->K * 2},
                     {{a->g_codes, blocks, (int64_t)a->N * 128}, {a->g_scales, blocks, (int64_t)a->N * 4},
                      {a->x_codes, blocks, (int64_t)a->K * 128}, {a->x_scales, blocks, (int64_t)a->K * 4}}))
        return MOE_ERR_INVALID_ARG;
    BlockWgradArgs p{};
    p.offsets = a->g ? a->g->offsets : nullptr;
    p.rows = a->rows;
    p.n = a->g ? a->g->e_end - a->g->e_begin : 1;
    p.N = a->N;
    p.K = a->K;
    p.g_codes = a->g_codes;
    p.x_codes = a->x_codes;
    p.g_scales = a->g_scales;
    p.x_scales = a->x_scales;
    p.dw = a->dw;
    return status_of(launch_block_wgrad(p, (hipStream_t)stream));
}

}  // extern "C"
