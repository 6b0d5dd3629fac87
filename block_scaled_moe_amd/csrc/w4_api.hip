// w4_api.hip - host side of the C ABI declared in include/moe_w4.h: argument validation (pure host code, no HIP
// call) and the launches on the caller's stream.
#include "w4_internal.h"

#include "api_common.h"

using namespace moe;

namespace {

int32_t check_sizes(const moe_w4_weights *w) {
    if (!w || w->E < 1 || w->E > 4096 || w->N < 1 || w->K < 1) return MOE_ERR_INVALID_ARG;
    if (w->scale_type != MOE_W4_SCALE_BF16 && w->scale_type != MOE_W4_SCALE_FP16) return MOE_ERR_INVALID_ARG;
    if (w->group != 32 && w->group != 64 && w->group != 128) return MOE_ERR_UNSUPPORTED;
    if (w->K % w->group || w->N > (1 << 20) || w->K > (1 << 20) || (int64_t)w->N * w->K >= (1ll << 36)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
int64_t code_bytes(const moe_w4_weights &w) { return w.E * w4_tiles(w) * w4_steps(w) * 2048; }
int64_t zero_bytes(const moe_w4_weights &w) { return w.E * w4_tiles(w) * w4_steps(w) * (kW4Rows * kW4Step / w.group); }

int32_t check_weights(const moe_w4_weights *w) {
    const int32_t rc = check_sizes(w);
    if (rc != MOE_OK) return rc;
    if (!w->codes || !w->scales) return MOE_ERR_INVALID_ARG;
    return aligned(w->codes, 16) && aligned(w->scales, 16) && aligned(w->zeros, 16) ? MOE_OK : MOE_ERR_ALIGNMENT;
}

}  // namespace

extern "C" {

int32_t moe_w4_abi_version(void) { return MOE_W4_ABI_VERSION; }

size_t moe_w4_code_bytes(const moe_w4_weights *w) { return check_sizes(w) == MOE_OK ? (size_t)code_bytes(*w) : 0; }
size_t moe_w4_scale_bytes(const moe_w4_weights *w) { return check_sizes(w) == MOE_OK ? 2 * (size_t)zero_bytes(*w) : 0; }
size_t moe_w4_zero_bytes(const moe_w4_weights *w) { return check_sizes(w) == MOE_OK ? (size_t)zero_bytes(*w) : 0; }

int32_t moe_w4_pack(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, const moe_w4_weights *w, void *stream) {
    const int32_t rc = check_weights(w);
    if (rc != MOE_OK) return rc;
    if (!codes || !scales || !zeros != !w->zeros) return MOE_ERR_INVALID_ARG;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(zeros, 16)) return MOE_ERR_ALIGNMENT;
    const int64_t rows = (int64_t)w->E * w->N, groups = w->K / w->group;
    if (outputs_meet({{w->codes, 1, code_bytes(*w)}, {w->scales, 2, zero_bytes(*w)}, {w->zeros, 1, zero_bytes(*w)}},
                     {{codes, rows, w->K / 2}, {scales, rows, 2 * groups}, {zeros, rows, groups}}))
        return MOE_ERR_INVALID_ARG;
    return status_of(launch_w4_pack(codes, scales, zeros, *w, (hipStream_t)stream));
}

int32_t moe_w4_gemm(const moe_w4_gemm_args *a, void *stream) {
    if (!a || a->rows < 0 || !type_ok(a->out_dtype)) return MOE_ERR_INVALID_ARG;
    int32_t rc = check_weights(&a->w);
    if (rc != MOE_OK) return rc;
    if (a->swiglu && a->w.N % 2) return MOE_ERR_INVALID_ARG;
    if (a->g) {
        rc = check_filled_groups(a->g);
        if (rc != MOE_OK) return rc;
        if (a->w.E != a->g->e_end - a->g->e_begin) return MOE_ERR_INVALID_ARG;
        if (a->rows != (a->by_token ? a->g->T : a->g->T * a->g->top_k)) return MOE_ERR_INVALID_ARG;
    } else if (a->by_token || a->w.E != 1) {
        return MOE_ERR_INVALID_ARG;
    }
    if (a->rows >= (1 << 25) || (int64_t)a->rows * a->w.K >= (1ll << 36)) return MOE_ERR_UNSUPPORTED;
    if (a->rows == 0) return MOE_OK;
    if (!a->x || !a->out) return MOE_ERR_INVALID_ARG;
    if (!aligned(a->x, 16) || !aligned(a->out, 16)) return MOE_ERR_ALIGNMENT;
    W4GemmArgs p{};
    p.v = group_view(a->g, a->rows);
    p.by_token = a->by_token ? 1 : 0;
    p.swiglu = a->swiglu ? 1 : 0;
    p.out_dtype = a->out_dtype;
    p.x = a->x;
    p.w = a->w;
    p.tiles = (int32_t)w4_tiles(a->w);
    p.steps = (int32_t)w4_steps(a->w);
    p.C = a->swiglu ? a->w.N / 2 : a->w.N;
    p.slot_factor = (uint32_t)(((1ull << 31) + p.v.top_k - 1) / p.v.top_k);
    p.out = a->out;
    const int64_t out_rows = a->g ? a->g->T * a->g->top_k : a->rows;
    if (outputs_meet({{a->out, out_rows, p.C * type_bytes(a->out_dtype)}},
                     {{a->x, a->rows, (int64_t)a->w.K * 2}, {a->w.codes, 1, code_bytes(a->w)}, {a->w.scales, 2, zero_bytes(a->w)},
                      {a->w.zeros, 1, zero_bytes(a->w)}}))
        return MOE_ERR_INVALID_ARG;
    return status_of(launch_w4_gemm(p, (hipStream_t)stream));
}

}  // extern "C"
