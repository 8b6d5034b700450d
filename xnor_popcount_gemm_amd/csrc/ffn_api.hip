// C ABI of the feed-forward calls: argument validation and dispatch.  As in
// bnn_api.hip every check runs before anything is launched; the semantics of
// each entry point are documented in include/bnn.h.
#include <math.h>

#include "bnn.h"
#include "expert_kernel.hpp"

namespace {

constexpr int64_t MAX_ROWS = (int64_t)1 << 30;
constexpr int64_t MAX_LD = (int64_t)1 << 40;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
hipStream_t as_stream(bnn_stream_t s) { return reinterpret_cast<hipStream_t>(s); }
bnn_status from_hip(hipError_t e) { return e == hipSuccess ? BNN_OK : BNN_ERR_HIP; }
bool is_type(int32_t t) { return t == BNN_F32 || t == BNN_BF16 || t == BNN_F16; }

// A matrix of `rows` rows of D values, each row `ld` values after the one
// before, aligned to its type.  Byte offsets stay below 2^62.
bnn_status check_matrix(const void* p, int64_t rows, int64_t D, int64_t ld, int64_t bytes) {
    if (!p) return BNN_ERR_NULL;
    if (ld < D || ld > MAX_LD || rows * ((ld * bytes + 1023) / 1024) > ((int64_t)1 << 52)) return BNN_ERR_LD;
    return misaligned(p, (uintptr_t)bytes) ? BNN_ERR_ALIGN : BNN_OK;
}

bnn_status check_vector(const void* p) { return misaligned(p, 4) ? BNN_ERR_ALIGN : BNN_OK; }

// Whether rows can be read 4 values at a time.
bool by_four(const void* p, int64_t ld, int64_t bytes) { return !misaligned(p, (uintptr_t)(4 * bytes)) && ld % 4 == 0; }

}  // namespace

#define BNN_TRY(x) do { const bnn_status st_ = (x); if (st_ != BNN_OK) return st_; } while (0)

#pragma GCC visibility push(default)
extern "C" {

bnn_status bnn_block_norm(const bnn_norm_args* a, bnn_stream_t stream) {
    if (!a) return BNN_ERR_NULL;
    if (a->M < 0 || a->M > MAX_ROWS || a->D < 1 || a->D > BNN_MAX_NORM_D) return BNN_ERR_SHAPE;
    if (!a->x && !a->branch) return BNN_ERR_NULL;
    if ((a->x || a->x_out) && !is_type(a->x_dtype)) return BNN_ERR_UNSUPPORTED;
    if (a->branch && !is_type(a->b_dtype)) return BNN_ERR_UNSUPPORTED;
    if (a->y && !is_type(a->y_dtype)) return BNN_ERR_UNSUPPORTED;
    for (const int32_t k : {a->post, a->pre})
        if (k != BNN_NORM_NONE && k != BNN_NORM_RMS && k != BNN_NORM_LAYER) return BNN_ERR_UNSUPPORTED;
    if (!isfinite(a->x_scale) || !isfinite(a->branch_scale) || !(a->eps >= 0.f) || !isfinite(a->eps)) return BNN_ERR_UNSUPPORTED;
    if (!a->branch && (a->place || a->gate || a->post != BNN_NORM_NONE)) return BNN_ERR_UNSUPPORTED;
    if (!a->x_out && !a->y && !a->Xq && !a->Xb) return BNN_ERR_NULL;
    if ((a->Xq || a->Xb) && !a->xscale) return BNN_ERR_NULL;
    if (a->Xb && !a->xsum) return BNN_ERR_NULL;
    if (!a->Xq && !a->Xb && (a->xscale || a->xsum)) return BNN_ERR_NULL;
    const int64_t xb = bnn::type_bytes(a->x_dtype), bb = bnn::type_bytes(a->b_dtype), yb = bnn::type_bytes(a->y_dtype);
    if (a->x) BNN_TRY(check_matrix(a->x, a->M, a->D, a->ldx, xb));
    if (a->branch) {
        if (a->b_rows < 0 || a->b_rows > MAX_ROWS || (!a->place && a->b_rows < a->M)) return BNN_ERR_SHAPE;
        BNN_TRY(check_matrix(a->branch, a->b_rows, a->D, a->ldb, bb));
    }
    if (a->place && (a->parts < 1 || a->parts > 64)) return BNN_ERR_SHAPE;
    if (a->gate) {
        if (a->ld_gate != 0) BNN_TRY(check_matrix(a->gate, a->M, a->D, a->ld_gate, 4));
        BNN_TRY(check_vector(a->gate));
    }
    for (const void* p : {(const void*)a->used, (const void*)a->place, (const void*)a->weight, (const void*)a->post_weight, (const void*)a->post_bias,
                          (const void*)a->pre_weight, (const void*)a->pre_bias, (const void*)a->xsum, (const void*)a->xscale})
        BNN_TRY(check_vector(p));
    if (a->x_out) BNN_TRY(check_matrix(a->x_out, a->M, a->D, a->ldxo, xb));
    if (a->y) BNN_TRY(check_matrix(a->y, a->M, a->D, a->ldy, yb));
    if (a->Xq) BNN_TRY(check_matrix(a->Xq, a->M, a->D, a->ldXq, 1));
    if (a->Xb) {
        BNN_TRY(check_matrix(a->Xb, 8 * a->M, (a->D + 31) / 32, a->ldXb, 4));
        if (misaligned(a->Xb, 16) || a->ldXb % 4 != 0) return BNN_ERR_ALIGN;
    }
    if (a->M == 0) return BNN_OK;
    bnn::NormArgs r = {};
    r.M = a->M; r.D = (int32_t)a->D;
    r.used = a->used;
    r.x = (const char*)a->x; r.ldx = a->ldx; r.x_type = a->x_dtype;
    r.b = (const char*)a->branch; r.ldb = a->ldb; r.b_type = a->b_dtype; r.b_rows = (int32_t)a->b_rows;
    r.place = a->place; r.weight = a->weight; r.parts = (int32_t)a->parts;
    r.post = a->post; r.post_w = a->post_weight; r.post_b = a->post_bias;
    r.gate = a->gate; r.ld_gate = a->ld_gate;
    r.x_scale = a->x_scale; r.b_scale = a->branch_scale;
    r.pre = a->pre; r.pre_w = a->pre_weight; r.pre_b = a->pre_bias;
    r.eps = a->eps;
    r.xo = (char*)a->x_out; r.ldxo = a->ldxo;
    r.y = (char*)a->y; r.ldy = a->ldy; r.y_type = a->y_dtype;
    r.Xq = a->Xq; r.ldXq = a->ldXq;
    r.Xb = a->Xb; r.ldXb = a->ldXb;
    r.xsum = a->xsum; r.xscale = a->xscale;
    r.vec = (by_four(a->x, a->ldx, xb) ? bnn::V_X : 0) | (by_four(a->branch, a->ldb, bb) ? bnn::V_B : 0) |
            (by_four(a->gate, a->ld_gate, 4) ? bnn::V_GATE : 0) | (by_four(a->x_out, a->ldxo, xb) ? bnn::V_XO : 0) |
            (by_four(a->y, a->ldy, yb) ? bnn::V_Y : 0) | (!misaligned(a->Xq, 16) && a->ldXq % 16 == 0 ? bnn::V_Q : 0) |
            (misaligned(a->post_weight, 16) ? 0 : bnn::V_POST_W) | (misaligned(a->post_bias, 16) ? 0 : bnn::V_POST_B) |
            (misaligned(a->pre_weight, 16) ? 0 : bnn::V_PRE_W) | (misaligned(a->pre_bias, 16) ? 0 : bnn::V_PRE_B);
    return from_hip(bnn::launch_block_norm(r, as_stream(stream)));
}

static bnn_status check_route(int64_t rows, int64_t experts, int64_t top) {
    if (experts < 1 || experts > BNN_MAX_EXPERTS || top < 1 || top > 64 || top > experts) return BNN_ERR_SHAPE;
    return rows < 0 || rows > MAX_ROWS || rows * top >= MAX_ROWS ? BNN_ERR_SHAPE : BNN_OK;
}

int64_t bnn_expert_route_workspace(int64_t rows, int64_t experts, int64_t top) {
    return check_route(rows, experts, top) == BNN_OK ? bnn::expert_route_work(rows, experts, top) : -1;
}

bnn_status bnn_expert_route(const bnn_route_args* a, bnn_stream_t stream) {
    if (!a) return BNN_ERR_NULL;
    BNN_TRY(check_route(a->rows, a->experts, a->top));
    if (!is_type(a->dtype)) return BNN_ERR_UNSUPPORTED;
    if (a->score != BNN_ROUTE_SOFTMAX && a->score != BNN_ROUTE_SIGMOID) return BNN_ERR_UNSUPPORTED;
    if (!isfinite(a->scale)) return BNN_ERR_UNSUPPORTED;
    BNN_TRY(check_matrix(a->logits, a->rows, a->experts, a->ld, bnn::type_bytes(a->dtype)));
    for (const void* p : {(const void*)a->expert, (const void*)a->weight, (const void*)a->offsets, (const void*)a->order, (const void*)a->place}) {
        if (!p) return BNN_ERR_NULL;
        BNN_TRY(check_vector(p));
    }
    BNN_TRY(check_vector(a->used));
    BNN_TRY(check_vector(a->bias));
    const int64_t need = bnn::expert_route_work(a->rows, a->experts, a->top);
    if (need > 0) {
        if (!a->workspace) return BNN_ERR_NULL;
        if (misaligned(a->workspace, 16)) return BNN_ERR_ALIGN;
        if (a->workspace_bytes < need) return BNN_ERR_SHAPE;
    }
    bnn::RouteArgs r;
    r.logits = (const char*)a->logits; r.ld = a->ld; r.type = a->dtype;
    r.rows = (int32_t)a->rows; r.experts = (int32_t)a->experts; r.top = (int32_t)a->top;
    r.used = a->used;
    r.sigmoid = a->score == BNN_ROUTE_SIGMOID;
    r.bias = a->bias;
    r.renorm = a->renorm != 0; r.scale = a->scale;
    r.expert = a->expert; r.weight = a->weight;
    r.offsets = a->offsets; r.order = a->order; r.place = a->place;
    r.work = (int32_t*)a->workspace;
    return from_hip(bnn::launch_expert_route(r, as_stream(stream)));   // without rows too: the offsets are zeros
}

int64_t bnn_expert_pack_bytes(int64_t experts, int64_t N, int64_t K, int32_t ternary) {
    if (experts < 0 || experts > BNN_MAX_EXPERTS || N < 0 || N > ((int64_t)1 << 24) || K < 1 || K > BNN_MAX_K_I8) return -1;
    const int64_t ck = bnn::chunk_k(ternary != 0);
    return experts * ((N + 15) / 16) * ((K + ck - 1) / ck) * 1024;   // below 2^50
}

bnn_status bnn_expert_pack(const uint32_t* Wp, const uint32_t* Zp, int64_t ldWp, int64_t w_expert, int64_t experts, int64_t N, int64_t K, void* out,
                           int64_t out_bytes, bnn_stream_t stream) {
    const int64_t bytes = bnn_expert_pack_bytes(experts, N, K, Zp != nullptr);
    if (bytes < 0) return BNN_ERR_SHAPE;
    if (!Wp || !out) return BNN_ERR_NULL;
    if (ldWp < (K + 31) / 32 || ldWp > MAX_LD || w_expert < 0 || w_expert > MAX_LD || N * ldWp > ((int64_t)1 << 50)) return BNN_ERR_LD;
    if (experts > 1 && w_expert < N * ldWp) return BNN_ERR_LD;
    if (misaligned(Wp, 16) || misaligned(Zp, 16) || ldWp % 4 != 0 || misaligned(out, 16)) return BNN_ERR_ALIGN;
    if (out_bytes < bytes) return BNN_ERR_SHAPE;
    if (bytes >> 12 >= (int64_t)1 << 32) return BNN_ERR_SHAPE;   // more workgroups than a launch takes
    if (bytes == 0) return BNN_OK;
    return from_hip(bnn::launch_expert_pack(Wp, Zp, ldWp, w_expert, experts, N, K, out, as_stream(stream)));
}

static bnn_status check_scales(const bnn_expert_matrix& m, int64_t experts, int64_t N, bnn::ExpertMatrix& k) {
    if (!m.W || !m.alpha) return BNN_ERR_NULL;
    if (misaligned(m.W, 16)) return BNN_ERR_ALIGN;
    if (m.ld_alpha != 0) BNN_TRY(check_matrix(m.alpha, experts, N, m.ld_alpha, 4));
    if (m.bias) BNN_TRY(check_matrix(m.bias, experts, N, m.ld_bias, 4));
    BNN_TRY(check_vector(m.alpha));
    k.W = (const uint4*)m.W;
    k.alpha = m.alpha; k.ld_alpha = m.ld_alpha;
    k.bias = m.bias; k.ld_bias = m.ld_bias;
    return BNN_OK;
}

bnn_status bnn_expert_linear(const bnn_expert_args* a, bnn_stream_t stream) {
    if (!a) return BNN_ERR_NULL;
    if (a->experts < 1 || a->experts > BNN_MAX_EXPERTS || a->positions < 0 || a->positions > MAX_ROWS || a->rows < 0 || a->rows > MAX_ROWS)
        return BNN_ERR_SHAPE;
    if (bnn_expert_pack_bytes(a->experts, a->N, a->K, a->ternary) < 0) return BNN_ERR_SHAPE;
    if (!a->offsets && a->experts != 1) return BNN_ERR_NULL;
    if (a->act < BNN_ACT_NONE || a->act > BNN_ACT_GELU_TANH || !is_type(a->y_dtype)) return BNN_ERR_UNSUPPORTED;
    if (a->order ? a->per_row < 1 || a->per_row > MAX_ROWS : a->rows < a->positions) return BNN_ERR_SHAPE;
    BNN_TRY(check_matrix(a->Xq, a->rows, a->K, a->ldXq, 1));
    if (misaligned(a->Xq, 16) || a->ldXq % 16 != 0) return BNN_ERR_ALIGN;
    for (const void* p : {(const void*)a->xscale, (const void*)a->order, (const void*)a->offsets}) BNN_TRY(check_vector(p));
    bnn::ExpertArgs r = {};
    BNN_TRY(check_scales(a->main, a->experts, a->N, r.m));
    if (a->up.W) BNN_TRY(check_scales(a->up, a->experts, a->N, r.u));
    const int64_t yb = bnn::type_bytes(a->y_dtype);
    if (a->residual) BNN_TRY(check_matrix(a->residual, a->positions, a->N, a->ldr, yb));
    BNN_TRY(check_matrix(a->y, a->positions, a->N, a->ldy, yb));
    r.Xq = a->Xq; r.ldXq = a->ldXq;
    r.xscale = a->xscale;
    r.rows = (int32_t)a->rows;
    r.order = a->order; r.per_row = bnn::make_fastdiv((uint32_t)(a->order ? a->per_row : 1));
    r.offsets = a->offsets;
    r.experts = (int32_t)a->experts; r.positions = (int32_t)a->positions; r.N = (int32_t)a->N; r.K = (int32_t)a->K;
    r.act = a->act;
    r.r = (const char*)a->residual; r.ldr = a->ldr;
    r.y = (char*)a->y; r.ldy = a->ldy; r.y_type = a->y_dtype;
    if (a->positions == 0 || a->N == 0 || a->rows == 0) return BNN_OK;
    if (!bnn::expert_linear_fits(r, a->ternary != 0)) return BNN_ERR_SHAPE;   // more workgroups than a launch takes
    return from_hip(bnn::launch_expert_linear(r, a->ternary != 0, as_stream(stream)));
}

}  // extern "C"
#pragma GCC visibility pop

namespace bnn {

bool expert_linear_fits(const ExpertArgs& a, bool ternary) { return expert_tile_takes(a) || expert_rows_fits(a, ternary); }

hipError_t launch_expert_linear(const ExpertArgs& a, bool ternary, hipStream_t s) {
    return expert_tile_takes(a) ? launch_expert_tile(a, ternary, s) : launch_expert_rows(a, ternary, s);
}

}  // namespace bnn
