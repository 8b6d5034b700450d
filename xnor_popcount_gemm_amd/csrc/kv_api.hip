// C ABI of the calls over the key/value cache: argument validation and
// dispatch.  As in bnn_api.hip every check runs before anything is launched;
// the semantics of each entry point are documented in include/bnn.h.
#include <math.h>

#include "bnn.h"
#include "kv_launch.hpp"

namespace {

using bnn::KvBatch;
using bnn::KvCache;

constexpr int64_t MAX_SLOTS = (int64_t)1 << 30;
constexpr int64_t MAX_STRIDE = (int64_t)1 << 47;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
hipStream_t as_stream(bnn_stream_t s) { return reinterpret_cast<hipStream_t>(s); }
bnn_status from_hip(hipError_t e) { return e == hipSuccess ? BNN_OK : BNN_ERR_HIP; }

// Whether n steps of this stride (0 .. MAX_STRIDE) pass the 64-bit byte offsets of the kernels.
bool past(int64_t n, int64_t stride) { return n > 1 && stride > ((int64_t)1 << 60) / n; }

// Sizes, types and strides of a cache; its pointers too unless `sizes_only`.
bnn_status make_cache(const bnn_kv_cache* c, int64_t B, KvCache& k, bool sizes_only = false) {
    if (!c) return BNN_ERR_NULL;
    if (c->dtype != BNN_BF16 && c->dtype != BNN_F16) return BNN_ERR_UNSUPPORTED;
    if (c->dim != 64 && c->dim != 96 && c->dim != 128 && c->dim != 256) return BNN_ERR_UNSUPPORTED;
    if (c->page_size < 1 || c->page_size > MAX_SLOTS || c->num_pages < 0 || c->num_pages > INT32_MAX) return BNN_ERR_SHAPE;
    if (c->kv_heads < 1 || c->kv_heads > 65535 || B < 0 || B > 65535) return BNN_ERR_SHAPE;
    if (c->table && (c->ld_table < 1 || c->ld_table > MAX_SLOTS)) return BNN_ERR_LD;
    if (B * c->kv_heads > ((int64_t)1 << 28)) return BNN_ERR_SHAPE;
    const int64_t capacity = c->table ? c->ld_table * c->page_size : c->page_size;   // below 2^60
    if (capacity > MAX_SLOTS) return BNN_ERR_SHAPE;
    if (!sizes_only) {
        if (!c->K || !c->V) return BNN_ERR_NULL;
        if (misaligned(c->K, 16) || misaligned(c->V, 16) || (c->table && misaligned(c->table, 4))) return BNN_ERR_ALIGN;
        for (const int64_t s : {c->k_page, c->k_slot, c->k_head, c->v_page, c->v_slot, c->v_head})
            if (s < 0 || s > MAX_STRIDE) return BNN_ERR_LD;
        if (past(c->num_pages, c->k_page) || past(c->num_pages, c->v_page)) return BNN_ERR_LD;
        for (const int64_t s : {c->k_page, c->k_slot, c->k_head, c->v_page, c->v_slot, c->v_head})
            if (s % 8 != 0) return BNN_ERR_ALIGN;
    }
    k.K = (char*)c->K; k.k_page = 2 * c->k_page; k.k_slot = 2 * c->k_slot; k.k_head = 2 * c->k_head;
    k.V = (char*)c->V; k.v_page = 2 * c->v_page; k.v_slot = 2 * c->v_slot; k.v_head = 2 * c->v_head;
    k.table = c->table; k.ld_table = c->ld_table;
    k.num_pages = (uint32_t)c->num_pages;
    k.page = bnn::make_fastdiv((uint32_t)c->page_size);
    k.capacity = (int32_t)capacity;
    k.kv_heads = (int32_t)c->kv_heads;
    k.dim = (int32_t)c->dim;
    return BNN_OK;
}

bnn_status make_batch(const bnn_kv_batch* b, KvBatch& k, bool sizes_only = false) {
    if (!b) return BNN_ERR_NULL;
    if (b->B < 0 || b->B > 65535 || b->rows < 0 || b->rows > MAX_SLOTS) return BNN_ERR_SHAPE;
    if (b->max_nodes < 0 || b->max_nodes > MAX_SLOTS || b->max_ctx < 0 || b->max_ctx > MAX_SLOTS) return BNN_ERR_SHAPE;
    if (!sizes_only) {
        if (!b->indptr || !b->ctx) return BNN_ERR_NULL;
        if (misaligned(b->indptr, 4) || misaligned(b->ctx, 4)) return BNN_ERR_ALIGN;
    }
    k.indptr = b->indptr; k.ctx = b->ctx;
    k.B = (int32_t)b->B; k.rows = (int32_t)b->rows;
    k.max_nodes = (int32_t)(b->max_nodes < b->rows ? b->max_nodes : b->rows);
    k.max_ctx = (int32_t)b->max_ctx;
    return BNN_OK;
}

bnn_status check_heads(int64_t heads, int64_t kv_heads) {
    if (heads < 1 || heads > 65535) return BNN_ERR_SHAPE;
    return heads % kv_heads == 0 ? BNN_OK : BNN_ERR_SHAPE;
}

// A token tensor [rows, heads, dim] whose rows are read or written in pieces
// of `unit` elements, the first at an address that is a multiple of `align` bytes.
bnn_status check_rows(const void* p, int64_t rows, int64_t row, int64_t head, int64_t unit, int64_t align) {
    if (!p) return BNN_ERR_NULL;
    if (row < 0 || row > MAX_STRIDE || head < 0 || head > MAX_STRIDE || past(rows, row)) return BNN_ERR_LD;
    if (row % unit != 0 || head % unit != 0 || misaligned(p, (uintptr_t)align)) return BNN_ERR_ALIGN;
    return BNN_OK;
}

bnn_status check_packed_rows(const uint32_t* p, int64_t ld) {
    if (!p) return BNN_OK;
    if (ld < 1 || ld > MAX_SLOTS) return BNN_ERR_LD;
    return misaligned(p, 4) ? BNN_ERR_ALIGN : BNN_OK;
}

bnn_status check_work(const void* p, int64_t have, int64_t need) {
    if (need == 0) return BNN_OK;
    if (!p) return BNN_ERR_NULL;
    if (misaligned(p, 16)) return BNN_ERR_ALIGN;
    return have < need ? BNN_ERR_SHAPE : BNN_OK;
}

}  // namespace

#define BNN_TRY(x) do { const bnn_status st_ = (x); if (st_ != BNN_OK) return st_; } while (0)

#pragma GCC visibility push(default)
extern "C" {

bnn_status bnn_qk_norm_rope(const bnn_kv_cache* cache, const bnn_kv_batch* batch, const bnn_rope_args* a, bnn_stream_t stream) {
    if (!cache || !batch || !a) return BNN_ERR_NULL;
    KvCache c;
    KvBatch b;
    BNN_TRY(make_batch(batch, b));
    BNN_TRY(make_cache(cache, batch->B, c));
    if (a->heads < 1 || a->heads > 65535) return BNN_ERR_SHAPE;
    if (a->src_dtype != BNN_F32 && a->src_dtype != cache->dtype) return BNN_ERR_UNSUPPORTED;
    if (a->rot < 0 || a->rot > cache->dim) return BNN_ERR_SHAPE;
    if (a->rot % 8 != 0) return BNN_ERR_UNSUPPORTED;
    const int64_t bytes = a->src_dtype == BNN_F32 ? 4 : 2;
    BNN_TRY(check_rows(a->q, b.rows, a->q_row, a->q_head, 4, 4 * bytes));
    BNN_TRY(check_rows(a->k, b.rows, a->k_row, a->k_head, 4, 4 * bytes));
    BNN_TRY(check_rows(a->v, b.rows, a->v_row, a->v_head, 4, 4 * bytes));
    BNN_TRY(check_rows(a->q_out, b.rows, a->qo_row, a->qo_head, 8, 16));
    if (!a->positions) return BNN_ERR_NULL;
    if (misaligned(a->positions, 4)) return BNN_ERR_ALIGN;
    if (a->rot > 0) {
        if (!a->turns) return BNN_ERR_NULL;
        if (a->max_pos < 0 || a->max_pos > MAX_SLOTS) return BNN_ERR_SHAPE;
        if (misaligned(a->turns, 16)) return BNN_ERR_ALIGN;
    }
    if (misaligned(a->q_weight, 16) || misaligned(a->k_weight, 16)) return BNN_ERR_ALIGN;
    if ((a->q_weight || a->k_weight) && !(a->eps >= 0.f)) return BNN_ERR_UNSUPPORTED;
    if (a->pos || a->score) {
        if (a->ld_slots < c.capacity) return BNN_ERR_LD;
        if (misaligned(a->pos, 4) || misaligned(a->score, 4)) return BNN_ERR_ALIGN;
    }
    if (b.rows == 0 || b.B == 0) return BNN_OK;
    bnn::RopeArgs r;
    r.q = (const char*)a->q; r.q_row = bytes * a->q_row; r.q_head = bytes * a->q_head;
    r.k = (const char*)a->k; r.k_row = bytes * a->k_row; r.k_head = bytes * a->k_head;
    r.v = (const char*)a->v; r.v_row = bytes * a->v_row; r.v_head = bytes * a->v_head;
    r.heads = (int32_t)a->heads;
    r.qo = (char*)a->q_out; r.qo_row = 2 * a->qo_row; r.qo_head = 2 * a->qo_head;
    r.positions = a->positions;
    r.turns = a->turns; r.max_pos = (int32_t)a->max_pos; r.rot = (int32_t)a->rot;
    r.qw = a->q_weight; r.kw = a->k_weight; r.eps = a->eps;
    r.pos = a->pos; r.score = a->score; r.ld_slots = a->ld_slots;
    return from_hip(bnn::launch_qk_norm_rope(c, b, r, cache->dtype, a->src_dtype, a->interleaved != 0, as_stream(stream)));
}

bnn_status bnn_rope_turns_host(int64_t max_pos, int64_t rot, double base, int32_t kind, double factor, double old_ctx,
                               double beta_fast, double beta_slow, float* turns) {
    if (!turns) return BNN_ERR_NULL;
    if (max_pos < 0 || max_pos > MAX_SLOTS || rot < 2 || rot > 65536 || rot % 2 != 0) return BNN_ERR_SHAPE;
    if (!(base > 1.0) || !isfinite(base) || !(factor >= 1.0) || !isfinite(factor)) return BNN_ERR_UNSUPPORTED;
    if (kind < BNN_ROPE_PLAIN || kind > BNN_ROPE_BANDS) return BNN_ERR_UNSUPPORTED;
    const bool parts = kind == BNN_ROPE_RAMP || kind == BNN_ROPE_BANDS;
    if (parts && (!(old_ctx > 0.0) || !(beta_slow > 0.0) || !(beta_fast > beta_slow))) return BNN_ERR_UNSUPPORTED;
    if (kind == BNN_ROPE_BASE && rot == 2) return BNN_ERR_UNSUPPORTED;
    const double two_pi = 6.283185307179586476925286766559;
    const int64_t half = rot / 2;
    const double b = kind == BNN_ROPE_BASE ? base * pow(factor, (double)rot / (double)(rot - 2)) : base;
    const double gain = kind == BNN_ROPE_RAMP && factor > 1.0 ? 0.1 * log(factor) + 1.0 : 1.0;
    // the pair index that turns beta times over old_ctx
    const auto pair_of = [&](double beta) { return rot * log(old_ctx / (beta * two_pi)) / (2.0 * log(base)); };
    double lo = 0, hi = 0;
    if (kind == BNN_ROPE_RAMP) {
        lo = fmax(floor(pair_of(beta_fast)), 0.0);
        hi = fmin(ceil(pair_of(beta_slow)), (double)(rot - 1));
        if (hi <= lo) hi = lo + 0.001;
    }
    for (int64_t i = 0; i < half; ++i) {
        double theta = pow(b, -2.0 * (double)i / (double)rot);
        if (kind == BNN_ROPE_LINEAR) theta /= factor;
        if (parts) {
            double keep;   // share of the unscaled angle
            if (kind == BNN_ROPE_RAMP) keep = 1.0 - fmin(fmax(((double)i - lo) / (hi - lo), 0.0), 1.0);
            else keep = fmin(fmax((old_ctx * theta / two_pi - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0);
            theta = theta * keep + theta / factor * (1.0 - keep);
        }
        for (int64_t p = 0; p < max_pos; ++p) {
            turns[p * rot + i] = (float)(gain * cos((double)p * theta));
            turns[p * rot + half + i] = (float)(gain * sin((double)p * theta));
        }
    }
    return BNN_OK;
}

bnn_status bnn_tree_mask_host(const int32_t* parent, int64_t T, uint32_t* mask, int64_t ld) {
    if (T < 0 || T > MAX_SLOTS) return BNN_ERR_SHAPE;
    if (!parent || !mask) return BNN_ERR_NULL;
    if (ld < (T + 31) / 32) return BNN_ERR_LD;
    for (int64_t i = 0; i < T; ++i)
        if (parent[i] < -1 || parent[i] >= i) return BNN_ERR_UNSUPPORTED;
    for (int64_t i = 0; i < T; ++i) {
        uint32_t* row = mask + i * ld;
        for (int64_t w = 0; w < ld; ++w) row[w] = parent[i] < 0 ? 0u : mask[parent[i] * ld + w];
        row[i >> 5] |= 1u << (i & 31);
    }
    return BNN_OK;
}

int64_t bnn_tree_attention_workspace(const bnn_kv_cache* cache, const bnn_kv_batch* batch, int64_t heads) {
    if (!cache || !batch) return -1;
    KvCache c;
    KvBatch b;
    if (make_batch(batch, b, true) != BNN_OK || make_cache(cache, batch->B, c, true) != BNN_OK) return -1;
    if (check_heads(heads, c.kv_heads) != BNN_OK) return -1;
    return bnn::tree_attention_work(c, b, (int32_t)heads);
}

bnn_status bnn_tree_attention(const bnn_kv_cache* cache, const bnn_kv_batch* batch, const bnn_attn_args* a, bnn_stream_t stream) {
    if (!cache || !batch || !a) return BNN_ERR_NULL;
    KvCache c;
    KvBatch b;
    BNN_TRY(make_batch(batch, b));
    BNN_TRY(make_cache(cache, batch->B, c));
    BNN_TRY(check_heads(a->heads, c.kv_heads));
    if (a->out_dtype != BNN_F32 && a->out_dtype != cache->dtype) return BNN_ERR_UNSUPPORTED;
    if (!isfinite(a->scale)) return BNN_ERR_UNSUPPORTED;
    BNN_TRY(check_rows(a->q, b.rows, a->q_row, a->q_head, 8, 16));
    BNN_TRY(check_packed_rows(a->mask, a->ld_mask));
    const int64_t obytes = a->out_dtype == BNN_F32 ? 4 : 2;
    BNN_TRY(check_rows(a->out, b.rows, a->o_row, a->o_head, 8, 16));
    if (a->lse) {
        if (a->ld_lse < a->heads) return BNN_ERR_LD;
        if (misaligned(a->lse, 4)) return BNN_ERR_ALIGN;
    }
    if (a->workspace_bytes < 0) return BNN_ERR_SHAPE;
    BNN_TRY(check_work(a->workspace, a->workspace_bytes, a->workspace_bytes));
    if (!bnn::tree_attention_fits(c, b, (int32_t)a->heads, a->workspace_bytes)) return BNN_ERR_SHAPE;   // more workgroups than a launch takes
    if (b.rows == 0 || b.B == 0 || b.max_nodes == 0) return BNN_OK;
    bnn::AttnArgs r;
    r.q = (const char*)a->q; r.q_row = 2 * a->q_row; r.q_head = 2 * a->q_head;
    r.heads = (int32_t)a->heads; r.group = (int32_t)(a->heads / c.kv_heads);
    r.mask = a->mask; r.ld_mask = a->ld_mask;
    r.scale = a->scale;
    r.out = (char*)a->out; r.o_row = obytes * a->o_row; r.o_head = obytes * a->o_head;
    r.lse = a->lse; r.ld_lse = a->ld_lse;
    r.work = (char*)a->workspace; r.work_bytes = a->workspace_bytes;
    return from_hip(bnn::launch_tree_attention(c, b, r, cache->dtype, a->out_dtype, as_stream(stream)));
}

bnn_status bnn_cache_score_add(const bnn_kv_cache* cache, const bnn_kv_batch* batch, const bnn_score_args* a, bnn_stream_t stream) {
    if (!cache || !batch || !a) return BNN_ERR_NULL;
    KvCache c;
    KvBatch b;
    BNN_TRY(make_batch(batch, b));
    BNN_TRY(make_cache(cache, batch->B, c));
    BNN_TRY(check_heads(a->heads, c.kv_heads));
    if (!isfinite(a->scale)) return BNN_ERR_UNSUPPORTED;
    BNN_TRY(check_rows(a->q, b.rows, a->q_row, a->q_head, 8, 16));
    BNN_TRY(check_packed_rows(a->mask, a->ld_mask));
    BNN_TRY(check_packed_rows(a->accept, a->ld_accept));
    if (!a->lse || !a->score_in || !a->score_out) return BNN_ERR_NULL;
    if (a->ld_lse < a->heads || a->ld_slots < c.capacity) return BNN_ERR_LD;
    if (misaligned(a->lse, 4) || misaligned(a->score_in, 4) || misaligned(a->score_out, 4)) return BNN_ERR_ALIGN;
    if (b.B == 0) return BNN_OK;
    bnn::ScoreArgs r;
    r.q = (const char*)a->q; r.q_row = 2 * a->q_row; r.q_head = 2 * a->q_head;
    r.heads = (int32_t)a->heads; r.group = (int32_t)(a->heads / c.kv_heads);
    r.lse = a->lse; r.ld_lse = a->ld_lse;
    r.mask = a->mask; r.ld_mask = a->ld_mask;
    r.accept = a->accept; r.ld_accept = a->ld_accept;
    r.scale = a->scale;
    r.in = a->score_in; r.out = a->score_out; r.ld_slots = a->ld_slots;
    return from_hip(bnn::launch_cache_score_add(c, b, r, cache->dtype, as_stream(stream)));
}

int64_t bnn_cache_evict_workspace(const bnn_kv_cache* cache, int64_t B) {
    KvCache c;
    if (make_cache(cache, B, c, true) != BNN_OK) return -1;
    return B * c.kv_heads * bnn::evict_work_words(c.capacity) * 4;   // at most 2^28 heads of 2^32 bytes and a little
}

bnn_status bnn_cache_evict(const bnn_kv_cache* cache, const bnn_kv_batch* batch, const bnn_evict_args* a, bnn_stream_t stream) {
    if (!cache || !batch || !a) return BNN_ERR_NULL;
    KvCache c;
    KvBatch b;
    BNN_TRY(make_batch(batch, b));
    BNN_TRY(make_cache(cache, batch->B, c));
    BNN_TRY(check_packed_rows(a->accept, a->ld_accept));
    if (a->budget < 0 || a->recent < 0) return BNN_ERR_SHAPE;
    if (!a->pos_in || !a->pos_out || !a->score_in || !a->score_out || !a->ctx_out) return BNN_ERR_NULL;
    if (a->ld_slots < c.capacity) return BNN_ERR_LD;
    if (misaligned(a->pos_in, 4) || misaligned(a->pos_out, 4) || misaligned(a->score_in, 4) || misaligned(a->score_out, 4) ||
        misaligned(a->ctx_out, 4))
        return BNN_ERR_ALIGN;
    BNN_TRY(check_work(a->workspace, a->workspace_bytes, bnn_cache_evict_workspace(cache, batch->B)));
    if (b.B == 0) return BNN_OK;
    bnn::EvictArgs r;
    r.accept = a->accept; r.ld_accept = a->ld_accept;
    r.budget = (int32_t)(a->budget < INT32_MAX ? a->budget : INT32_MAX);
    r.recent = (int32_t)(a->recent < INT32_MAX ? a->recent : INT32_MAX);
    r.pos_in = a->pos_in; r.pos_out = a->pos_out;
    r.score_in = a->score_in; r.score_out = a->score_out;
    r.ld_slots = a->ld_slots;
    r.ctx_out = a->ctx_out;
    r.work = (int32_t*)a->workspace;
    return from_hip(bnn::launch_cache_evict(c, b, r, as_stream(stream)));
}

}  // extern "C"
#pragma GCC visibility pop
