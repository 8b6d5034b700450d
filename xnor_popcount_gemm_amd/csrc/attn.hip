// Tree attention: how a call is cut into workgroups, and its dispatch.
#include "attn_kernel.hpp"

namespace bnn {
namespace {

// Rows per (sequence, key head) decide the workgroup: up to 16 or 32 rows one
// row tile whose waves share out the slots, above that row tiles of 64 or 128
// whose waves share the fetched K and V.
AttnPlan make_plan(const KvCache& c, const KvBatch& b, int32_t heads) {
    const int32_t dim = c.dim, kv_heads = c.kv_heads;
    AttnPlan p;
    const int64_t rows = (int64_t)b.max_nodes * (heads / kv_heads);
    const int32_t kw = dim == 256 ? 2 : 4;
    if (rows <= 16) { p.R = 16; p.RW = 1; p.KW = kw; }
    else if (rows <= 32) { p.R = 32; p.RW = 1; p.KW = kw; }
    else if (rows <= 64) { p.R = 32; p.RW = 2; p.KW = 2; }
    else { p.R = 32; p.RW = 4; p.KW = 1; }
    const int64_t tile = p.R * p.RW;
    const int64_t tiles = (rows + tile - 1) / tile;
    p.row_tiles = (int32_t)tiles;
    const int64_t bound = (int64_t)b.max_ctx + b.max_nodes, slots = bound < c.capacity ? bound : c.capacity;
    const int64_t unit = p.RW == 4 ? 256 : 128;      // slots of whole steps, whatever the variant
    // About the 512 workgroups that are resident at once (256 compute units, 2 each): twice as many cost the
    // compute-bound cases 7 to 17% (the partial results of more chunks are written and read again).  Streaming
    // cases keep chunks of at most 2048 slots, so that sequences of unequal lengths balance.
    const int64_t heads_all = (int64_t)b.B * kv_heads * tiles;
    int64_t want = heads_all > 0 ? (512 + heads_all / 2) / heads_all : 1;
    if (want < 1) want = 1;
    int64_t chunk = (slots + want - 1) / want;
    chunk = (chunk + unit - 1) / unit * unit;
    if (chunk < unit) chunk = unit;
    if (chunk > 2048 && p.RW < 4) chunk = 2048;
    p.chunk = (int32_t)chunk;
    p.chunks = (int32_t)((slots + chunk - 1) / chunk);
    if (p.chunks < 1) p.chunks = 1;
    const int64_t groups = (int64_t)b.B * kv_heads * p.chunks;
    p.groups = groups < 0x7FFFFFFF / 16 && (groups + 8) * tiles < 0x7FFFFFFF ? (int32_t)groups : -1;   // -1: past one launch
    return p;
}

}  // namespace

int64_t tree_attention_work(const KvCache& c, const KvBatch& b, int32_t heads) {
    const AttnPlan p = make_plan(c, b, heads);
    if (p.groups < 0) return -1;
    return p.chunks == 1 ? 0 : (int64_t)p.chunks * b.rows * heads * (c.dim * 4 + 8);
}

hipError_t launch_tree_attention(const KvCache& c, const KvBatch& b, const AttnArgs& a, int32_t dtype, int32_t out_dtype,
                                 hipStream_t s) {
    const AttnPlan p = make_plan(c, b, a.heads);
    if (dtype == KV_BF16) return out_dtype == KV_F32 ? attn_bf16_f32(c, b, a, p, s) : attn_bf16(c, b, a, p, s);
    return out_dtype == KV_F32 ? attn_f16_f32(c, b, a, p, s) : attn_f16(c, b, a, p, s);
}

}  // namespace bnn
