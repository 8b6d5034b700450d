// Tree attention: how a call is cut into workgroups, and its dispatch.
#include "attn_kernel.hpp"

namespace bnn {
namespace {

constexpr int64_t WANT = 512;    // workgroups
constexpr int64_t LONG = 2048;   // slots of a chunk at most, up to 64 rows

int64_t slots_of(const KvCache& c, const KvBatch& b) {
    const int64_t bound = (int64_t)b.max_ctx + b.max_nodes;
    return bound < c.capacity ? bound : c.capacity;
}

// Slots of whole steps, whatever the variant.
int64_t unit_of(int64_t tile) { return tile == 128 ? 256 : 128; }

// Rows per (sequence, key head) decide the workgroup: up to 16 or 32 rows one
// row tile whose waves share out the slots, above that row tiles of 64 or 128
// whose waves share the fetched K and V.  work_bytes bounds the chunks, whose
// partial results it holds; one needs none.
AttnPlan make_plan(const KvCache& c, const KvBatch& b, int32_t heads, int64_t work_bytes) {
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
    const int64_t slots = slots_of(c, b), unit = unit_of(tile);
    // About the 512 workgroups that are resident at once (256 compute units, 2 each): twice as many cost the
    // compute-bound cases 7 to 17% (the partial results of more chunks are written and read again).  Streaming
    // cases keep chunks of at most 2048 slots, so that sequences of unequal lengths balance.
    const int64_t heads_all = (int64_t)b.B * kv_heads * tiles;
    int64_t want = heads_all > 0 ? (WANT + heads_all / 2) / heads_all : 1;
    if (want < 1) want = 1;
    int64_t chunk = (slots + want - 1) / want;
    chunk = (chunk + unit - 1) / unit * unit;
    if (chunk < unit) chunk = unit;
    if (chunk > LONG && p.RW < 4) chunk = LONG;
    if ((slots + chunk - 1) / chunk > 1) {
        const int64_t one = part_rows(b.rows, heads) * (dim * 4 + 8);   // bytes of one chunk's
        const int64_t most = one > 0 && work_bytes / one > 1 ? work_bytes / one : 1;
        if ((slots + chunk - 1) / chunk > most) chunk = ((slots + most - 1) / most + unit - 1) / unit * unit;
    }
    p.chunk = (int32_t)chunk;
    p.chunks = (int32_t)((slots + chunk - 1) / chunk);
    if (p.chunks < 1) p.chunks = 1;
    const int64_t groups = (int64_t)b.B * kv_heads * p.chunks;
    // -1: more rows or workgroups than the kernel counts
    p.groups = rows < 0x7FFFFFFF - tile && groups < 0x7FFFFFFF / 16 && (groups + 8) * tiles < 0x7FFFFFFF ? (int32_t)groups : -1;
    return p;
}

}  // namespace

bool tree_attention_fits(const KvCache& c, const KvBatch& b, int32_t heads, int64_t work_bytes) {
    return make_plan(c, b, heads, work_bytes).groups >= 0;
}

// Chunks are made for about WANT workgroups, so calls of fewer sequences or
// tokens have more of them, over fewer rows.  What is returned covers, besides
// this call, every smaller one whose rows are its sequences' new tokens at most:
// with x = B kv_heads row_tiles it has (WANT + x / 2) / x chunks or one for each
// LONG slots, whichever is more.  Its rows are B nodes <= x tile / heads, so the
// former give at most (WANT + x / 2) tile / heads partial rows, with x at most
// 2 WANT / 3 where there are two chunks.
int64_t tree_attention_work(const KvCache& c, const KvBatch& b, int32_t heads) {
    if (b.B == 0 || b.rows == 0 || b.max_nodes == 0) return 0;
    const AttnPlan p = make_plan(c, b, heads, INT64_MAX);
    if (p.groups < 0) return -1;
    const int64_t group = heads / c.kv_heads, rows_most = b.max_nodes * group, slots = slots_of(c, b);
    const int64_t row_bytes = (int64_t)heads * (c.dim * 4 + 8);
    int64_t need = p.chunks == 1 ? 0 : p.chunks * b.rows * row_bytes;
    for (const int64_t tile : {16, 32, 64, 128}) {
        if (tile > 16 && rows_most <= tile / 2) break;   // a smaller tile holds all rows
        int64_t nodes = tile == 128 ? b.max_nodes : tile / group;   // of a sequence, where this tile is taken
        if (nodes > b.max_nodes) nodes = b.max_nodes;
        const int64_t rows = b.B * nodes < b.rows ? b.B * nodes : b.rows;
        const int64_t most = (slots + unit_of(tile) - 1) / unit_of(tile);
        if (most <= 1) continue;
        int64_t wanted = WANT / c.kv_heads + 1;
        if (wanted > most) wanted = most;
        int64_t parts = (WANT + WANT / 3) * tile / heads + 1;
        if (parts > rows * wanted) parts = rows * wanted;
        const int64_t by_length = tile < 128 ? rows * ((slots + LONG - 1) / LONG) : 0;
        if (parts < by_length) parts = by_length;
        if (parts * row_bytes > need) need = parts * row_bytes;
    }
    return need;
}

hipError_t launch_tree_attention(const KvCache& c, const KvBatch& b, const AttnArgs& a, int32_t dtype, int32_t out_dtype,
                                 hipStream_t s) {
    const AttnPlan p = make_plan(c, b, a.heads, a.work_bytes);
    if (dtype == KV_BF16) return out_dtype == KV_F32 ? attn_bf16_f32(c, b, a, p, s) : attn_bf16(c, b, a, p, s);
    return out_dtype == KV_F32 ? attn_f16_f32(c, b, a, p, s) : attn_f16(c, b, a, p, s);
}

}  // namespace bnn
