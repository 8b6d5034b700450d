// Host-side launchers of the kernels over the key/value cache (internal to
// libbnn).  kv_api.hip validates every argument before calling these.
#pragma once

#include "kv.hpp"

namespace bnn {

enum : int32_t { KV_BF16 = 1, KV_F16 = 2, KV_F32 = 3 };

struct RopeArgs {
    const char* q; int64_t q_row, q_head;   // strides in bytes
    const char* k; int64_t k_row, k_head;
    const char* v; int64_t v_row, v_head;
    int32_t heads;
    char* qo; int64_t qo_row, qo_head;
    const int32_t* positions;
    const float* turns; int32_t max_pos, rot;
    const float* qw; const float* kw;
    float eps;
    int32_t* pos; float* score; int64_t ld_slots;
};

hipError_t launch_qk_norm_rope(const KvCache& c, const KvBatch& b, const RopeArgs& a, int32_t dtype, int32_t src_dtype,
                               bool interleaved, hipStream_t s);

struct AttnArgs {
    const char* q; int64_t q_row, q_head;   // strides in bytes
    int32_t heads, group;
    const uint32_t* mask; int64_t ld_mask;
    float scale;
    char* out; int64_t o_row, o_head;       // strides in bytes
    float* lse; int64_t ld_lse;
    char* work; int64_t work_bytes;
};

bool tree_attention_fits(const KvCache& c, const KvBatch& b, int32_t heads, int64_t work_bytes);   // a launch takes the grid
// Workspace bytes; -1 where a launch would not take the grid.
int64_t tree_attention_work(const KvCache& c, const KvBatch& b, int32_t heads);
hipError_t launch_tree_attention(const KvCache& c, const KvBatch& b, const AttnArgs& a, int32_t dtype, int32_t out_dtype,
                                 hipStream_t s);

struct ScoreArgs {
    const char* q; int64_t q_row, q_head;   // strides in bytes
    int32_t heads, group;
    const float* lse; int64_t ld_lse;
    const uint32_t* mask; int64_t ld_mask;
    const uint32_t* accept; int64_t ld_accept;
    float scale;
    const float* in; float* out; int64_t ld_slots;
};

hipError_t launch_cache_score_add(const KvCache& c, const KvBatch& b, const ScoreArgs& a, int32_t dtype, hipStream_t s);

struct EvictArgs {
    const uint32_t* accept; int64_t ld_accept;
    int32_t budget, recent;
    const int32_t* pos_in; int32_t* pos_out;
    const float* score_in; float* score_out;
    int64_t ld_slots;
    int32_t* ctx_out;
    int32_t* work;
};

// Workspace of a (sequence, key head) in 32-bit words.
__host__ __device__ inline int64_t evict_work_words(int64_t capacity) { return (capacity + 3) / 4 * 4 + 16; }
hipError_t launch_cache_evict(const KvCache& c, const KvBatch& b, const EvictArgs& a, hipStream_t s);

}  // namespace bnn
