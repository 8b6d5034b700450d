// Rejected drafts out of the cache, and the cache cut to a budget.
//
// A first kernel, one workgroup per (sequence, key head), finds which tokens
// stay.  Scores become 32-bit keys in the same order (a recent token takes
// the highest key, NaN that of -inf); the key of the last token that stays is
// found bit by bit from the top, counting the tokens at or above each trial
// key.  Then one walk over the slots in order settles ties (the lowest slots
// first) and pairs the free slots below the new length with the kept tokens
// above it.  Sources are all at or above the new length and destinations all
// below it, so a second kernel moves K and V rows in any order.
#include <math.h>

#include "bnn_device.hpp"
#include "kv_launch.hpp"

namespace bnn {
namespace {

constexpr int EV = 1024;   // threads of the selecting workgroup

// Monotone in the score; -0 as +0, NaN as -inf.  0xFFFFFFFF is left for recent tokens.
__device__ __forceinline__ uint32_t score_key(float x) {
    x = x != x ? -INFINITY : x + 0.0f;
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

// Sum over the workgroup, the same in every thread.  part: EV / 64 words.
__device__ __forceinline__ int block_sum(int v, int* part) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int i = 0; i < EV / 64; ++i) s += part[i];
    return s;
}

__device__ __forceinline__ int block_max(int v, int* part) {
#pragma unroll
    for (int m = 32; m; m >>= 1) { const int o = __shfl_xor(v, m, 64); v = o > v ? o : v; }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    int s = part[0];
#pragma unroll
    for (int i = 1; i < EV / 64; ++i) s = part[i] > s ? part[i] : s;
    return s;
}

// Number of threads before this one whose flag is set, and the total.
__device__ __forceinline__ int block_rank(bool flag, int* part, int& total) {
    const uint64_t m = __ballot(flag);
    const int w = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[w] = __popcll(m);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < EV / 64; ++i) { before += i < w ? part[i] : 0; all += part[i]; }
    total = all;
    return before + __popcll(m & ((1ull << (threadIdx.x & 63)) - 1));
}

__global__ __launch_bounds__(EV) void k_evict_select(KvCache c, KvBatch b, EvictArgs a) {
    __shared__ int part[EV / 64];
    const int kh = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x;
    const Seq sq = sequence(c, b, seq);
    const int64_t at = ((int64_t)seq * c.kv_heads + kh) * a.ld_slots;
    const float* score = a.score_in + at;
    const int32_t* pos = a.pos_in + at;
    auto valid = [&](int s) {
        return s < sq.ctx || (s < sq.total && (!a.accept || packed_bit(a.accept + seq * a.ld_accept, a.ld_accept, s - sq.ctx)));
    };
    int n = 0, last = INT32_MIN;
    for (int s = tid; s < sq.total; s += EV)
        if (valid(s)) { ++n; last = pos[s] > last ? pos[s] : last; }
    n = block_sum(n, part);
    last = block_max(last, part);
    const int keep = n < a.budget ? n : a.budget;
    const int64_t since = (int64_t)last - a.recent;
    auto key = [&](int s) { return pos[s] > since ? 0xFFFFFFFFu : score_key(score[s]); };

    // the largest key that at least keep tokens reach
    uint32_t edge = 0;
    int above = 0;   // tokens above it
    if (keep < n && keep > 0) {
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t trial = edge | (1u << bit);
            int cnt = 0;
            for (int s = tid; s < sq.total; s += EV) cnt += valid(s) && key(s) >= trial;
            cnt = block_sum(cnt, part);
            if (cnt >= keep) edge = trial;
        }
        int cnt = 0;
        for (int s = tid; s < sq.total; s += EV) cnt += valid(s) && key(s) > edge;
        above = block_sum(cnt, part);
    }
    const int ties = keep - above;   // of the tokens at the edge, the first ones

    int32_t* work = a.work + ((int64_t)seq * c.kv_heads + kh) * evict_work_words(c.capacity);
    int32_t* from = work + 16;
    int32_t* to = from + evict_work_words(c.capacity) / 2 - 8;
    int tied = 0, holes = 0, movers = 0;
    for (int s0 = 0; s0 < sq.total; s0 += EV) {
        const int s = s0 + tid;
        bool kept = valid(s);
        bool tie = false;
        if (kept && keep < n) {
            const uint32_t k = keep > 0 ? key(s) : 0;
            tie = keep > 0 && k == edge;
            kept = keep > 0 && k > edge;
        }
        int count;
        const int r = block_rank(tie, part, count);
        kept = kept || (tie && tied + r < ties);
        tied += count;
        const bool hole = s < keep && !kept, mover = s >= keep && kept;
        const int rh = block_rank(hole, part, count);
        if (hole) to[holes + rh] = s;
        holes += count;
        const int rm = block_rank(mover, part, count);
        if (mover) from[movers + rm] = s;
        movers += count;
    }
    __syncthreads();
    __threadfence_block();
    for (int s = tid; s < keep; s += EV) {
        a.pos_out[at + s] = pos[s];
        a.score_out[at + s] = score[s];
    }
    __syncthreads();
    for (int i = tid; i < movers; i += EV) {
        a.pos_out[at + to[i]] = pos[from[i]];
        a.score_out[at + to[i]] = score[from[i]];
    }
    __syncthreads();
    for (int s = keep + tid; s < sq.total; s += EV) {
        a.pos_out[at + s] = -1;
        a.score_out[at + s] = 0.f;
    }
    if (tid == 0) { work[0] = movers; work[1] = keep; }
}

__global__ __launch_bounds__(256) void k_evict_move(KvCache c, EvictArgs a) {
    const int kh = blockIdx.y, seq = blockIdx.z, units = c.dim / 8;
    const int32_t* work = a.work + ((int64_t)seq * c.kv_heads + kh) * evict_work_words(c.capacity);
    const int32_t* from = work + 16;
    const int32_t* to = from + evict_work_words(c.capacity) / 2 - 8;
    const int64_t n = (int64_t)work[0] * units;
    if (blockIdx.x == 0 && kh == 0 && threadIdx.x == 0) a.ctx_out[seq] = work[1];
    for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
        const int m = (int)(i / units), u = (int)(i % units);
        uint32_t sp, dp;
        const int32_t spg = slot_page(c, seq, from[m], sp), dpg = slot_page(c, seq, to[m], dp);
        if (spg < 0 || dpg < 0) continue;
        *(u32x4*)(c.K + dpg * c.k_page + dp * c.k_slot + kh * c.k_head + u * 16) =
            *(const u32x4*)(c.K + spg * c.k_page + sp * c.k_slot + kh * c.k_head + u * 16);
        *(u32x4*)(c.V + dpg * c.v_page + dp * c.v_slot + kh * c.v_head + u * 16) =
            *(const u32x4*)(c.V + spg * c.v_page + sp * c.v_slot + kh * c.v_head + u * 16);
    }
}

}  // namespace

hipError_t launch_cache_evict(const KvCache& c, const KvBatch& b, const EvictArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_evict_select, dim3(c.kv_heads, b.B), dim3(EV), 0, s, c, b, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t rows = (int64_t)b.max_ctx + b.max_nodes;
    int64_t most = a.budget < rows ? a.budget : rows;   // moves of a head
    if (rows - most < most && rows - most > 0) most = rows - most;
    int64_t blocks = (most * (c.dim / 8) + 255) / 256;
    if (blocks < 1) blocks = 1;
    if (blocks > 4096) blocks = 4096;
    hipLaunchKernelGGL(k_evict_move, dim3((unsigned)blocks, c.kv_heads, b.B), dim3(256), 0, s, c, a);
    return hipGetLastError();
}

}  // namespace bnn
