// Rejected drafts out of the cache, and the cache cut to a budget.
//
// A first kernel, one workgroup per (sequence, key head), finds which tokens
// stay.  Scores become 32-bit keys in the same order (a recent token takes the
// highest key, NaN that of -inf).  The key of the last token that stays is
// found 8 bits at a time from the top, by a histogram of the tokens that share
// the bits found so far; each of its 256 counters has 32 copies, one per LDS
// bank, because scores cluster (a handful of exponents) and equal addresses of
// one LDS add run one after the other.  Keys are made once and stay in
// registers (up to 32 per thread; in LDS instead, 32000 slots took 58 us against
// 51); those of longer sequences are made again at each pass.  Ties go to the
// lowest slots.  Where recent tokens are among those that leave, they alone fill
// the new length, and the search is made again over them, by their scores.  The
// free slots below the new length are paired in order with the kept tokens above
// it: a wave owns a run of slots, so three joins of the waves' counts give every
// rank.
//
// Sources are all at or above the new length and destinations all below it, so
// a second kernel moves K and V rows (and positions and scores) in any order.
// It is bound by memory: 117 MB of reads and writes in 30 us, 3.9 TB/s, where a
// plain copy reaches 5.1.  The first kernel is bound by its passes in one
// workgroup per head: 13 us at 2048 slots, 50 at 32000.
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

// This wave's share joined with the others': the sum of the waves before it,
// and of all.  part: EV / 64 words of its own.
__device__ __forceinline__ int before_wave(int v, int* part, int& total) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[w] = v;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < EV / 64; ++i) { before += i < w ? part[i] : 0; all += part[i]; }
    total = all;
    return before;
}

struct EvictLds {
    uint32_t hist[256 * 32];
    uint32_t bins[256];
    int part[6][EV / 64];
};

// The highest of all threads' values.  part: EV / 64 words of its own.
__device__ __forceinline__ void block_max(int& last, int* part) {
#pragma unroll
    for (int m = 32; m; m >>= 1) { const int o = __shfl_xor(last, m, 64); last = o > last ? o : last; }
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = last;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EV / 64; ++i) last = part[i] > last ? part[i] : last;
}

// KPT: keys per thread that stay in registers; 0: any number, made again.
// Returns false, with nothing written, where KPT > 0 and recent tokens leave:
// keys of a second search beside the first's would not stay in registers (20 us
// more at 32000 slots for every call).
constexpr int BATCH = 16;
template <int KPT>
__device__ __forceinline__ bool evict_select(const KvCache& c, const EvictArgs& a, const Seq& sq, int seq, int kh, EvictLds& lds) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t at = ((int64_t)seq * c.kv_heads + kh) * a.ld_slots;
    const float* const score = a.score_in + at;
    const int32_t* const pos = a.pos_in + at;
    const int steps = (sq.total + EV - 1) / EV;     // of 64 slots, for each wave
    const int first = wave * steps * 64 + lane;     // this thread's slots: first + 64 i
    auto valid_at = [&](int s) {
        return s < sq.ctx || (s < sq.total && (!a.accept || packed_bit(a.accept + seq * a.ld_accept, a.ld_accept, s - sq.ctx)));
    };
    constexpr int N = KPT > 0 ? KPT : 1;
    const int mine = (wave + 1) * steps * 64 < sq.total ? (wave + 1) * steps * 64 : sq.total;   // end of the wave's slots
    auto valid_in_run = [&](int s) {
        bool v = s < mine;
        if (__any(v && s >= sq.ctx)) v = v && valid_at(s);
        return v;
    };
    uint32_t key[N], valid = 0;   // valid: bit i for slot first + 64 i
    int n = 0, last = INT32_MIN;
    if constexpr (KPT > 0) {
        int32_t p[N];
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const int s = first + 64 * i, in = s < mine ? s : 0;   // a lane past the end reads a slot that is there
            p[i] = sq.total ? pos[in] : 0;
            key[i] = __float_as_uint(sq.total ? score[in] : 0.f);
        }
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const bool v = valid_in_run(first + 64 * i);
            valid |= (uint32_t)v << i;
            n += __popcll(__ballot(v));
            last = v && p[i] > last ? p[i] : last;
        }
        block_max(last, lds.part[1]);
        const int64_t since = (int64_t)last - a.recent;
#pragma unroll
        for (int i = 0; i < KPT; ++i) key[i] = p[i] > since ? 0xFFFFFFFFu : score_key(__uint_as_float(key[i]));
    } else {
        for (int i0 = 0; i0 < steps; i0 += BATCH) {   // so many loads at a time
            int32_t p[BATCH];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int s = first + 64 * (i0 + j);
                p[j] = pos[s < mine ? s : 0];
            }
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const bool v = valid_in_run(first + 64 * (i0 + j));
                n += __popcll(__ballot(v));
                last = v && p[j] > last ? p[j] : last;
            }
        }
        block_max(last, lds.part[1]);
    }
    int all;
    before_wave(n, lds.part[0], all);
    n = all;
    const int keep = n < a.budget ? n : a.budget;
    const int64_t since = (int64_t)last - a.recent;
    const int low = keep < mine ? keep : mine;   // this wave's slots below the new length end here
    bool crowded = false;   // recent tokens leave: only they may stay, by score
    // f(i, slot, may stay, key) for this thread's slots, every thread of a wave alike
    auto each = [&](auto f) {
        if constexpr (KPT > 0) {
#pragma unroll
            for (int i = 0; i < KPT; ++i)
                f(i, first + 64 * i, (valid >> i & 1u) != 0, key[i]);
        } else {
            for (int i = 0; i < steps; ++i) {
                const int s = first + 64 * i;
                const bool v = valid_at(s), recent = v && pos[s] > since;
                f(i, s, crowded ? recent : v, !v ? 0u : recent && !crowded ? 0xFFFFFFFFu : score_key(score[s]));
            }
        }
    };

    // the largest key that at least keep tokens reach, and how many of its tokens stay
    uint32_t edge = 0;
    int ties = keep;
    const bool cut = keep < n && keep > 0;
    if (cut) {
        for (int shift = 24; shift >= 0;) {
            for (int i = tid; i < 256 * 32; i += EV) lds.hist[i] = 0;
            __syncthreads();
            each([&](int, int, bool v, uint32_t k) {
                if (v && (shift == 24 || k >> ((shift + 8) & 31) == edge >> ((shift + 8) & 31)))
                    atomicAdd(&lds.hist[(k >> shift & 255u) * 32 + (lane & 31)], 1u);
            });
            __syncthreads();
            {   // four threads per counter, eight copies each
                const int bin = tid >> 2;
                uint32_t t = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) t += lds.hist[bin * 32 + (tid & 3) * 8 + ((j + bin) & 7)];
                t += __shfl_xor(t, 1, 64);
                t += __shfl_xor(t, 2, 64);
                if ((tid & 3) == 0) lds.bins[bin] = t;
            }
            __syncthreads();
            // from the top: each lane takes four counters, lane 0 the highest
            uint32_t b4[4], mine = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) { b4[j] = lds.bins[255 - 4 * lane - j]; mine += b4[j]; }
            uint32_t upto = mine;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) { const uint32_t o = __shfl_up(upto, m, 64); upto += lane >= m ? o : 0u; }
            const int hit = __ffsll((unsigned long long)__ballot(upto >= (uint32_t)ties)) - 1;   // ties >= 1: some lane
            uint32_t above = upto - mine, digit = 0;
            bool found = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (!found && above + b4[j] >= (uint32_t)ties) { found = true; digit = 255 - 4 * lane - j; }
                if (!found) above += b4[j];
            }
            edge |= (uint32_t)__builtin_amdgcn_readlane(digit, hit) << shift;
            ties -= __builtin_amdgcn_readlane(above, hit);
            shift -= 8;
            if (shift < 0 && edge == 0xFFFFFFFFu && !crowded && lds.bins[255] > (uint32_t)ties) {
                if (KPT > 0) return false;
                crowded = true;
                shift = 24;
                edge = 0;
                ties = keep;
            }
        }
    }

    // which stay: bit i of a word per thread, or again where they are not in registers
    int tied = 0;
    if (cut) {
        int t = 0;
        each([&](int, int, bool v, uint32_t k) { t += __popcll(__ballot(v && k == edge)); });
        tied = before_wave(t, lds.part[2], all);
    }
    const uint64_t below = (1ull << lane) - 1;
    auto stays = [&](bool v, uint32_t k, int& tie) {
        if (!cut) return v && keep > 0;
        const uint64_t m = __ballot(v && k == edge);
        const bool s = v && (k > edge || (k == edge && tie + __popcll(m & below) < ties));
        tie += __popcll(m);
        return s;
    };
    int holes = 0, movers = 0;
    uint32_t kept = 0;
    {
        int tie = tied;
        each([&](int i, int s, bool v, uint32_t k) {
            const bool st = stays(v, k, tie);
            if (KPT > 0) kept |= (uint32_t)st << i;
            holes += __popcll(__ballot(s < low && !st));
            movers += __popcll(__ballot(s >= keep && st));
        });
    }
    const int hole0 = before_wave(holes, lds.part[3], all), mover0 = before_wave(movers, lds.part[4], all);
    int32_t* const work = a.work + ((int64_t)seq * c.kv_heads + kh) * evict_work_words(c.capacity);
    int32_t* const from = work + 16;
    int32_t* const to = from + evict_work_words(c.capacity) / 2 - 8;
    {
        int tie = tied, h = hole0, m = mover0;
        each([&](int i, int s, bool v, uint32_t k) {
            const bool st = KPT > 0 ? (kept >> (i & 31) & 1u) != 0 : stays(v, k, tie);
            const bool hole = s < low && !st, mover = s >= keep && st;
            const uint64_t hm = __ballot(hole), mm = __ballot(mover);
            if (hole) to[h + __popcll(hm & below)] = s;
            if (mover) from[m + __popcll(mm & below)] = s;
            h += __popcll(hm);
            m += __popcll(mm);
            if (s < keep && st && a.pos_out != a.pos_in) a.pos_out[at + s] = pos[s];
            if (s < keep && st && a.score_out != a.score_in) a.score_out[at + s] = score[s];
            if (s >= keep && s < mine && !st) {   // freed; what moves is cleared once it has been read
                a.pos_out[at + s] = -1;
                a.score_out[at + s] = 0.f;
            }
        });
    }
    if (tid == 0) { work[0] = all; work[1] = keep; }
    return true;
}

template <int KPT>
__global__ __launch_bounds__(EV) void k_evict_select(KvCache c, KvBatch b, EvictArgs a) {
    __shared__ EvictLds lds;
    const int kh = blockIdx.x, seq = blockIdx.y;
    const Seq sq = sequence(c, b, seq);
    if (sq.total > EV * KPT || !evict_select<KPT>(c, a, sq, seq, kh, lds)) evict_select<0>(c, a, sq, seq, kh, lds);
}

__global__ __launch_bounds__(256) void k_evict_move(KvCache c, EvictArgs a) {
    const int kh = blockIdx.y, seq = blockIdx.z, units = c.dim / 8;
    const int32_t* work = a.work + ((int64_t)seq * c.kv_heads + kh) * evict_work_words(c.capacity);
    const int32_t* from = work + 16;
    const int32_t* to = from + evict_work_words(c.capacity) / 2 - 8;
    const int64_t at = ((int64_t)seq * c.kv_heads + kh) * a.ld_slots;
    const int64_t n = (int64_t)work[0] * units;
    if (blockIdx.x == 0 && kh == 0 && threadIdx.x == 0) a.ctx_out[seq] = work[1];
    for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
        const int m = (int)(i / units), u = (int)(i % units);
        const int f = from[m], t = to[m];
        if (u == 0) {   // its position and score, and the slot it leaves
            const int32_t p = a.pos_in[at + f];
            const float x = a.score_in[at + f];
            a.pos_out[at + t] = p;
            a.score_out[at + t] = x;
            a.pos_out[at + f] = -1;
            a.score_out[at + f] = 0.f;
        }
        uint32_t sp, dp;
        const int32_t spg = slot_page(c, seq, f, sp), dpg = slot_page(c, seq, t, dp);
        if (dpg < 0) continue;
        u32x4 k = {0, 0, 0, 0}, v = {0, 0, 0, 0};   // of a page that is not there
        if (spg >= 0) {
            k = *(const u32x4*)(c.K + spg * c.k_page + sp * c.k_slot + kh * c.k_head + u * 16);
            v = *(const u32x4*)(c.V + spg * c.v_page + sp * c.v_slot + kh * c.v_head + u * 16);
        }
        *(u32x4*)(c.K + dpg * c.k_page + dp * c.k_slot + kh * c.k_head + u * 16) = k;
        *(u32x4*)(c.V + dpg * c.v_page + dp * c.v_slot + kh * c.v_head + u * 16) = v;
    }
}

}  // namespace

hipError_t launch_cache_evict(const KvCache& c, const KvBatch& b, const EvictArgs& a, hipStream_t s) {
    const int64_t bound = (int64_t)b.max_ctx + b.max_nodes, rows = bound < c.capacity ? bound : c.capacity;
    const dim3 heads(c.kv_heads, b.B);
    if (rows <= 4 * EV) hipLaunchKernelGGL((k_evict_select<4>), heads, dim3(EV), 0, s, c, b, a);
    else if (rows <= 8 * EV) hipLaunchKernelGGL((k_evict_select<8>), heads, dim3(EV), 0, s, c, b, a);
    else if (rows <= 16 * EV) hipLaunchKernelGGL((k_evict_select<16>), heads, dim3(EV), 0, s, c, b, a);
    else hipLaunchKernelGGL((k_evict_select<32>), heads, dim3(EV), 0, s, c, b, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    int64_t most = a.budget < rows ? a.budget : rows;   // moves of a head
    if (rows - most < most && rows - most > 0) most = rows - most;
    int64_t blocks = (most * (c.dim / 8) + 255) / 256;
    if (blocks < 1) blocks = 1;
    if (blocks > 4096) blocks = 4096;
    hipLaunchKernelGGL(k_evict_move, dim3((unsigned)blocks, c.kv_heads, b.B), dim3(256), 0, s, c, a);
    return hipGetLastError();
}

}  // namespace bnn
