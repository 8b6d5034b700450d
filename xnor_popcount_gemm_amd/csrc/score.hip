// The attention weight each cached slot received from the accepted new
// tokens, added to its running sum:
//
//     out_j = in_j + sum over accepted rows i that see j and the group's heads g
//             of exp(scale <q_ig, k_j> - lse_ig)
//
// Bound by the read of K.  A wave works on 32 slots at a time: their K rows go
// straight to LDS (8 lanes fetch a line of 128 bytes), from there to registers,
// as the second operand of S = Q K^T in 16x16x32 matrix products, and the next
// 32 rows are on their way to the same LDS while these are worked on.  Up to
// 32 accepted rows (new tokens times query heads of the group) stay in LDS
// over all slots, and nothing but K is waited for in the loop: a load behind the
// next K rows would hold their whole latency.  More rows, and those of more than
// 64 new tokens, pass by in batches of 32 at each tile, each waited for with the
// next K rows: that is bound by these waits (the case below with 36 rows 116 us
// instead of 76, a chunk of 1024 tokens over 8192 424 us).
// A lane holds one slot's products with 4 rows, so the sum over rows runs in
// registers and two lane swaps finish it; no atomics, a fixed order.
//
// Places without a row hold Q = 0 and lse = +inf, which gives a weight of 0
// unless K holds an infinity or NaN, and so does lse = -inf of a row that saw
// nothing.  A sum that is not finite is therefore taken again row by row by
// what each sees, as in the tiles that hold new tokens.
//
// The grid is what fits the chip at once, and each wave takes an equal run of
// all tiles in the order sequence, key head, tile: sequences of any lengths
// are balanced, and a wave's start (page lookup, list of rows, Q) is paid once
// or twice.  16 sequences of 9000 to 16000 slots, 20 rows: 76 us, 4.9 TB/s (the
// same loads alone, nothing computed: 6.2).
#include <math.h>

#include "bnn_device.hpp"
#include "bnn_launch.hpp"
#include "kv_launch.hpp"

namespace bnn {
namespace {

__device__ __forceinline__ f32x4 mma16(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f32x4 mma16(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

constexpr int NB = 2;     // 16-slot blocks of a wave's tile
constexpr int ROWS = 32;  // rows of a batch

// Sums over the four lanes of a slot: of s0 for lane col, of s1 for lane 16 + col.
__device__ __forceinline__ float over_rows(float s0, float s1) {
    auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(s0), __float_as_uint(s1), false, false);
    const uint32_t x = __float_as_uint(__uint_as_float(p[0]) + __uint_as_float(p[1]));
    auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// Cost of a key head of a sequence: its 32-slot tiles, and START for the start
// of a run and its masked tiles (so that no wave gets many short sequences one
// after the other); nothing where nothing is to be added.
constexpr int START = 3;
static_assert(64 * (((int64_t)1 << 30) / 32 + START) < (int64_t)1 << 32, "the costs of 64 sequences of 2^30 slots are added in 32 bits");
__device__ __forceinline__ uint32_t cost_of(const KvCache& c, const KvBatch& b, int s) {
    const Seq q = sequence(c, b, s);
    return q.nodes ? (q.total + 31) / 32 + START : 0;
}

template <typename T, int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_cache_score_add(KvCache c, KvBatch b, ScoreArgs a) {
    typedef typename T::vec8 vec8;
    constexpr int QS = D / 32;    // products of a 16 x 16 block
    constexpr int GRP = 32 * D;   // bytes of 16 rows
    __shared__ __align__(1024) char lds[4][4 * GRP];   // K, then Q, of each wave
    __shared__ __align__(16) float lows[4][ROWS];
    __shared__ int node_of[4][ROWS];
    __shared__ __align__(16) uint32_t vis_of[4][ROWS];
    __shared__ int taken[4][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quad = lane >> 4;
    typedef Block16<D, true> B;
    constexpr int KV = B::PIECES / 4;      // reads of K that differ in more than a constant offset
    const int fr = lane / B::PIECES;       // row this lane fetches of a block, and of a Q block
    const int qr = lane >> 2;
    const uint32_t my_lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds[wave];
    const char* const qread = lds[wave] + 2 * GRP + col * 64 + ((quad ^ ((col >> 1) & 3)) * 16);
    const char* kread[KV];
#pragma unroll
    for (int i = 0; i < KV; ++i) kread[i] = lds[wave] + B::place_of(col, 4 * i + quad, B::k_swap(col));
    const float c2 = a.scale * 1.44269504088896340736f;
    const bool copies = a.out != a.in;
    const int64_t waves = (int64_t)gridDim.x * 4, me = (int64_t)blockIdx.x * 4 + wave;

    // this wave's share of the cost, in the order sequence, key head, tile; 64 sequences per step
    int64_t all = 0;
    uint32_t cost0 = 0, upto0 = 0;   // of sequence `lane`: its cost, and that of the sequences up to it
    for (int s0 = 0; s0 < b.B; s0 += 64) {
        const uint32_t n = s0 + lane < b.B ? cost_of(c, b, s0 + lane) : 0;
        uint32_t upto = n;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) { const uint32_t x = __shfl_up(upto, m, 64); upto += lane >= m ? x : 0; }
        if (s0 == 0) { cost0 = n; upto0 = upto; }
        all += (uint32_t)__builtin_amdgcn_readlane(upto, 63);
    }
    all *= c.kv_heads;
    int64_t left = all * (me + 1) / waves - all * me / waves, skip = all * me / waves;
    int seq = 0, mine = 0;   // the sequence of the first unit, and its cost
    if (left > 0)
        for (int s0 = 0;; s0 += 64) {
            uint32_t n = cost0, upto = upto0;
            if (s0 > 0) {
                n = s0 + lane < b.B ? cost_of(c, b, s0 + lane) : 0;
                upto = n;
#pragma unroll
                for (int m = 1; m < 64; m <<= 1) { const uint32_t x = __shfl_up(upto, m, 64); upto += lane >= m ? x : 0; }
            }
            const int before = __popcll(__ballot((int64_t)upto * c.kv_heads <= skip));   // whole sequences skipped
            if (before < 64) {
                seq = s0 + before;
                mine = __builtin_amdgcn_readlane(n, before);
                skip -= (int64_t)((uint32_t)__builtin_amdgcn_readlane(upto, before) - (uint32_t)mine) * c.kv_heads;
                break;
            }
            skip -= (int64_t)(uint32_t)__builtin_amdgcn_readlane(upto, 63) * c.kv_heads;
        }
    int kh = left > 0 ? (int)(skip / mine) : 0, unit = left > 0 ? (int)(skip % mine) : 0;

    while (left > 0) {
        const Seq sq = sequence(c, b, seq);
        const int nodes = sq.nodes < b.max_nodes ? sq.nodes : b.max_nodes;
        const int64_t at = ((int64_t)seq * c.kv_heads + kh) * a.ld_slots;
        const int run = (int)(left < mine - unit ? left : mine - unit);
        const int tile = unit > START ? unit - START : 0, end = unit + run - START;
        const int32_t* const table = c.table ? c.table + (int64_t)seq * c.ld_table : nullptr;
        const char* const kbase = c.K + kh * c.k_head + ((lane % B::PIECES) ^ B::k_swap(fr)) * 16;
        // page entries: 64 of the table at a time, one per lane, so that a tile's lookups are lane reads
        const int64_t pages = table ? c.ld_table : 0;
        int32_t held = -1;
        int64_t held0 = -64;
        const char* ptr[NB * B::HALVES];
        auto locate = [&](int t) {   // the rows of tile t
            const uint32_t first_page = fastdiv((uint32_t)t * 32, c.page);
            uint32_t last_slot = (uint32_t)t * 32 + 31;
            last_slot = last_slot < (uint32_t)sq.total ? last_slot : (uint32_t)sq.total - 1;
            if (table && fastdiv(last_slot, c.page) >= held0 + 64) {
                held0 = first_page;
                held = held0 + lane < pages ? table[held0 + lane] : -1;
                asm volatile("" : "+v"(held));   // waited for here: at its use the wait would take in the rows on their way
            }
#pragma unroll
            for (int n = 0; n < NB * B::HALVES; ++n) {
                const uint32_t slot = (uint32_t)t * 32 + 16 / B::HALVES * n + fr, pg = fastdiv(slot, c.page);
                const uint32_t place = slot - pg * c.page.d;
                int32_t entry = seq;
                if (table) entry = __shfl(held, (int)(pg - held0), 64);
                const bool there = slot < (uint32_t)sq.total && (uint32_t)entry < c.num_pages;
                ptr[n] = there ? kbase + entry * c.k_page + place * c.k_slot : (const char*)zero_row;
            }
        };
        auto fetch = [&] {
#pragma unroll
            for (int n = 0; n < NB * B::HALVES; ++n)
#pragma unroll
                for (int s = 0; s < B::COLS; ++s) {
                    const char* p = ptr[n] + 16 * B::PIECES * s;
                    const uint32_t to = my_lds + (n * B::COLS + s) * 1024;
                    B::WIDE ? dma16_once(p, to) : dma16(p, to);   // read once; half lines would come twice
                }
        };
        auto before = [&](int t) {   // lanes 0 .. 31 write a slot each
            const int64_t slot = (int64_t)t * 32 + lane;
            return lane < 16 * NB && slot < sq.total ? a.in[at + slot] : 0.f;
        };
        // the accepted of 64 new tokens from n0 on, in order, as this wave's list
        auto list = [&](int n0) {
            const int nd = n0 + lane;
            const bool in = nd < nodes && (!a.accept || packed_bit(a.accept + seq * a.ld_accept, a.ld_accept, nd));
            const uint64_t got = __ballot(in);
            if (in) taken[wave][__popcll(got & ((1ull << lane) - 1))] = nd;
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            return __popcll(got) * a.group;
        };
        // rows r0 .. r0 + 31 of the list: Q to LDS, lse in base 2 (+inf where there is no row: its weight is 0), new token
        auto stage = [&](int r0, int rows) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int r = r0 + 16 * g + qr;
                const bool live = r < rows;
                const int rank = live ? r / a.group : 0;
                const int node = taken[wave][rank];
                const int64_t row = sq.row0 + node;
                const int head = kh * a.group + (live ? r - rank * a.group : 0);
                const char* q = live ? a.q + row * a.q_row + head * a.q_head + ((lane & 3) ^ ((qr >> 1) & 3)) * 16 : (const char*)zero_row;
#pragma unroll
                for (int s = 0; s < QS; ++s) dma16(q + 64 * s, my_lds + (2 + g) * GRP + 1024 * s);
                if ((lane & 3) == 0) {
                    const float lse = live ? a.lse[row * a.ld_lse + head] * 1.44269504088896340736f : INFINITY;
                    lows[wave][16 * g + qr] = lse == -INFINITY ? INFINITY : lse;
                    node_of[wave][16 * g + qr] = live && lse != -INFINITY ? node : -1;
                }
            }
        };

        // of each row of the batch which of the 32 slots from s0 on it sees
        auto sight = [&](int64_t s0) {
            if (lane < ROWS) {
                const int node = node_of[wave][lane];
                const int64_t rel = s0 - sq.ctx;
                uint32_t vis = 0;
                if (node >= 0) {
                    if (rel <= -32) {
                        vis = ~0u;
                    } else if (!a.mask) {
                        const int64_t n = node - rel + 1;
                        vis = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1;
                    } else {
                        const uint32_t* mr = a.mask + (sq.row0 + node) * a.ld_mask;
                        if (rel >= 0) {
                            const int64_t w = rel >> 5;
                            const uint64_t lo = w < a.ld_mask ? mr[w] : 0u, hi = w + 1 < a.ld_mask ? mr[w + 1] : 0u;
                            vis = (uint32_t)((lo | hi << 32) >> (rel & 31));
                        } else {
                            vis = (mr[0] << -rel) | ((1u << -rel) - 1);
                        }
                    }
                }
                vis_of[wave][lane] = vis;
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        };

        const int first = list(0);
        const bool few = nodes <= 64 && first <= ROWS;   // all rows stay in LDS
        if (end <= tile) {                               // the start alone
        } else if (few && first == 0) {                  // nothing to add
            if (copies)
                for (int64_t s = (int64_t)tile * 32 + lane; s < (int64_t)end * 32 && s < sq.total; s += 64) a.out[at + s] = a.in[at + s];
        } else {
            locate(tile);
            if (few) stage(0, first);
            fetch();
            float next = before(tile), done = 0.f;
            if (tile + 1 < end) locate(tile + 1);
            for (int t = tile; t < end; ++t) {
                wait_all();
                vec8 k[NB][QS];
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int s = 0; s < QS; ++s) k[n][s] = *(const vec8*)(kread[s % KV] + n * GRP + s / KV * 1024);
                const float old = next;
                const int64_t s0 = (int64_t)t * 32;
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before it is overwritten
                if (t + 1 < end) fetch();
                // behind the fetch, so that it does not hold the next wait up
                if (t > tile && lane < 32) a.out[at + s0 - 32 + lane] = done;
                if (t + 1 < end) {
                    next = before(t + 1);
                    if (t + 2 < end) locate(t + 2);
                }
                float sum[NB];
#pragma unroll 1
                for (bool masked = s0 + 32 > sq.ctx;; masked = true) {
#pragma unroll
                    for (int n = 0; n < NB; ++n) sum[n] = 0.f;
#pragma unroll 1
                    for (int n0 = 0; n0 < nodes; n0 += 64) {
                        const int rows = few ? first : list(n0);
#pragma unroll 1
                        for (int r0 = 0; r0 < rows; r0 += ROWS) {
                            if (!few) {
                                stage(r0, rows);
                                wait_all();
                            }
                            if (masked) sight(s0);
#pragma unroll 1
                            for (int g = 0; g < 2 && r0 + 16 * g < rows; ++g) {
                                f32x4 x[NB] = {};
#pragma unroll
                                for (int s = 0; s < QS; ++s) {
                                    const vec8 q = *(const vec8*)(qread + g * GRP + 1024 * s);
#pragma unroll
                                    for (int n = 0; n < NB; ++n) x[n] = mma16(q, k[n][s], x[n]);
                                }
                                const f32x4 low = *(const f32x4*)&lows[wave][16 * g + 4 * quad];
#pragma unroll
                                for (int n = 0; n < NB; ++n)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) x[n][i] = __builtin_amdgcn_exp2f(fmaf(x[n][i], c2, -low[i]));
                                if (masked) {
                                    const u32x4 v = *(const u32x4*)&vis_of[wave][16 * g + 4 * quad];
#pragma unroll
                                    for (int n = 0; n < NB; ++n)
#pragma unroll
                                        for (int i = 0; i < 4; ++i) x[n][i] = (v[i] >> (16 * n + col)) & 1u ? x[n][i] : 0.f;
                                }
#pragma unroll
                                for (int n = 0; n < NB; ++n) sum[n] += (x[n][0] + x[n][1]) + (x[n][2] + x[n][3]);
                            }
                        }
                    }
                    if (masked || !__any(!(fabsf(sum[0]) < INFINITY) || !(fabsf(sum[1]) < INFINITY))) break;
                }
                done = old + over_rows(sum[0], sum[1]);
            }
            const int64_t slot = (int64_t)end * 32 - 32 + lane;
            if (lane < 32 && slot < sq.total) a.out[at + slot] = done;
        }
        left -= run;
        unit += run;
        if (unit == mine) {
            unit = 0;
            if (++kh == c.kv_heads) {
                kh = 0;
                if (left > 0) do mine = cost_of(c, b, ++seq); while (mine == 0);
            }
        }
    }

    if (copies) {   // slots that hold no token or gain nothing, 1024 of a row at a time
        const int64_t pieces = (a.ld_slots + 1023) / 1024, jobs = pieces * b.B * c.kv_heads;
        for (int64_t j = me; j < jobs; j += waves) {
            const int64_t row = j / pieces, i0 = j % pieces * 1024;
            const Seq sq = sequence(c, b, (int)(row / c.kv_heads));
            const int64_t from = sq.nodes ? sq.total : 0;
            if (i0 + 1024 <= from) continue;
            const float* in = a.in + row * a.ld_slots;
            float* out = a.out + row * a.ld_slots;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int64_t e = i0 + 64 * i + lane;
                if (e >= from && e < a.ld_slots) x[i] = in[e];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int64_t e = i0 + 64 * i + lane;
                if (e >= from && e < a.ld_slots) out[e] = x[i];
            }
        }
    }
}

template <typename T, int D>
void launch_one(const KvCache& c, const KvBatch& b, const ScoreArgs& a, hipStream_t s) {
    constexpr int PER_CU = D == 64 ? 4 : D == 96 ? 3 : D == 128 ? 2 : 1;   // by LDS
    const int64_t bound = (int64_t)b.max_ctx + b.max_nodes, slots = bound < c.capacity ? bound : c.capacity;
    const int64_t tiles = (slots / 32 + 1 + START) * c.kv_heads * b.B;
    int64_t blocks = (tiles + 3) / 4;
    const int64_t most = (int64_t)num_cus() * PER_CU;   // what is resident at once
    if (blocks > most) blocks = most;
    hipLaunchKernelGGL((k_cache_score_add<T, D>), dim3((unsigned)blocks), dim3(256), 0, s, c, b, a);
}

template <typename T>
void launch_dim(const KvCache& c, const KvBatch& b, const ScoreArgs& a, hipStream_t s) {
    if (c.dim == 64) launch_one<T, 64>(c, b, a, s);
    else if (c.dim == 96) launch_one<T, 96>(c, b, a, s);
    else if (c.dim == 128) launch_one<T, 128>(c, b, a, s);
    else launch_one<T, 256>(c, b, a, s);
}

}  // namespace

hipError_t launch_cache_score_add(const KvCache& c, const KvBatch& b, const ScoreArgs& a, int32_t dtype, hipStream_t s) {
    if (dtype == KV_BF16) launch_dim<Bf16>(c, b, a, s);
    else launch_dim<F16>(c, b, a, s);
    return hipGetLastError();
}

}  // namespace bnn
