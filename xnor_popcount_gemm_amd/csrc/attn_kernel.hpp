// Attention of a step's new tokens over the paged cache, on the matrix cores.
//
//     s_j = scale <q, k_j> ;  out = sum_j exp(s_j - lse) v_j ;  lse = ln sum_j exp(s_j)
//
// The rows of a (sequence, key head) are its new tokens times the query heads
// that share the key head, so one pass over K and V serves them all.
//
// Products.  Scores are computed transposed, S^T = K Q^T: a lane then holds one
// row's scores for 8 or 16 of a step's 32 slots, so the softmax statistics are
// a few in-lane operations and one or two lane swaps, and the weights are
// already laid out as the second operand of O^T = V^T P^T: no weight crosses a
// lane.  That operand has the cache's 16 bits.  With a 16-bit output a weight
// is rounded once to it, by half an ulp like the output itself (errors against
// 64 bits a third larger than with exact weights, 0.0023 for 0.0017); with fp32
// output it is split into the terms that keep it, two of float16 or three of
// bfloat16, each a product more: 1024 tokens over 8192 take 291 us instead of
// 183, in float16 246 instead of 192.  What V^T needs is a transposed read of
// V's rows, which ds_read_b64_tr_b16 gives.  R = 16 rows per wave use 16x16x32
// matrix instructions, R = 32 rows 32x32x16.
//
// Running maximum.  Weights are taken relative to a reference that is only
// raised when a score passes it by more than 2^8 (in the base-2 logarithm):
// the result is the same, and the accumulators are rescaled a few times
// instead of at every step.  bfloat16 weights have fp32's exponents, so that is
// all; float16 ones end at 2^-24, and slots far below one that dominates the
// row (whose V may be near 0) would be lost.  There the reference follows each
// step's maximum both ways, so that the step's largest weight lies in
// 2^5 .. 2^15.5 (2^10 where it is moved, at most 2^48 below its peak): a weight
// is then off by its rounding or by 2^-30 of the largest of its 32 or 64 slots.
// Trees of 63 tokens over 32000 slots take 198 us that way (193 without, 201
// where it is moved to 2^12: some row of a wave does so at most steps).
//
// Tiles.  K and V rows go from global memory straight to LDS (16 bytes per
// lane); the next step's rows are in flight while one is worked on, in a
// second buffer where the waves of a workgroup share the tile.  With up to 32
// rows each wave has tiles of its own, which pass on to registers so that one
// buffer will do and twice the waves fit a compute unit.  A wave's load brings
// 1 KiB.  With up to 32 rows that is 8 rows of 128 bytes, whole cache lines (16
// rows of 64 for 96 dimensions), read without keeping them in the caches: 64
// sequences of about 6200 slots take 285 us that way (5.6 TB/s) and 311 kept; in
// half lines 396 and 327.  With more rows the row tiles share the caches, and a
// load brings 16 rows of 64 bytes, which halves a lane's page lookups.  The
// 16-byte pieces of row r are permuted by XOR so that the lanes served together
// read different banks: of 128-byte rows by r % 8 for K (b128 reads of one piece
// of 8 slots) and by 2 (r % 4) for V (transposed reads of two pieces of 4 slots),
// of 64-byte rows by (r / 2) % 4 and 2 ((r / 2) % 2), which leaves a third of the
// LDS cycles to conflicts.  Rows past the end are read from a block of zeros.
//
// Masks.  Committed slots are seen by every row and cost nothing, and so do the
// new tokens of a causal run up to the first row's own (a prompt of 4096
// tokens: 182 us; 212 with these steps among the masked ones).  Steps that hold
// other new tokens take one 32-bit word per row and 32 slots, and run as the
// others do where every row sees them whole.  An unseen token must not matter
// even where its V is NaN or infinite, and 0 * NaN is NaN, so a masked step
// takes such values as 0 in the products and notes, as bits per row and
// dimension, which rows saw an infinity of which sign (NaN: both); the
// infinities are added at the end.  A plain step has no such care: a weight
// that was rounded to 0, or the negative remainder of one, makes NaN of a
// committed infinity.  Where a wave's result is not finite it reads V of the
// slots that all rows see once more for what they hold.
//
// What bounds it.  Few rows: the read of K and V; 285 us for 1.59 GB, where the
// same paged rows fetched and not used take about 265.  Many rows: neither the
// matrix cores (busy 41% of the time at a 1024-token chunk, 830 TFLOP/s) nor
// the vector unit (33%) nor LDS (31%) is full: two waves per SIMD wait for each
// other's products, exponentials and the shared tile in turn; without the
// fetches the same steps reach 940, those of trees 980 instead of 755.
#pragma once

#include <math.h>

#include <type_traits>

#include "bnn_device.hpp"
#include "kv_launch.hpp"

namespace bnn {

// How a call is cut into workgroups, from what the host knows.
struct AttnPlan {
    int32_t R, RW, KW;     // rows per wave, waves along rows, waves along slots
    int32_t row_tiles;     // of a (sequence, key head), at most
    int32_t chunk;         // slots per workgroup
    int32_t chunks;        // of a sequence, at most
    int32_t groups;        // chunks of all sequences and key heads
};

namespace {

template <typename T> struct Mma;
template <> struct Mma<Bf16> {
    static __device__ __forceinline__ f32x16 m32(bf16x8 a, bf16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ f32x4 m16(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};
template <> struct Mma<F16> {
    static __device__ __forceinline__ f32x16 m32(f16x8 a, f16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ f32x4 m16(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};

// Maximum / sum over the lanes that hold one row: l ^ 32, and l ^ 16 for 16 rows.
template <int R>
__device__ __forceinline__ float row_max(float x) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    if (R == 16) {
        auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
    }
    return x;
}

template <int R>
__device__ __forceinline__ float row_sum(float x) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    if (R == 16) {
        auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(q[0]) + __uint_as_float(q[1]);
    }
    return x;
}

// Factor of sums taken relative to m where they join others relative to M.  Never 0 but where nothing was
// seen: infinities stay infinities.
__device__ __forceinline__ float joined(float m, float M) {
    return m == -INFINITY ? 0.f : fmaxf(__builtin_amdgcn_exp2f(m - M), 0x1p-126f);
}

template <int R> struct Acc;
template <> struct Acc<16> { typedef f32x4 type; };
template <> struct Acc<32> { typedef f32x16 type; };

// Partial results of a chunk: out rows and (maximum, sum) per row.
__host__ __device__ inline int64_t part_rows(int64_t rows, int64_t heads) { return rows * heads; }

template <typename T, int D, int R, int RW, int KW, int NS, typename O>
struct Attn {
    typedef typename T::vec8 vec8;
    typedef typename T::vec4 vec4;
    typedef typename T::elem elem;
    typedef typename Acc<R>::type acc;

    static constexpr int WAVES = RW * KW;
    static constexpr int BN = RW == 4 && D < 256 ? 64 : 32;     // slots per step and slot group
    static constexpr int SUB = BN / 32;
    static constexpr int NSC = R / 2;                           // scores per lane and 32 slots
    static constexpr int QS = R == 32 ? D / 16 : D / 32;        // products of a 32-slot score block
    static constexpr int OB = R == 32 ? D / 32 : D / 16;        // accumulator blocks
    static constexpr int GRP = 32 * D;                          // bytes of 16 slots
    static constexpr int VOFF = BN * D * 2;                     // V after K in a buffer
    static constexpr int STAGE = 2 * VOFF;
    static constexpr bool REGS = RW == 1;                       // tiles pass through registers: one buffer
    static constexpr bool ONCE = REGS && Block16<D, true>::WIDE;         // one row tile reads K and V, by whole lines
    static constexpr int KR = R == 32 ? QS : 2 * QS;            // operands of a 32-slot tile of K; of V as many
    static constexpr int GROUP_LDS = (REGS ? 1 : 2) * STAGE;    // buffers of a slot group
    static constexpr int OPAD = D + 4;
    static constexpr int MERGE = KW > 1 ? KW * RW * R * OPAD * 4 + KW * RW * R * 8 : 4 * 32 * 36 * 4;
    static constexpr int LDS = KW * GROUP_LDS > MERGE ? KW * GROUP_LDS : MERGE;
    typedef Block16<D, RW == 1> B;
    static constexpr int PIECES = B::PIECES, HALVES = B::HALVES, COLS = B::COLS;
    // reads of one operand that differ in more than a constant offset
    static constexpr int KV = R == 32 ? PIECES / 2 : PIECES / 4, VV = R == 32 ? PIECES / 4 : PIECES / 2;
    static constexpr int VSTEP = R == 16 ? GRP : B::WIDE ? COLS * 1024 : 512;   // to the other 4 slots of an operand

    // 16-slot groups that a wave fetches per step, and whether it fetches both K and V of them
    static constexpr int FETCH = RW == 1 ? 2 : 1;
    static constexpr bool SPLIT_KV = RW == 4 && BN == 32;

    static __device__ __forceinline__ int slot_of(int i, int lane) {
        return R == 32 ? 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) : 16 * (i >> 2) + 4 * (lane >> 4) + (i & 3);
    }

    static __device__ __forceinline__ vec8 v_frag(const char* base, int o) {
        typedef __attribute__((address_space(3))) s16x4* tp;
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tp)(base + o));
        const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tp)(base + o + VSTEP));
        return __builtin_bit_cast(vec8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }

    // base-2 logarithms of a float16 step's largest weight: bounds, where it is put, and how far the reference may sink
    static constexpr bool NARROW = std::is_same<T, F16>::value;
    static constexpr float HIGH = NARROW ? 15.5f : 8.f, LOW = 5.f, AIM = 10.f, DEEP = 48.f;

    static constexpr int PW = (OB * (int)sizeof(acc) / 4 + 31) / 32;   // words of a bit per accumulator

    // Whether the low 16 bits are NaN or an infinity.
    static __device__ __forceinline__ uint32_t special(uint32_t h) { return (h & T::special) == T::special; }

    // NaN and infinities as 0.
    static __device__ __forceinline__ vec8 finite(vec8 v) {
        u32x4 x = __builtin_bit_cast(u32x4, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (special(x[i])) x[i] &= 0xFFFF0000u;
            if (special(x[i] >> 16)) x[i] &= 0x0000FFFFu;
        }
        return __builtin_bit_cast(vec8, x);
    }

    static __device__ __forceinline__ acc mma(vec8 a, vec8 b, acc c) {
        if constexpr (R == 32) return Mma<T>::m32(a, b, c);
        else return Mma<T>::m16(a, b, c);
    }
};

template <typename T, int D, int R, int RW, int KW, int NS, typename O>
__global__ __launch_bounds__(RW * KW * 64, (D == 256 ? 1 : 2)) void k_tree_attention(KvCache c, KvBatch b, AttnArgs a, AttnPlan pl) {
    typedef Attn<T, D, R, RW, KW, NS, O> A;
    typedef typename A::vec8 vec8;
    typedef typename A::acc acc;
    __shared__ __align__(1024) char lds[A::LDS];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int rw = wave % RW, kw = wave / RW;
    // Workgroups go to the 8 XCDs in turn, and each XCD has its own L2: the row tiles of a chunk of a key head,
    // which read the same K and V, take every eighth place.
    const uint32_t block = wide_index(blockIdx.y), idx = block / 8, group = idx / pl.row_tiles * 8 + block % 8;
    if (group >= (uint32_t)pl.groups) return;
    const int rt = idx % pl.row_tiles, ci = group % pl.chunks, pair = group / pl.chunks, kh = pair % c.kv_heads, seq = pair / c.kv_heads;

    const int k0 = ci * pl.chunk;

    // fetch of K and V rows: a lane takes 16-byte pieces of one row per block
    char* const my = lds + kw * A::GROUP_LDS;
    const uint32_t my_lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)my;
    const int fr = lane / A::PIECES, fp = lane % A::PIECES;   // row (of the first block) and place in it
    const char* const kbase = c.K + kh * c.k_head + (fp ^ A::B::k_swap(fr)) * 16;
    const char* const vbase = c.V + kh * c.v_head + (fp ^ A::B::v_swap(fr)) * 16;
    const int32_t* const table = c.table ? c.table + (int64_t)seq * c.ld_table : nullptr;
    int32_t entry[A::FETCH * A::HALVES];
    uint32_t place[A::FETCH * A::HALVES];
    auto slot_of_fetch = [&](int step, int f) {
        const int g = RW == 1 ? f / A::HALVES : rw % (A::BN / 16);
        return k0 + (step * KW + kw) * A::BN + 16 * g + 8 * (f % A::HALVES) + fr;
    };
    auto lookup = [&](int step, int end) {
#pragma unroll
        for (int f = 0; f < A::FETCH * A::HALVES; ++f) {
            const int slot = slot_of_fetch(step, f);
            entry[f] = -1;
            if (slot < end) {
                const uint32_t p = fastdiv(slot, c.page);
                place[f] = slot - p * c.page.d;
                entry[f] = table ? table[p] : seq;
            }
        }
    };
    lookup(0, c.capacity);   // before the sequence's length is known

    const Seq sq = sequence(c, b, seq);
    const int nodes = sq.nodes < b.max_nodes ? sq.nodes : b.max_nodes;
    const int rows = nodes * a.group, tile0 = rt * R * RW;
    if (tile0 >= rows) return;
    int nchunk = (sq.total + pl.chunk - 1) / pl.chunk;
    nchunk = nchunk < 1 ? 1 : nchunk > pl.chunks ? pl.chunks : nchunk;
    if (ci >= nchunk) return;
    // slots of this workgroup; without a mask none past the last row's own
    const int last_row = (tile0 + R * RW < rows ? tile0 + R * RW : rows) - 1;
    int end = sq.total;
    if (!a.mask) { const int64_t own = (int64_t)sq.ctx + last_row / a.group + 1; end = own < end ? (int)own : end; }
    int k1 = ci == nchunk - 1 ? end : k0 + pl.chunk;
    k1 = k1 < end ? k1 : end;
    const int steps = k1 > k0 ? (k1 - k0 + KW * A::BN - 1) / (KW * A::BN) : 0;

    // this lane's row and its query, the second operand of S^T = K Q^T
    const int lr = lane & (R - 1);
    const int r = tile0 + rw * R + lr;
    const bool live = r < rows;
    const int node = live ? r / a.group : 0;
    const int64_t row = sq.row0 + node;
    const int head = kh * a.group + (live ? r - node * a.group : 0);
    const float c2 = fabsf(a.scale) * 1.44269504088896340736f;
    vec8 qf[A::QS];
    {
        const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
        const char* q = a.q + row * a.q_row + head * a.q_head + (lane / R) * 16;
#pragma unroll
        for (int s = 0; s < A::QS; ++s) {
            u32x4 x = {0, 0, 0, 0};
            if (live) x = *(const u32x4*)(q + s * (R == 32 ? 32 : 64));
            x ^= flip;
            qf[s] = __builtin_bit_cast(vec8, x);
        }
    }

    auto fetch = [&](int buf) {
#pragma unroll
        for (int f = 0; f < A::FETCH * A::HALVES; ++f) {
            const int g = RW == 1 ? f / A::HALVES : rw % (A::BN / 16);
            const bool there = (uint32_t)entry[f] < c.num_pages;
            const uint32_t to = my_lds + buf * A::STAGE + g * A::GRP + (f % A::HALVES) * A::COLS * 1024;
            if (!A::SPLIT_KV || rw < 2) {
                const char* p = there ? kbase + entry[f] * c.k_page + place[f] * c.k_slot : (const char*)zero_row;
#pragma unroll
                for (int j = 0; j < A::COLS; ++j) A::ONCE ? dma16_once(p + 16 * A::PIECES * j, to + 1024 * j) : dma16(p + 16 * A::PIECES * j, to + 1024 * j);
            }
            if (!A::SPLIT_KV || rw >= 2) {
                const char* p = there ? vbase + entry[f] * c.v_page + place[f] * c.v_slot : (const char*)zero_row;
#pragma unroll
                for (int j = 0; j < A::COLS; ++j) A::ONCE ? dma16_once(p + 16 * A::PIECES * j, to + A::VOFF + 1024 * j) : dma16(p + 16 * A::PIECES * j, to + A::VOFF + 1024 * j);
            }
        }
    };

    // LDS offsets of this lane's operand reads: read q of K is kread[q % KV] + q / KV KiB, block i of V alike
    int kread[A::KV], vread[A::VV];
    if constexpr (R == 32) {
        const int r = lane & 15, hi = lane >> 5, d = (lane >> 4) & 1, key = 4 * hi + (r >> 2);
#pragma unroll
        for (int q = 0; q < A::KV; ++q) kread[q] = d * A::GRP + A::B::place_of(r, 2 * q + hi, A::B::k_swap(r));
#pragma unroll
        for (int i = 0; i < A::VV; ++i) vread[i] = A::VOFF + A::B::place_of(key, 4 * i + 2 * d + ((r & 3) >> 1), A::B::v_swap(key)) + (r & 1) * 8;
    } else {
        const int r = lane & 15, quad = lane >> 4, key = 4 * quad + (r >> 2);
#pragma unroll
        for (int q = 0; q < A::KV; ++q) kread[q] = A::B::place_of(r, 4 * q + quad, A::B::k_swap(r));
#pragma unroll
        for (int i = 0; i < A::VV; ++i) vread[i] = A::VOFF + A::B::place_of(key, 2 * i + ((r & 3) >> 1), A::B::v_swap(key)) + (r & 1) * 8;
    }

    acc o[A::OB];
#pragma unroll
    for (int i = 0; i < A::OB; ++i) o[i] = acc{};
    float m = -INFINITY, l = 0.f;   // reference (base-2 logarithm) and this lane's share of the sum
    float peak = -INFINITY, least = A::LOW;   // the highest reference so far; what lowers it
    // which of this lane's dimensions saw +inf / -inf: bit 4 i + e of dimension e of its piece i of 4
    uint32_t plus[A::PW], minus[A::PW];
#pragma unroll
    for (int i = 0; i < A::PW; ++i) plus[i] = minus[i] = 0;

    // which of the 32 slots from each kb0 + 32 sub on this lane's row sees; 0: no row sees any, 2: all see all, else 1
    auto sight = [&](const int kb0, uint32_t (&vis)[A::SUB]) {
        bool any = false, part = false;
#pragma unroll
        for (int sub = 0; sub < A::SUB; ++sub) {
            const int kb = kb0 + 32 * sub, rel = kb - sq.ctx;
            uint32_t v = 0xFFFFFFFFu;
            if (live && rel > -32) {
                if (!a.mask) {
                    const int n = node - rel + 1;
                    v = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1;
                } else {
                    const uint32_t* mr = a.mask + row * a.ld_mask;
                    if (rel >= 0) {
                        const int w = rel >> 5;
                        const uint64_t lo = w < a.ld_mask ? mr[w] : 0u, hi = w + 1 < a.ld_mask ? mr[w + 1] : 0u;
                        v = (uint32_t)((lo | hi << 32) >> (rel & 31));
                    } else {
                        v = (mr[0] << -rel) | ((1u << -rel) - 1);
                    }
                }
            }
            if (k1 - kb < 32) v &= k1 > kb ? (1u << (k1 - kb)) - 1 : 0u;
            vis[sub] = v;
            any |= live && v != 0;
            part |= v != 0xFFFFFFFFu;
        }
        return !__any(any) ? 0 : __any(part) ? 1 : 2;
    };

    // one step: BN slots, in the buffer buf; with kr, vr their operands already in registers
    auto work = [&](auto is_masked, const char* buf, const uint32_t (&vis)[A::SUB], const vec8* kr, const vec8* vr) {
        constexpr bool MASKED = decltype(is_masked)::value;
        constexpr bool REGS = A::REGS && !MASKED;

        // scores
        float sc[A::SUB][A::NSC];
#pragma unroll
        for (int sub = 0; sub < A::SUB; ++sub) {
            if constexpr (R == 32) {
                f32x16 s = {};
#pragma unroll
                for (int q = 0; q < A::QS; ++q)
                    s = Mma<T>::m32(REGS ? kr[q] : *(const vec8*)(buf + sub * 2 * A::GRP + kread[q % A::KV] + q / A::KV * 1024), qf[q], s);
#pragma unroll
                for (int i = 0; i < 16; ++i) sc[sub][i] = s[i];
            } else {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    f32x4 s = {};
#pragma unroll
                    for (int q = 0; q < A::QS; ++q)
                        s = Mma<T>::m16(REGS ? kr[g * A::QS + q] : *(const vec8*)(buf + g * A::GRP + kread[q % A::KV] + q / A::KV * 1024), qf[q], s);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[sub][4 * g + i] = s[i];
                }
            }
        }
        if (MASKED) {
#pragma unroll
            for (int sub = 0; sub < A::SUB; ++sub)
#pragma unroll
                for (int i = 0; i < A::NSC; ++i) sc[sub][i] = (vis[sub] >> A::slot_of(i, lane)) & 1u ? sc[sub][i] : -INFINITY;
        }
        float mx = sc[0][0];
#pragma unroll
        for (int sub = 0; sub < A::SUB; ++sub)
#pragma unroll
            for (int i = 0; i < A::NSC; ++i) mx = fmaxf(mx, sc[sub][i]);
        mx = row_max<R>(mx) * c2;
        const float over = mx - m;
        if (__any(over > A::HIGH || (A::NARROW && over < least))) {
            float mn = fmaxf(m, mx);
            if constexpr (A::NARROW) {
                mn = m;
                if (mx > -INFINITY && (over > A::HIGH || over < least)) mn = fmaxf(mx - A::AIM, peak - A::DEEP);
                peak = fmaxf(peak, mn);
                least = mn > peak - A::DEEP ? A::LOW : -INFINITY;
            }
            const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int i = 0; i < A::OB; ++i) o[i] *= f;
        }
        const float ms = m == -INFINITY ? 0.f : m;
        float ls[2] = {0.f, 0.f};
#pragma unroll
        for (int sub = 0; sub < A::SUB; ++sub)
#pragma unroll
            for (int i = 0; i < A::NSC; ++i) {
                float p = __builtin_amdgcn_exp2f(fmaf(sc[sub][i], c2, -ms));
                if (MASKED) p = (vis[sub] >> A::slot_of(i, lane)) & 1u ? p : 0.f;   // a scale of 0 makes NaN of an unseen one's -inf
                sc[sub][i] = p;
                ls[i & 1] += p;
            }
        l += ls[0] + ls[1];

#pragma unroll
        for (int sub = 0; sub < A::SUB; ++sub) {
            // weights as 16-bit operands: one term where the output is rounded as much, or as many as keep them whole
            vec8 pf[A::NSC / 8][NS];
#pragma unroll
            for (int g = 0; g < A::NSC / 8; ++g) {
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const typename A::elem p = (typename A::elem)sc[sub][8 * g + i];
                        pf[g][n][i] = p;
                        if (n + 1 < NS) sc[sub][8 * g + i] -= (float)p;
                    }
            }
            const char* vb = buf + sub * 2 * A::GRP;
#pragma unroll
            for (int g = 0; g < A::NSC / 8; ++g)
#pragma unroll
                for (int i = 0; i < A::OB; ++i) {
                    vec8 v = REGS ? vr[g * A::OB + i]
                           : A::v_frag(vb, vread[i % A::VV] + i / A::VV * 1024 + (R == 32 ? g * A::GRP : 0));
                    if (MASKED) v = A::finite(v);
#pragma unroll
                    for (int n = 0; n < NS; ++n) o[i] = A::mma(v, pf[g][n], o[i]);
                }
            if (MASKED) {
                uint32_t bad = 0;
#pragma unroll 4
                for (int i = 0; i < D / 16; ++i) {
                    const u32x4 x = *(const u32x4*)(vb + A::VOFF + (i * 64 + lane) * 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j) bad |= A::special(x[j]) | A::special(x[j] >> 16);
                }
                if (__any(bad)) {   // rare: slot by slot
#pragma unroll 1
                    for (int key = 0; key < 32; ++key) {
                        const bool saw = (vis[sub] >> key) & 1u;
                        const char* vr = vb + A::VOFF + (key >> 4) * A::GRP;
#pragma unroll
                        for (int w = 0; w < A::PW; ++w) {
                            uint32_t up = 0, down = 0;
#pragma unroll 1
                            for (int q = 0; q < 8; ++q) {
                                const int piece = 8 * w + q;   // 4 dimensions of this lane's row
                                if (piece >= A::OB * (R == 32 ? 4 : 1)) break;
                                const int d = R == 32 ? 8 * piece + 4 * (lane >> 5) : 16 * piece + 4 * (lane >> 4);
                                const u32x2 x = *(const u32x2*)(vr + A::B::place_of(key & 15, d >> 3, A::B::v_swap(key & 15)) + (d & 4) * 2);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t h = (e < 2 ? x[0] : x[1]) >> (16 * (e & 1)) & 0xFFFFu;
                                    const bool nan = (h & 0x7FFFu) > T::special;
                                    up |= (uint32_t)(nan || h == T::special) << (4 * q + e);
                                    down |= (uint32_t)(nan || h == (T::special | 0x8000u)) << (4 * q + e);
                                }
                            }
                            plus[w] |= saw ? up : 0u;
                            minus[w] |= saw ? down : 0u;
                        }
                    }
                }
            }
        }
    };

    // Slots of the chunk that all rows see: the committed ones; of a causal run also the new tokens up to the first row's own.
    const int64_t shared = (int64_t)sq.ctx + (a.mask ? 0 : tile0 / a.group + 1);
    const int sure = k1 < shared ? k1 : (int)shared;
    // steps of these alone, then the others
    int plain = sure > k0 ? (sure - k0) / (KW * A::BN) : 0;
    plain = plain < steps ? plain : steps;
    if (steps > 0) {
#pragma unroll
        for (int f = 0; f < A::FETCH * A::HALVES; ++f)
            if (slot_of_fetch(0, f) >= k1) entry[f] = -1;
        fetch(0);
        if (steps > 1) lookup(1, k1);
    }
    int st = 0;
    uint32_t vis[A::SUB] = {};
    if constexpr (A::REGS) {
        // a wave's own tile: once it is in registers, the next one comes to the same place
        vec8 kr[A::KR], vr[A::KR];
        for (; st < plain; ++st) {
            wait_all();
            if constexpr (R == 32) {
#pragma unroll
                for (int q = 0; q < A::QS; ++q) kr[q] = *(const vec8*)(my + kread[q % A::KV] + q / A::KV * 1024);
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int i = 0; i < A::OB; ++i) vr[g * A::OB + i] = A::v_frag(my, vread[i % A::VV] + i / A::VV * 1024 + g * A::GRP);
            } else {
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int q = 0; q < A::QS; ++q) kr[g * A::QS + q] = *(const vec8*)(my + g * A::GRP + kread[q % A::KV] + q / A::KV * 1024);
#pragma unroll
                for (int i = 0; i < A::OB; ++i) vr[i] = A::v_frag(my, vread[i % A::VV] + i / A::VV * 1024);
            }
            wait_lds();
            if (st + 1 < steps) {
                fetch(0);
                if (st + 2 < steps) lookup(st + 2, k1);
            }
            work(std::false_type{}, my, vis, kr, vr);
        }
        for (; st < steps; ++st) {
            wait_all();
            if (sight(k0 + (st * KW + kw) * A::BN, vis) != 0) work(std::true_type{}, my, vis, nullptr, nullptr);
            wait_lds();
            if (st + 1 < steps) {
                fetch(0);
                if (st + 2 < steps) lookup(st + 2, k1);
            }
        }
    } else {
        auto next = [&](int st) {   // step st is in LDS; the next one is on its way
            wait_all();
            if (RW > 1) {
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");   // no read of the tile moves up over the barrier
            }
            if (st + 1 < steps) {
                fetch((st + 1) & 1);
                if (st + 2 < steps) lookup(st + 2, k1);
            }
            return my + (st & 1) * A::STAGE;
        };
        // two loops: in one, which also runs the masked steps, the plain steps took 10% longer
        for (; st < plain; ++st) {
            const char* buf = next(st);
            work(std::false_type{}, buf, vis, nullptr, nullptr);
        }
        for (; st < steps; ++st) {
            const char* buf = next(st);
            const int seen = sight(k0 + (st * KW + kw) * A::BN, vis);
            if (D < 256 && seen == 2) work(std::false_type{}, buf, vis, nullptr, nullptr);   // at 256 dimensions it spills
            else if (seen != 0) work(std::true_type{}, buf, vis, nullptr, nullptr);
        }
    }
    l = row_sum<R>(l);
    if (l != l) m = INFINITY;   // NaN among the logits: outweighs the other slot groups and chunks, whatever the maximum here
    {
        float odd = 0.f;   // NaN where a result is not finite
#pragma unroll
        for (int i = 0; i < A::OB; ++i)
#pragma unroll
            for (int e = 0; e < (int)(sizeof(acc) / 4); ++e) odd = fmaf(o[i][e], 0.f, odd);
        uint32_t any = 0;
#pragma unroll
        for (int w = 0; w < A::PW; ++w) any |= plus[w] | minus[w];
        if (__any(any || odd != odd)) {
            // of the slots that all rows see, 16-byte pieces of several at a time; bits 0-7: +inf or NaN in that dimension, 8-15: -inf or NaN
            constexpr int PER = D / 8, ROWS = 64 / PER;
            const int piece = lane % PER;
            const char* const base = vbase - (fp ^ A::B::v_swap(fr)) * 16 + piece * 16;
            uint32_t found = 0;
            if (lane < PER * ROWS) {
#pragma unroll 4
                for (int s = k0 + lane / PER; s < sure; s += ROWS) {
                    const uint32_t p = fastdiv(s, c.page);
                    const int32_t page = table ? table[p] : seq;
                    const u32x4 x = *(const u32x4*)((uint32_t)page < c.num_pages ? base + page * c.v_page + (s - p * c.page.d) * c.v_slot : (const char*)zero_row);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t h = x[e / 2] >> (16 * (e & 1)) & 0xFFFFu;
                        const bool nan = (h & 0x7FFFu) > T::special;
                        found |= (uint32_t)(nan || h == T::special) << e | (uint32_t)(nan || h == (T::special | 0x8000u)) << (8 + e);
                    }
                }
            }
            uint32_t all = 0;   // lane p: of dimensions 8 p ..
#pragma unroll
            for (int t = 0; t < ROWS; ++t) all |= __shfl(found, piece + t * PER, 64);
            const uint32_t saw = m == -INFINITY ? 0u : ~0u;   // a row that saw nothing here counts for nothing in the joins
            const float none = l == l ? 0.f : l;
#pragma unroll
            for (int i = 0; i < A::OB; ++i)
#pragma unroll
                for (int q = 0; q < (int)(sizeof(acc) / 16); ++q) {
                    const int d = R == 32 ? 32 * i + 8 * q + 4 * (lane >> 5) : 16 * i + 4 * (lane >> 4);
                    const uint32_t bits = (uint32_t)__shfl(all, d >> 3, 64) >> (d & 4) & saw;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int at = (int)(sizeof(acc) / 4) * i + 4 * q + e;
                        const bool up = (plus[at / 32] >> (at % 32) | bits >> e) & 1u, down = (minus[at / 32] >> (at % 32) | bits >> (8 + e)) & 1u;
                        if (up || down) o[i][4 * q + e] = none + (up ? INFINITY : 0.f) - (down ? INFINITY : 0.f);
                    }
                }
        }
    }

    // join the slot groups of the workgroup, then write rows
    const bool last = nchunk == 1;
    const int64_t prow = part_rows(b.rows, a.heads);
    float* const pout = (float*)a.work;
    float2* const pml = (float2*)(a.work + (int64_t)pl.chunks * prow * D * 4);
    __syncthreads();
    if constexpr (KW > 1) {
        float* const ol = (float*)lds;
        float2* const ml = (float2*)(lds + KW * RW * R * A::OPAD * 4);
        if (lane < R) ml[(kw * RW + rw) * R + lr] = make_float2(m, l);
        __syncthreads();
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < KW; ++k) M = fmaxf(M, ml[(k * RW + rw) * R + lr].x);
        const float f = joined(m, M);
        float* mine = ol + ((kw * RW + rw) * R + lr) * A::OPAD;
        if constexpr (R == 32) {
#pragma unroll
            for (int i = 0; i < A::OB; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *(f32x4*)(mine + 32 * i + 8 * q + 4 * (lane >> 5)) = f32x4{o[i][4 * q], o[i][4 * q + 1], o[i][4 * q + 2], o[i][4 * q + 3]} * f;
        } else {
#pragma unroll
            for (int i = 0; i < A::OB; ++i) *(f32x4*)(mine + 16 * i + 4 * (lane >> 4)) = *(const f32x4*)&o[i] * f;
        }
        __syncthreads();
        constexpr int PER = D / 4, N = RW * R * PER;
        for (int e = tid; e < N; e += RW * KW * 64) {
            const int tr = e / PER, d = (e % PER) * 4, rr = tile0 + tr;
            if (rr >= rows) continue;
            float Mr = -INFINITY, lr_ = 0.f;
#pragma unroll
            for (int k = 0; k < KW; ++k) Mr = fmaxf(Mr, ml[k * RW * R + tr].x);
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                const float2 x = ml[k * RW * R + tr];
                if (x.x != -INFINITY) lr_ += x.y * joined(x.x, Mr);
            }
            f32x4 y = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KW; ++k) y += *(const f32x4*)(ol + (k * RW * R + tr) * A::OPAD + d);
            const int nd = rr / a.group;
            const int64_t orow = sq.row0 + nd;
            const int oh = kh * a.group + rr - nd * a.group;
            if (last) {
                y *= lr_ == 0.f ? 0.f : 1.f / lr_;
                typedef O ov __attribute__((ext_vector_type(4)));
                *(ov*)(a.out + orow * a.o_row + oh * a.o_head + d * sizeof(O)) = __builtin_convertvector(y, ov);
                if (d == 0 && a.lse) a.lse[orow * a.ld_lse + oh] = lr_ == 0.f ? -INFINITY : (Mr + log2f(lr_)) * 0.69314718055994530942f;
            } else {
                const int64_t at = ci * prow + orow * a.heads + oh;
                *(f32x4*)(pout + at * D + d) = y;
                if (d == 0) pml[at] = make_float2(Mr, lr_);
            }
        }
    } else {
        // 32 dimensions of the wave's rows at a time through LDS: whole row pieces leave together
        float* const mine = (float*)lds + wave * 32 * 36;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int i = 0; i < A::OB; ++i) {
            const acc x = last ? o[i] * inv : o[i];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(f32x4*)(mine + lr * 36 + 8 * q + 4 * (lane >> 5)) = f32x4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int tr = p * 8 + (lane >> 3), rr = tile0 + rw * R + tr;
                const f32x4 y = *(const f32x4*)(mine + tr * 36 + (lane & 7) * 4);
                if (rr < rows) {
                    const int nd = rr / a.group, d = 32 * i + (lane & 7) * 4;
                    const int64_t orow = sq.row0 + nd;
                    const int oh = kh * a.group + rr - nd * a.group;
                    if (last) {
                        typedef O ov __attribute__((ext_vector_type(4)));
                        *(ov*)(a.out + orow * a.o_row + oh * a.o_head + d * sizeof(O)) = __builtin_convertvector(y, ov);
                    } else {
                        *(f32x4*)(pout + (ci * prow + orow * a.heads + oh) * D + d) = y;
                    }
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        if (live && lane < R) {
            if (!last) pml[ci * prow + row * a.heads + head] = make_float2(m, l);
            else if (a.lse) a.lse[row * a.ld_lse + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
        }
    }
}

// Joins the chunks of the rows whose sequence was cut.  A wave per (row, head):
// a lane per chunk for the weights, then D / 4 lanes per row, 64 / (D / 4) rows
// at a time.  AHEAD: up to EARLY rounds of chunks are read before it is known
// how many there are; the lookups that tell take as long (5.2 instead of 8.4 us
// for 32 rows of 32 chunks, but 45 instead of 15 for 32768 rows of 2: only where
// all waves run at once).
template <int D, typename O, bool AHEAD>
__global__ __launch_bounds__(256) void k_join_chunks(KvCache c, KvBatch b, AttnArgs a, AttnPlan pl) {
    constexpr int PER = D / 4, PARTS = 64 / PER, EARLY = 16;
    const int row = wide_index(blockIdx.z), lane = threadIdx.x & 63;
    const int h = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (row >= b.rows || h >= a.heads) return;
    const int64_t prow = part_rows(b.rows, a.heads), at = (int64_t)row * a.heads + h;
    const float* const pout = (const float*)a.work + at * D;
    const float2* const pml = (const float2*)(a.work + (int64_t)pl.chunks * prow * D * 4) + at;
    const int part = lane / PER, d = (lane % PER) * 4;
    const bool early = AHEAD && pl.chunks <= EARLY * PARTS;
    f32x4 pre[AHEAD ? EARLY : 1];
    float2 first = make_float2(-INFINITY, 0.f);
    if constexpr (AHEAD) if (early) {
        if (lane < pl.chunks) first = pml[lane * prow];
#pragma unroll
        for (int i = 0; i < EARLY; ++i) {
            const int k = i * PARTS + part;
            pre[i] = f32x4{0, 0, 0, 0};
            if (k < pl.chunks) pre[i] = *(const f32x4*)(pout + (int64_t)k * prow * D + d);
        }
    }
    const int seq = row_sequence(b, row, lane);
    if (seq < 0) return;
    const Seq sq = sequence(c, b, seq);
    int nchunk = (sq.total + pl.chunk - 1) / pl.chunk;
    nchunk = nchunk > pl.chunks ? pl.chunks : nchunk;
    if (nchunk <= 1 || row - sq.row0 >= b.max_nodes) return;
    float M = -INFINITY, l = 0.f;
    f32x4 y = {0, 0, 0, 0};
    for (int k0 = 0; k0 < nchunk; k0 += 64) {
        float2 x = make_float2(-INFINITY, 0.f);
        if (k0 + lane < nchunk) x = early ? first : pml[(k0 + lane) * prow];
        float top = x.x;
#pragma unroll
        for (int t = 32; t; t >>= 1) top = fmaxf(top, __shfl_xor(top, t, 64));
        const float Mn = fmaxf(M, top);
        if (Mn == -INFINITY) continue;   // nothing seen so far
        const float f = joined(x.x, Mn);
        float ls = f == 0.f ? 0.f : x.y * f;
#pragma unroll
        for (int t = 32; t; t >>= 1) ls += __shfl_xor(ls, t, 64);
        const float keep = joined(M, Mn);
        l = l * keep + ls;
        y *= keep;
        M = Mn;
        const int n = nchunk - k0 < 64 ? nchunk - k0 : 64;
        // every lane takes every turn: the weights are lane reads, 0 where a chunk holds nothing for this row, whatever
        // its memory
        if (AHEAD && early) {
#pragma unroll
            for (int i = 0; i < (AHEAD ? EARLY : 1); ++i) {
                const int k = i * PARTS + part;
                const float w = __shfl(f, k & 63, 64);
                if (k < n && w != 0.f) y += pre[i] * w;
            }
        } else {
            for (int kb = 0; kb < n; kb += PARTS) {
                const int k = kb + part;
                const float w = __shfl(f, k & 63, 64);
                f32x4 v = {0, 0, 0, 0};
                if (k < n) v = *(const f32x4*)(pout + (int64_t)(k0 + k) * prow * D + d);
                if (k < n && w != 0.f) y += v * w;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (PARTS >= 2) y[i] += __shfl(y[i], (lane + PER) & 63, 64);
        if (PARTS == 4) y[i] += __shfl(y[i], (lane + 2 * PER) & 63, 64);
    }
    if (part != 0) return;
    y *= l == 0.f ? 0.f : 1.f / l;
    typedef O ov __attribute__((ext_vector_type(4)));
    *(ov*)(a.out + row * a.o_row + h * a.o_head + d * sizeof(O)) = __builtin_convertvector(y, ov);
    if (d == 0 && a.lse) a.lse[row * a.ld_lse + h] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994530942f;
}

template <typename T, int D, int R, int RW, int KW, int NS, typename O>
void launch_tiles(const KvCache& c, const KvBatch& b, const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
    const int64_t blocks = ((int64_t)pl.groups + 7) / 8 * 8 * pl.row_tiles;
    const dim3 grid(wide(blocks), parts(blocks));
    hipLaunchKernelGGL((k_tree_attention<T, D, R, RW, KW, NS, O>), grid, dim3(RW * KW * 64), 0, s, c, b, a, pl);
}

template <typename T, int D, int NS, typename O>
hipError_t launch_dim(const KvCache& c, const KvBatch& b, const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
    constexpr int KW = D == 256 ? 2 : 4;
    if (pl.R == 16) launch_tiles<T, D, 16, 1, KW, NS, O>(c, b, a, pl, s);
    else if (pl.RW == 1) launch_tiles<T, D, 32, 1, KW, NS, O>(c, b, a, pl, s);
    else if (pl.RW == 2) launch_tiles<T, D, 32, 2, 2, NS, O>(c, b, a, pl, s);
    else launch_tiles<T, D, 32, 4, 1, NS, O>(c, b, a, pl, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || pl.chunks == 1) return e;
    const dim3 grid(wide(b.rows), (a.heads + 3) / 4, parts(b.rows));
    if ((int64_t)b.rows * a.heads <= 2048) hipLaunchKernelGGL((k_join_chunks<D, O, true>), grid, dim3(256), 0, s, c, b, a, pl);
    else hipLaunchKernelGGL((k_join_chunks<D, O, false>), grid, dim3(256), 0, s, c, b, a, pl);
    return hipGetLastError();
}

template <typename T, int NS, typename O>
hipError_t launch_type(const KvCache& c, const KvBatch& b, const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
    if (c.dim == 64) return launch_dim<T, 64, NS, O>(c, b, a, pl, s);
    if (c.dim == 96) return launch_dim<T, 96, NS, O>(c, b, a, pl, s);
    if (c.dim == 128) return launch_dim<T, 128, NS, O>(c, b, a, pl, s);
    return launch_dim<T, 256, NS, O>(c, b, a, pl, s);
}

}  // namespace

// One instantiation per file (attn_*.hip): the cache's type and the output's.
hipError_t attn_bf16(const KvCache&, const KvBatch&, const AttnArgs&, const AttnPlan&, hipStream_t);
hipError_t attn_bf16_f32(const KvCache&, const KvBatch&, const AttnArgs&, const AttnPlan&, hipStream_t);
hipError_t attn_f16(const KvCache&, const KvBatch&, const AttnArgs&, const AttnPlan&, hipStream_t);
hipError_t attn_f16_f32(const KvCache&, const KvBatch&, const AttnArgs&, const AttnPlan&, hipStream_t);

}  // namespace bnn
