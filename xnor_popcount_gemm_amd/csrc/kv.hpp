// What the kernels over the decoder's paged key/value cache share: the cache
// and batch descriptors as they are passed to a kernel, slot addressing, the
// lookup of a token's sequence, and the 16-bit types.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bnn {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// n / d for 0 <= n < 2^31 without a division: q = (umulhi(n, mul) + n) >> shift
// with shift = ceil(log2 d), mul = floor(2^32 (2^shift - d) / d) + 1.
struct FastDiv {
    uint32_t d, mul, shift;
};

inline FastDiv make_fastdiv(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)((((1ull << f.shift) - d) << 32) / d + 1);
    return f;
}

__device__ __forceinline__ uint32_t fastdiv(uint32_t n, FastDiv f) {
    return (__umulhi(n, f.mul) + n) >> f.shift;
}

// A paged cache.  Strides are in bytes.
struct KvCache {
    char* K; int64_t k_page, k_slot, k_head;
    char* V; int64_t v_page, v_slot, v_head;
    const int32_t* table; int64_t ld_table;
    uint32_t num_pages;
    FastDiv page;       // page size
    int32_t capacity;   // slots per sequence
    int32_t kv_heads, dim;
};

// The new tokens of a step.
struct KvBatch {
    const int32_t* indptr;
    const int32_t* ctx;
    int32_t B, rows, max_nodes, max_ctx;
};

// The rows of the token tensors that belong to a sequence and its slots.
struct Seq {
    int32_t row0, nodes;   // first row, new tokens (rows within the buffer only)
    int32_t ctx, total;    // committed slots; slots in use, both within the capacity
};

__device__ __forceinline__ Seq sequence(const KvCache& c, const KvBatch& b, int s) {
    const int64_t r0 = b.indptr[s], r1 = b.indptr[s + 1];
    const int64_t lo = r0 < 0 ? 0 : (r0 < b.rows ? r0 : b.rows), hi = r1 < lo ? lo : (r1 < b.rows ? r1 : b.rows);
    const int32_t held = b.ctx[s];
    Seq q;
    q.row0 = (int32_t)lo;
    q.nodes = (int32_t)(hi - lo);
    q.ctx = held < 0 ? 0 : (held < c.capacity ? held : c.capacity);
    q.total = (int32_t)((int64_t)q.ctx + q.nodes < c.capacity ? (int64_t)q.ctx + q.nodes : c.capacity);
    return q;
}

// Page of slot s of sequence b and the slot's place in it; a page outside
// the cache is reported as negative.
__device__ __forceinline__ int32_t slot_page(const KvCache& c, int b, uint32_t s, uint32_t& place) {
    const uint32_t p = fastdiv(s, c.page);
    place = s - p * c.page.d;
    const int32_t pg = c.table ? c.table[(int64_t)b * c.ld_table + p] : b;
    return (uint32_t)pg < c.num_pages ? pg : -1;
}

// Sequence of a row: the last s with indptr[s] <= row; each lane tests one
// entry per step, so a step covers 64 sequences.  -1: the row is past the
// last sequence (or before the first).
__device__ __forceinline__ int row_sequence(const KvBatch& b, int row, int lane) {
    int n = 0;
    for (int s0 = 0; s0 <= b.B; s0 += 64) {
        const int s = s0 + lane;
        const bool at = s <= b.B && b.indptr[s <= b.B ? s : b.B] <= row;
        n += __popcll(__ballot(at));
    }
    return n > b.B ? -1 : n - 1;
}

// The bit of a packed row; bits past the row's words are 0.
__device__ __forceinline__ bool packed_bit(const uint32_t* row, int64_t words, int32_t i) {
    return (i >> 5) < words && ((row[i >> 5] >> (i & 31)) & 1u);
}

// A launch takes fewer than 2^32 threads along a dimension; more than 2^20
// workgroups go on in a second one, `part`.
constexpr int64_t WIDE = (int64_t)1 << 20;
inline unsigned wide(int64_t groups) { return (unsigned)(groups < WIDE ? groups : WIDE); }
inline unsigned parts(int64_t groups) { return (unsigned)((groups + WIDE - 1) / WIDE); }
__device__ __forceinline__ uint32_t wide_index(uint32_t part) { return part * (uint32_t)WIDE + blockIdx.x; }

// A row of zeros, read in place of a row that is not there.
namespace {
__device__ __align__(64) const uint32_t zero_row[128] = {};
}

// 16 bytes per lane from g to LDS at lds + 16 * lane.  In asm so that the
// compiler does not make every LDS read wait for it; the caller waits.
__device__ __forceinline__ void dma16(const char* g, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" :: "s"(lds), "v"(g) : "memory");
}

// The same, not kept in the caches: for rows that are read once, and only by
// whole 128-byte lines (half lines came from memory twice).
__device__ __forceinline__ void dma16_once(const char* g, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" :: "s"(lds), "v"(g) : "memory");
}

__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void wait_all() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }

// K or V rows of 16 slots in LDS, as loads of 1 KiB per wave bring them: blocks
// of 8 rows of 128 bytes (LINES, if the dimensions are a multiple of 64), or 16
// rows of 64.  Whole lines are needed to read past the caches; half lines take
// half the page lookups per lane.
// Piece c (8 dimensions) of row r lies at place_of(r, c, swap), its place in
// the row permuted by the XOR of k_swap(r) or v_swap(r).
template <int D, bool LINES>
struct Block16 {
    static constexpr bool WIDE = LINES && D % 64 == 0;
    static constexpr int PIECES = WIDE ? 8 : 4;      // of a row in a block
    static constexpr int HALVES = WIDE ? 2 : 1;      // blocks over the 16 rows
    static constexpr int COLS = D / 8 / PIECES;      // blocks over a row
    static __host__ __device__ constexpr int k_swap(int r) { return WIDE ? r & 7 : (r >> 1) & 3; }
    static __host__ __device__ constexpr int v_swap(int r) { return WIDE ? 2 * (r & 3) : 2 * ((r >> 1) & 1); }
    static __device__ __forceinline__ int place_of(int r, int c, int swap) {
        const int half = WIDE ? r >> 3 : 0, in = WIDE ? r & 7 : r;
        return (half * COLS + c / PIECES) * 1024 + in * (16 * PIECES) + ((c % PIECES) ^ swap) * 16;
    }
};

struct Bf16 {
    typedef __bf16 elem;
    typedef bf16x8 vec8;
    typedef bf16x4 vec4;
    static constexpr uint32_t special = 0x7F80;  // exponent field of NaN and infinities
};

struct F16 {
    typedef _Float16 elem;
    typedef f16x8 vec8;
    typedef f16x4 vec4;
    static constexpr uint32_t special = 0x7C00;
};

}  // namespace bnn
