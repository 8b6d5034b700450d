// Grouped products with many rows to an expert: tiles of 64 or 128 positions x
// 256 weight rows (128 of each matrix with a gate) on the int8 matrix cores.
//
//     D[p, n] = sum_k q[row(p), k] w_e[n, k]    (exact int32), then the epilogue
//
// Bound by the matrix cores and what feeds them.  Four waves share the tile by
// weight rows: each has all its positions and 64 weight rows, so that every
// weight is expanded by one wave only, in registers, straight from global
// memory (a chunk of 256 or 512 k ahead), and serves 4 or 8 matrix
// instructions.  Only the INT8 rows go through LDS: stages of 128 k, brought
// by loads to LDS three stages ahead of their use (a ring of four), the
// 16-byte pieces of a row permuted by the row so that the 8 lanes that are
// served together fall on distinct banks.  LDS reads are 32 KiB a 64-k step
// for 128 positions, half of what the matrix cores' time allows.  Two
// workgroups share a compute unit, so that one's epilogue runs beside the
// other's products (256 positions in one workgroup: 406 against 388 us for
// 8192^3, 121 against 84 us for 2000 x 11008 -> 4096).  Weights are
// the rows of an instruction and positions its columns: a lane ends with 4
// neighbouring outputs of a position.
//
// Workgroups go to the 8 XCDs in turn; each XCD takes a contiguous run of the
// tiles, in groups of 8 position tiles by weight tile, so that what is in its
// L2 is used again.
//
// 8192^3 ternary: 404-411 us, 2680-2720 TOPS (the library's int8 product of the
// same values 415-423).  16384 positions of 8 experts, 4096 -> 2 x 11008 with a
// gate: 1239-1247 us, 2370-2390 TOPS: matrix instructions take 57% of the cycles
// and vector instructions, which a SIMD does not issue beside them, 39%.
#include <type_traits>

#include "expert_kernel.hpp"

namespace bnn {
namespace {

constexpr int THREADS = 256;                // 4 waves
constexpr int FN = 4;                       // weight fragments of a wave
constexpr int ST = 128, RING = 4;           // k of a stage; stages in LDS

typedef __attribute__((address_space(3))) void* lptr_t;
#define INLINE __attribute__((always_inline))   // lambdas that are called from many places and hold references to the sums

template <int I> using Ic = std::integral_constant<int, I>;

// s_waitcnt that leaves at most n vector-memory operations outstanding (vmcnt
// in bits 3:0 and 15:14) and no LDS access (lgkmcnt, bits 11:8).
constexpr unsigned vmcnt(int n) { return (unsigned)(n & 0xF) | ((unsigned)((n >> 4) & 3) << 14) | (0x7u << 4); }

// A barrier without the fence of __syncthreads(), which would wait for every
// load to LDS in flight.  The caller has waited for its loads that the others
// read next, and for its own reads of the buffer that is filled next.
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// MF: fragments of 16 positions in a tile.
template <bool TERN, bool GATED, int MF>
__global__ __launch_bounds__(THREADS, MF == 4 ? 3 : 2) void k_expert_tile(ExpertArgs a, int frags, int chunks, int tiles_n, uint32_t x_bytes) {
    constexpr int BM = 16 * MF, CK = chunk_k(TERN), CS = CK / ST;   // stages of a weight chunk
    constexpr int PIECES = BM * ST / 16 / THREADS;                  // 16-byte loads of a lane for a stage
    __shared__ __attribute__((aligned(16))) int8_t lds0[BM * ST], lds1[BM * ST], lds2[BM * ST], lds3[BM * ST];
    auto buf = [&](auto I) -> int8_t* {
        constexpr int i = decltype(I)::value % RING;
        if constexpr (i == 0) return lds0;
        else if constexpr (i == 1) return lds1;
        else if constexpr (i == 2) return lds2;
        else return lds3;
    };
    __shared__ int source[BM];
    __shared__ float factor[BM];
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // which tile
    const Tiles tiles(a, BM);
    const int slots = tiles.count();
    const int total = slots * tiles_n, run = (total + 7) / 8;
    const int place = (int)(blockIdx.x >> 3), tile = (int)(blockIdx.x & 7) * run + place;
    if (place >= run || tile >= total) return;
    constexpr int GROUP = 8;
    const int grp = tile / (GROUP * tiles_n), first = grp * GROUP, size = min(slots - first, GROUP), in = tile - first * tiles_n;
    const Tile t = tiles[first + in % size];
    if (t.e < 0) return;
    const int tn = in / size;

    if (tid < t.n) {
        const int src = source_row(a, t.p0 + tid);
        source[tid] = src;
        factor[tid] = a.xscale && src >= 0 ? a.xscale[src] : 1.f;
    }

    // INT8 rows: load i of the wave brings tile rows 8 (PIECES wave + i) .. + 7, lane l the piece of row l / 8
    // that belongs at place l % 8
    const __amdgpu_buffer_rsrc_t xr = rsrc_of(a.Xq, x_bytes);
    uint32_t off[PIECES];
    const uint32_t piece = (uint32_t)(((lane & 7) ^ (lane >> 3)) << 4);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int row = 8 * (PIECES * wave + i) + (lane >> 3);
        const int src = source_row(a, t.p0 + min(row, t.n - 1));
        off[i] = (uint32_t)max(src, 0) * (uint32_t)a.ldXq + piece;
    }
    auto issue = [&](auto I, int s) INLINE {
        int8_t* to = buf(I) + PIECES * wave * 1024;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lptr_t)(to + i * 1024), 16, (int)off[i], s * ST, 0, 0);
    };
    auto issue_last = [&](auto I, int s) INLINE {     // the stage that holds the rows' end, through registers
        int8_t* to = buf(I) + PIECES * wave * 1024;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) *(v4i*)(to + i * 1024 + 16 * lane) = masked16(a.Xq + (off[i] - piece), s * ST + (int)piece, a.K);
    };

    // weights: fragment q of the wave, a chunk at a time
    const uint4* w[FN];
#pragma unroll
    for (int q = 0; q < FN; ++q) {
        const int f = GATED ? 8 * tn + 2 * wave + (q >> 1) : 16 * tn + 4 * wave + q;
        w[q] = (GATED && (q & 1) ? a.u.W : a.m.W) + ((int64_t)t.e * frags + min(f, frags - 1)) * chunks * 64;
    }
    uint32_t now[FN][4], next[FN][4];
    auto fetch = [&](int c) INLINE {
        const int64_t to = (int64_t)min(c, chunks - 1) * 64;
#pragma unroll
        for (int q = 0; q < FN; ++q) {
            const uint4 b = (w[q] + to)[lane];
            next[q][0] = b.x; next[q][1] = b.y; next[q][2] = b.z; next[q][3] = b.w;
        }
    };

    v4i acc[MF][FN];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int q = 0; q < FN; ++q) acc[i][q] = v4i{0, 0, 0, 0};
    int at[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) at[u] = r16 * ST + (((4 * u + g) ^ (r16 & 7)) << 4);

    // The two 64-k steps of stage P of a chunk group.
    constexpr int AHEAD = 4;                   // row fragments that are read before their use
    auto compute = [&](auto P) INLINE {
        const int8_t* x = buf(P);
        constexpr int step = 2 * (decltype(P)::value % CS);
        v4i xv[AHEAD], b[FN];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) xv[i] = *(const v4i*)(x + at[0] + i * 16 * ST);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int q = 0; q < FN; ++q) b[q] = expand16<TERN>(now[q], step + u);
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                const int y = u * MF + i, z = y + AHEAD;
#pragma unroll
                for (int q = 0; q < FN; ++q) acc[i][q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[q], xv[y % AHEAD], acc[i][q], 0, 0, 0);
                if (z < 2 * MF) xv[y % AHEAD] = *(const v4i*)(x + at[z / MF] + (z % MF) * 16 * ST);
            }
        }
    };

    const int stages = (a.K + ST - 1) / ST, full = a.K / ST;
    auto issue_any = [&](auto I, int s) INLINE {
        if (s < full) issue(I, s);
        else if (s < stages) issue_last(I, s);
    };
    auto turn_chunk = [&](int s) INLINE {
#pragma unroll
        for (int q = 0; q < FN; ++q)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                now[q][d] = next[q][d];
                asm volatile("" : "+v"(now[q][d]));   // not expanded, and waited for, a stage earlier
            }
        fetch(s / CS + 1);
    };
    // A stage whose loads, and those that it starts, lie within the rows.  A
    // stage asks for weights (every CS stages), then for rows, so its own rows,
    // asked for three stages ago, are there when at most the rows of the next
    // two stages are outstanding, and the weights asked for in the last two.
    auto fast_stage = [&](int s, auto P) INLINE {
        constexpr int p = decltype(P)::value;
        constexpr int asked = (p + CS - 1) % CS == 0 || (p + CS - 2) % CS == 0 ? FN : 0;
        __builtin_amdgcn_s_waitcnt(vmcnt(2 * PIECES + asked));
        barrier();
        // With 64 positions the order is given (17 against 18.5 us for 64 experts; left free it also spills); with 128 it
        // is left to the compiler (2 x 11008 x 4096: 1325 against 1350 us).
        if constexpr (p % CS == 0) turn_chunk(s);
        if constexpr (MF == 4) {
            __builtin_amdgcn_sched_barrier(0);
            compute(P);
            __builtin_amdgcn_sched_barrier(0);
        }
        issue(Ic<p + 3>{}, s + 3);
        if constexpr (MF != 4) compute(P);
    };
    auto stage = [&](int s, auto P) INLINE {
        constexpr int p = decltype(P)::value;
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if constexpr (p % CS == 0) turn_chunk(s);
        issue_any(Ic<p + 3>{}, s + 3);
        compute(P);
    };
    int s = 0;
    if (s + 6 < full) {
        // the order of these loads is counted on: keep it
        issue(Ic<0>{}, 0);
        asm volatile("" ::: "memory");
        fetch(0);
        asm volatile("" ::: "memory");
        issue(Ic<1>{}, 1);
        asm volatile("" ::: "memory");
        issue(Ic<2>{}, 2);
        do {
            fast_stage(s, Ic<0>{});
            fast_stage(s + 1, Ic<1>{});
            fast_stage(s + 2, Ic<2>{});
            fast_stage(s + 3, Ic<3>{});
            s += 4;
        } while (s + 6 < full);
    } else {
        fetch(0);
        issue_any(Ic<0>{}, 0);
        issue_any(Ic<1>{}, 1);
        issue_any(Ic<2>{}, 2);
    }
    for (; s < stages; s += 4) {
        stage(s, Ic<0>{});
        if (s + 1 < stages) stage(s + 1, Ic<1>{});
        if (s + 2 < stages) stage(s + 2, Ic<2>{});
        if (s + 3 < stages) stage(s + 3, Ic<3>{});
    }

    // Epilogue.  The ring is free: each wave parks 32 columns of its sums at a time in a buffer of its own (16-byte
    // pieces permuted by the row, as above) and reads them back row by row, so that neighbouring lanes store
    // neighbouring columns and the code for an output stands here once.
    int8_t* mine = wave == 0 ? lds0 : wave == 1 ? lds1 : wave == 2 ? lds2 : lds3;
#pragma unroll
    for (int c = 0; c < FN / 2; ++c) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) *(v4i*)(mine + (16 * i + r16) * 128 + (((4 * h + g) ^ (r16 & 7)) << 4)) = acc[i][2 * c + h];
        __syncthreads();
        constexpr int LANES = GATED ? 4 : 8;          // of a row
        const int f = GATED ? 8 * tn + 2 * wave + c : 16 * tn + 4 * wave + 2 * c;
        const int j = lane % LANES, n = 16 * f + 4 * j;
        if (n < a.N) {
            const Scale4 sm = scale4(a.m, t.e, n, a.N), su = GATED ? scale4(a.u, t.e, n, a.N) : Scale4{};
#pragma unroll 1
            for (int row = lane / LANES; row < t.n; row += 64 / LANES) {
                if (source[row] < 0) continue;
                const int8_t* at_row = mine + row * 128;
                const v4i d = *(const v4i*)(at_row + ((j ^ (row & 7)) << 4));
                const v4i du = GATED ? *(const v4i*)(at_row + (((4 + j) ^ (row & 7)) << 4)) : v4i{0, 0, 0, 0};
                finish<GATED>(a, t.p0 + row, factor[row], n, d, du, sm, su);
            }
        }
    }
}

int64_t tiles_of(const ExpertArgs& a, int rows) {
    const int64_t cols = a.u.W ? 128 : 256;
    return (tile_slots(a, rows) * ((a.N + cols - 1) / cols) + 7) / 8 * 8;
}

// 128 positions where that gives two workgroups to each compute unit and an
// expert has so many, otherwise 64 (8 x 2048 positions, 4096 -> 11008 with a
// gate: 1353 against 1418 us; 8 x 256, 4096 -> 4096: 44 against 39).
int tile_rows(const ExpertArgs& a) { return a.positions / a.experts >= 96 && tiles_of(a, 128) >= 512 ? 128 : 64; }

}  // namespace

// From 24 rows of an expert where the tiles give two workgroups to each
// compute unit (8 x 32 rows, 4096 -> 2 x 11008: 48 against 62 us with
// expert_rows.hip), from 40 always (8 x 32 rows, 11008 -> 4096, 128 tiles: 48
// against 39; 8 x 48: 50 against 63).  Offsets into Xq are 32 bits here.
bool expert_tile_takes(const ExpertArgs& a) {
    const int64_t mean = a.positions / a.experts, tiles = tiles_of(a, 64);
    return (mean > 40 || (mean >= 24 && tiles >= 512)) && (int64_t)a.rows * a.ldXq < ((int64_t)1 << 31) && tiles < ((int64_t)1 << 24);
}

hipError_t launch_expert_tile(const ExpertArgs& a, bool ternary, hipStream_t s) {
    const int cols = a.u.W ? 128 : 256, frags = (a.N + 15) / 16, chunks = (a.K + chunk_k(ternary) - 1) / chunk_k(ternary);
    const int tiles_n = (a.N + cols - 1) / cols, rows = tile_rows(a);
    const uint32_t x_bytes = (uint32_t)(a.rows * a.ldXq);
    const dim3 grid((unsigned)tiles_of(a, rows)), block(THREADS);
    const bool gated = a.u.W != nullptr;
#define BNN_TILE(T, G, MF) hipLaunchKernelGGL((k_expert_tile<T, G, MF>), grid, block, 0, s, a, frags, chunks, tiles_n, x_bytes)
#define BNN_TILE_MF(T, G) do { if (rows == 128) BNN_TILE(T, G, 8); else BNN_TILE(T, G, 4); } while (0)
    if (ternary) { if (gated) BNN_TILE_MF(true, true); else BNN_TILE_MF(true, false); }
    else         { if (gated) BNN_TILE_MF(false, true); else BNN_TILE_MF(false, false); }
#undef BNN_TILE_MF
#undef BNN_TILE
    return hipGetLastError();
}

}  // namespace bnn
