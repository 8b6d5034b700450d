// Grouped products with few rows to an expert: each expert's matrix is read
// once, straight from memory into the registers of the wave that multiplies
// it.
//
//     D[p, n] = sum_k q[row(p), k] w_e[n, k]    (exact int32), then the epilogue
//
// Bound by the stream of weights (1 or 2 bits each).  A workgroup of 4 or 8 waves
// has 16 F weight rows (half of each matrix with a gate) and up to 16 MT
// positions of one expert; the waves share k, chunk by chunk, so that even a
// narrow matrix keeps every compute unit busy, and join their sums through
// LDS.  A wave's load is 1 KiB of packed weights; the loads of its next chunk
// are in flight while it multiplies.  Weights are the rows of a matrix
// instruction and positions its columns: a lane ends with 4 neighbouring
// outputs of one position.  The positions' INT8 rows come through the caches,
// once for F fragments.
//
// 8 experts, 128 rows in uneven shares, 11008 -> 4096, weights from memory:
// 28-33 us, 3 TB/s (from the last-level cache 18-24); 2 rows, 4096 -> 2 x
// 11008: 12.4 us, 3.6 TB/s, a third of it the lookups before the stream.
#include "bnn_device.hpp"
#include "expert_kernel.hpp"

namespace bnn {
namespace {

// Waves that share k: more where there are few workgroups (2 rows, 11008 -> 4096: 9.4 against 12.2 us), not otherwise
// (8 x 8 rows, 4096 -> 2 x 11008: 72 against 55).
constexpr int waves_of(int f) { return f == 2 ? 8 : 4; }

template <bool TERN, bool GATED, int MT, int F>
__global__ __launch_bounds__(64 * waves_of(F), MT * F > 4 ? 3 : 4) void k_expert_rows(ExpertArgs a, int frags, int chunks) {
    constexpr int WAVES = waves_of(F), CK = chunk_k(TERN), STEPS = CK / 64, COLS = GATED ? F / 2 : F;   // fragments of columns
    __shared__ v4i part[WAVES][F * MT][64];
    // The tiles that there are, not those that there could be, to neighbouring workgroups: with gaps between them some
    // compute units had twice as many as others (8 x 16 rows,
    // 11008 -> 4096, 8 of 15 possible tiles, weights in the last-level cache: 30 against 20 us).
    const Tiles tiles(a, 16 * MT);
    const uint32_t id = wide_index(blockIdx.y), slots = (uint32_t)tiles.count();
    if (slots == 0) return;
    const int f0 = (int)(id / slots) * COLS, slot = (int)(id % slots);
    if (f0 >= frags) return;
    const Tile t = tiles[slot];
    if (t.e < 0) return;   // the same in the whole workgroup
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    const uint4* w[F];
#pragma unroll
    for (int q = 0; q < F; ++q)
        w[q] = (GATED && q >= COLS ? a.u.W : a.m.W) + ((int64_t)t.e * frags + min(f0 + q % COLS, frags - 1)) * chunks * 64;
    v4i acc[F][MT];
#pragma unroll
    for (int q = 0; q < F; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[q][i] = v4i{0, 0, 0, 0};

    u32x4 next[F];
    const auto fetch = [&](int c) {
        const int64_t to = (int64_t)min(c, chunks - 1) * 64;
#pragma unroll
        for (int q = 0; q < F; ++q) {
            const u32x4* from = (const u32x4*)(w[q] + to) + lane;
            // past the caches where few an expert has more than one tile (8 x 8 rows, 11008 -> 4096: 22 against 24 us; with
            // two tiles to an expert 43 against 40)
            next[q] = MT == 1 ? __builtin_nontemporal_load(from) : *from;
        }
    };
    fetch(wave);   // on its way while the rows are looked up
    const int8_t* row[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int src = source_row(a, t.p0 + min(16 * i + r16, t.n - 1));
        row[i] = a.Xq + (int64_t)max(src, 0) * a.ldXq;
    }
    // the rows of the next chunk that lies within K, too, where they take few registers
    constexpr bool EARLY = STEPS * MT <= 4;
    v4i ahead[STEPS][MT];
    const int whole = a.K / CK;
    const auto load_rows = [&](v4i (&to)[STEPS][MT], int c) {
        const int k = CK * min(c, whole - 1) + 16 * g;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int i = 0; i < MT; ++i) to[s][i] = *(const v4i*)(row[i] + k + 64 * s);
    };
    if (EARLY && whole > 0) load_rows(ahead, wave);
    for (int c = wave; c < chunks; c += WAVES) {
        uint32_t bits[F][4];
#pragma unroll
        for (int q = 0; q < F; ++q) { bits[q][0] = next[q][0]; bits[q][1] = next[q][1]; bits[q][2] = next[q][2]; bits[q][3] = next[q][3]; }
        fetch(c + WAVES);
        const auto step = [&](int s, const v4i (&x)[MT]) {
#pragma unroll
            for (int q = 0; q < F; ++q) {
                const v4i b = expand16<TERN>(bits[q], s);
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[q][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b, x[i], acc[q][i], 0, 0, 0);
            }
        };
        const int k0 = CK * c + 16 * g;
        if (c < whole) {
            v4i x[STEPS][MT];
            if (EARLY) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
#pragma unroll
                    for (int i = 0; i < MT; ++i) x[s][i] = ahead[s][i];
                load_rows(ahead, c + WAVES);
            } else {
                load_rows(x, c);
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) step(s, x[s]);
        } else {
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
                if (CK * c + 64 * s < a.K) {
                    v4i x[MT];
#pragma unroll
                    for (int i = 0; i < MT; ++i) x[i] = masked16(row[i], k0 + 64 * s, a.K);
                    step(s, x);
                }
        }
    }
#pragma unroll
    for (int q = 0; q < F; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i) part[wave][q * MT + i][lane] = acc[q][i];
    __syncthreads();
    for (int j = wave; j < COLS * MT; j += WAVES) {
        const int q = j / MT, i = j % MT, in = 16 * i + r16, n = 16 * (f0 + q) + 4 * g;
        if (in >= t.n || n >= a.N) continue;
        const int p = t.p0 + in, src = source_row(a, p);
        if (src < 0) continue;
        v4i d = {0, 0, 0, 0}, du = {0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < WAVES; ++v) {
            d += part[v][j][lane];
            if (GATED) du += part[v][COLS * MT + j][lane];
        }
        finish<GATED>(a, p, a.xscale ? a.xscale[src] : 1.f, n, d, du, scale4(a.m, t.e, n, a.N), GATED ? scale4(a.u, t.e, n, a.N) : Scale4{});
    }
}

// 16-row fragments of a tile, by the average of an expert's rows: with 16 on average many an expert has more, and reads
// its weights twice (8 experts, 128 rows in uneven shares, 11008 -> 4096: 27 us with 1, 24 with 2; 64 rows: 18 and 19).
int rows_tile(const ExpertArgs& a) { return a.positions / a.experts <= 12 ? 1 : 2; }

int64_t groups_of(const ExpertArgs& a, int f) {
    const int cols = 16 * (a.u.W ? f / 2 : f);
    return tile_slots(a, 16 * rows_tile(a)) * ((a.N + cols - 1) / cols);
}

// Weight fragments of a wave: 4, to read the INT8 rows seldom (8 x 16 rows, 11008 -> 4096: 20 against 26 us), but 2 where
// that gives fewer than two workgroups to a compute unit (2 rows, 11008 -> 4096: 7.7 against 9.3).
int rows_frags(const ExpertArgs& a) { return groups_of(a, 4) >= 512 ? 4 : 2; }

}  // namespace

bool expert_rows_fits(const ExpertArgs& a, bool) { return groups_of(a, 2) < ((int64_t)1 << 31); }

hipError_t launch_expert_rows(const ExpertArgs& a, bool ternary, hipStream_t s) {
    const int mt = rows_tile(a), f = rows_frags(a), frags = (a.N + 15) / 16, chunks = (a.K + chunk_k(ternary) - 1) / chunk_k(ternary);
    const int64_t groups = groups_of(a, f);
    const dim3 grid(wide(groups), parts(groups)), block(64 * waves_of(f));
    const bool gated = a.u.W != nullptr;
#define BNN_ROWS(T, G, MT, F) hipLaunchKernelGGL((k_expert_rows<T, G, MT, F>), grid, block, 0, s, a, frags, chunks)
#define BNN_ROWS_F(T, G, MT) do { if (f == 4) BNN_ROWS(T, G, MT, 4); else BNN_ROWS(T, G, MT, 2); } while (0)
#define BNN_ROWS_MT(T, G) \
    do { if (mt == 1) BNN_ROWS_F(T, G, 1); else BNN_ROWS_F(T, G, 2); } while (0)
    if (ternary) { if (gated) BNN_ROWS_MT(true, true); else BNN_ROWS_MT(true, false); }
    else         { if (gated) BNN_ROWS_MT(false, true); else BNN_ROWS_MT(false, false); }
#undef BNN_ROWS_MT
#undef BNN_ROWS_F
#undef BNN_ROWS
    return hipGetLastError();
}

}  // namespace bnn
