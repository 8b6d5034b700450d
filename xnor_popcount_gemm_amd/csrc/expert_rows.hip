// Grouped products with few rows to an expert: each expert's matrix is read
// once, straight from memory into the registers of the wave that multiplies
// it.
//
//     D[p, n] = sum_k q[row(p), k] w_e[n, k]    (exact int32), then the epilogue
//
// Bound by the stream of weights (1 or 2 bits each).  A workgroup of 4 waves
// has 16 columns (of both matrices, with a gate) and up to 16 MT positions of
// one expert; the waves share k, chunk by chunk, so that even a narrow matrix
// keeps every compute unit busy, and join their sums through LDS.  A
// wave's load is 1 KiB of packed weights, its 64-k steps go through the int8
// matrix cores with the weights as rows and the positions as columns: a lane
// ends with 4 neighbouring outputs of one position.  The positions' rows come
// through the caches.
#include "expert_kernel.hpp"

namespace bnn {
namespace {

constexpr int WAVES = 4;

template <bool TERN, bool GATED, int MT>
__global__ __launch_bounds__(64 * WAVES) void k_expert_rows(ExpertArgs a, int frags, int chunks, int slots) {
    constexpr int H = GATED ? 2 : 1, CK = chunk_k(TERN), STEPS = CK / 64;
    __shared__ v4i part[WAVES][H * MT][64];
    const uint32_t id = wide_index(blockIdx.y);
    const int f = (int)(id / (uint32_t)slots), slot = (int)(id % (uint32_t)slots);
    if (f >= frags) return;
    const Tile t = find_tile(a, slot, 16 * MT);
    if (t.e < 0) return;   // the same in the whole workgroup
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r16 = lane & 15, g = lane >> 4;

    const int8_t* row[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int src = source_row(a, t.p0 + min(16 * i + r16, t.n - 1));
        row[i] = a.Xq + (int64_t)max(src, 0) * a.ldXq;
    }
    const int64_t at = ((int64_t)t.e * frags + f) * chunks * 64 + lane;
    const uint4* w[2] = {a.m.W + at, GATED ? a.u.W + at : nullptr};
    v4i acc[H][MT];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[h][i] = v4i{0, 0, 0, 0};

    for (int c = wave; c < chunks; c += WAVES) {
        uint32_t bits[H][4];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const uint4 b = w[h][(int64_t)c * 64];
            bits[h][0] = b.x; bits[h][1] = b.y; bits[h][2] = b.z; bits[h][3] = b.w;
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int k = CK * c + 64 * s;
            if (k < a.K) {
                v4i x[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if (k + 64 <= a.K) x[i] = *(const v4i*)(row[i] + k + 16 * g);
                    else x[i] = masked16(row[i], k + 16 * g, a.K);
                }
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const v4i b = expand16<TERN>(bits[h], s);
#pragma unroll
                    for (int i = 0; i < MT; ++i) acc[h][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b, x[i], acc[h][i], 0, 0, 0);
                }
            }
        }
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < MT; ++i) part[wave][h * MT + i][lane] = acc[h][i];
    __syncthreads();
    for (int i = wave; i < MT; i += WAVES) {
        const int in = 16 * i + r16;
        if (in >= t.n) continue;
        const int p = t.p0 + in, src = source_row(a, p), n = 16 * f + 4 * g;
        if (src < 0 || n >= a.N) continue;
        v4i d = part[0][i][lane], du = {0, 0, 0, 0};
#pragma unroll
        for (int v = 1; v < WAVES; ++v) d += part[v][i][lane];
        if (GATED)
#pragma unroll
            for (int v = 0; v < WAVES; ++v) du += part[v][(H - 1) * MT + i][lane];
        finish<GATED>(a, p, a.xscale ? a.xscale[src] : 1.f, n, d, du, scale4(a.m, t.e, n, a.N), GATED ? scale4(a.u, t.e, n, a.N) : Scale4{});
    }
}

int rows_tile(const ExpertArgs& a) {   // 16-row fragments of a tile, by the average of an expert's rows
    const int64_t mean = a.positions / a.experts;
    return mean <= 16 ? 1 : mean <= 32 ? 2 : 4;
}

int64_t groups_of(const ExpertArgs& a) { return tile_slots(a, 16 * rows_tile(a)) * ((a.N + 15) / 16); }

}  // namespace

bool expert_rows_fits(const ExpertArgs& a, bool) { return groups_of(a) < ((int64_t)1 << 31); }

hipError_t launch_expert_rows(const ExpertArgs& a, bool ternary, hipStream_t s) {
    const int mt = rows_tile(a), frags = (a.N + 15) / 16, chunks = (a.K + chunk_k(ternary) - 1) / chunk_k(ternary);
    const int slots = (int)tile_slots(a, 16 * mt);
    const int64_t groups = groups_of(a);
    const dim3 grid(wide(groups), parts(groups)), block(64 * WAVES);
    const bool gated = a.u.W != nullptr;
#define BNN_ROWS(T, G, MT) hipLaunchKernelGGL((k_expert_rows<T, G, MT>), grid, block, 0, s, a, frags, chunks, slots)
#define BNN_ROWS_MT(T, G) \
    do { if (mt == 1) BNN_ROWS(T, G, 1); else if (mt == 2) BNN_ROWS(T, G, 2); else BNN_ROWS(T, G, 4); } while (0)
    if (ternary) { if (gated) BNN_ROWS_MT(true, true); else BNN_ROWS_MT(true, false); }
    else         { if (gated) BNN_ROWS_MT(false, true); else BNN_ROWS_MT(false, false); }
#undef BNN_ROWS_MT
#undef BNN_ROWS
    return hipGetLastError();
}

}  // namespace bnn
