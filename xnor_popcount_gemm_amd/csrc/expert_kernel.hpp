// What the kernels of the grouped products share: which expert and positions a
// tile has, the expansion of packed weights, the epilogue.
#pragma once

#include "ffn.hpp"

namespace bnn {

typedef int v4i __attribute__((ext_vector_type(4)));

// 4 weights as bytes -1, 0, +1: codes at bits 2 d + {0, 8, 16, 24} of a
// ternary word, d < 4, or at bits d + {0, 8, 16, 24} of a binary one, d < 8.
template <bool TERN>
__device__ __forceinline__ int expand4(uint32_t w, int d) {
    return TERN ? (int)__builtin_amdgcn_perm(0u, 0xFF000100u, (w >> (2 * d)) & 0x03030303u)
                : (int)__builtin_amdgcn_perm(0u, 0x0000FF01u, (w >> d) & 0x01010101u);
}

// The 16 bytes of a lane's fragment of 64-k step s of its chunk.
template <bool TERN>
__device__ __forceinline__ v4i expand16(const uint32_t (&w)[4], int s) {
    v4i r;
#pragma unroll
    for (int d = 0; d < 4; ++d) r[d] = TERN ? expand4<true>(w[s], d) : expand4<false>(w[s >> 1], 4 * (s & 1) + d);
    return r;
}

// 16 bytes of an INT8 row from k on (a multiple of 16), 0 from K on.  A piece
// that begins below K ends within the row's stride, a multiple of 16.
__device__ __forceinline__ v4i masked16(const int8_t* row, int k, int K) {
    v4i v = {0, 0, 0, 0};
    if (k >= K) return v;
    v = *(const v4i*)(row + k);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int left = K - k - 4 * d;
        v[d] &= left >= 4 ? ~0 : left <= 0 ? 0 : (int)((1u << (8 * left)) - 1u);
    }
    return v;
}

// The positions cut into tiles of `size` within each expert.  Every lane of the
// wave calls its functions; the offsets of the first 64 experts are read once.
struct Tile {
    int e, p0, n;   // expert (-1: there are not so many tiles), first position, positions
};

class Tiles {
    // Lane l: positions lo .. hi-1 of expert e0 + l, their tiles, and the tiles up to and with them.
    struct Span {
        int lo, hi, n, sum;
    };

    __device__ __forceinline__ Span span(int e0) const {
        const int lane = threadIdx.x & 63, e = e0 + lane;
        Span s = {0, 0, 0, 0};
        if (e < a.experts) {   // offsets out of order or range give no positions
            s.lo = max(a.offsets[e], 0);
            s.hi = min(a.offsets[e + 1], a.positions);
        }
        s.sum = s.n = s.hi > s.lo ? (s.hi - s.lo + size - 1) / size : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(s.sum, d, 64);
            if (lane >= d) s.sum += o;
        }
        return s;
    }

    const ExpertArgs& a;
    const int size;
    Span first;

public:
    __device__ __forceinline__ Tiles(const ExpertArgs& args, int tile) : a(args), size(tile), first{0, 0, 0, 0} {
        if (a.offsets) first = span(0);
    }

    __device__ __forceinline__ int count() const {
        if (!a.offsets) return (a.positions + size - 1) / size;
        int all = __shfl(first.sum, 63, 64);
        for (int e0 = 64; e0 < a.experts; e0 += 64) all += __shfl(span(e0).sum, 63, 64);
        return __builtin_amdgcn_readfirstlane(all);
    }

    __device__ __forceinline__ Tile operator[](int slot) const {
        if (!a.offsets) {
            const int p0 = slot * size;
            return p0 < a.positions ? Tile{0, p0, min(size, a.positions - p0)} : Tile{-1, 0, 0};
        }
        int before = 0;
        Span s = first;
        for (int e0 = 0;;) {
            const uint64_t past = __ballot(before + s.sum > slot);
            if (past) {
                const int at = __ffsll((unsigned long long)past) - 1;
                const int i = slot - before - __shfl(s.sum - s.n, at, 64), end = __shfl(s.hi, at, 64);
                const int64_t p0 = __shfl(s.lo, at, 64) + (int64_t)i * size;
                if (i < 0 || p0 >= end) return {-1, 0, 0};   // offsets that decrease
                return {__builtin_amdgcn_readfirstlane(e0 + at), __builtin_amdgcn_readfirstlane((int)p0),
                        __builtin_amdgcn_readfirstlane(min(size, end - (int)p0))};
            }
            before += __shfl(s.sum, 63, 64);
            e0 += 64;
            if (e0 >= a.experts) return {-1, 0, 0};
            s = span(e0);
        }
    }
};

// Tiles that cover any offsets.
inline int64_t tile_slots(const ExpertArgs& a, int64_t size) {
    const int64_t p = a.positions, e = a.experts < p ? a.experts : p;
    if (!a.offsets) return (p + size - 1) / size;
    const int64_t n = (p + e * (size - 1)) / size;
    return n < p ? n : p;
}

// Row of Xq of a position; -1: none.
__device__ __forceinline__ int source_row(const ExpertArgs& a, int p) {
    if (!a.order) return p;
    const int o = a.order[p];
    const uint32_t r = o < 0 ? 0xFFFFFFFFu : fastdiv((uint32_t)o, a.per_row);
    return r < (uint32_t)a.rows ? (int)r : -1;
}

enum : int32_t { ACT_NONE = 0, ACT_RELU = 1, ACT_RELU2 = 2, ACT_SILU = 3, ACT_GELU = 4, ACT_GELU_TANH = 5 };

// z / (1 + exp(-t)): z s / (1 + s) for t < 0, z / (1 + s) otherwise, with s = exp(-|t|), which overflows for no t.  The
// hardware's exponential and reciprocal, an ulp each, because vector operations and matrix instructions take turns on a
// SIMD.  The exponent -|t| log2 e is cut at 2^-14, where it is exact, and what is left of it is multiplied on: as a
// rounded product it would put |t| 2^-24 into the result.  exp2 gives 2^40 s, because it takes what is below 2^-126 as 0
// and the result's range goes further.  In units of 2^-24 the result is off by 4.3 at most (8 by adding up the roundings);
// with expf and a division by 2.8, and 0 below t = -88.7; with exp2 of the rounded product by 33 for t in -40 .. -20.
// 16384 x 4096 -> 2 x 11008: 1246, 1282 and 1222 us.
__device__ __forceinline__ float sigmoid_times(float z, float t) {
    const float m = fminf(fabsf(t), 160.f);
    const float a = fmaf(m, -1.44269504f, 768.f), hi = a - 768.f;   // a in 512 .. 768: steps of 2^-14
    const float left = fmaf(hi, 1.90465421e-9f, fmaf(hi, -0.693147182f, -m));   // -m - hi ln 2
    float s = __builtin_amdgcn_exp2f(a - 728.f);
    s = fmaf(s, left, s);
    const float r = __builtin_amdgcn_rcpf(fmaf(s, 0x1p-40f, 1.f));
    return (t < 0.f ? z * s * 0x1p-40f : z) * r;
}

__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
    case ACT_RELU: return z < 0.f ? 0.f : z;   // NaN stays
    case ACT_RELU2: return z < 0.f ? 0.f : z * z;
    case ACT_SILU: return sigmoid_times(z, z);
    case ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    case ACT_GELU_TANH: {
        const float t = 1.5957691216057308f * (z + 0.044715f * z * z * z);   // 1 + tanh(t / 2) = 2 / (1 + exp(-t))
        return sigmoid_times(z, t);
    }
    default: return z;
    }
}

// Whether the 4 values from p on, column n, can be read or written together.
template <typename E>
__device__ __forceinline__ bool together(const E* p, int n, int N) { return n + 4 <= N && (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(E) - 1)) == 0; }

// alpha[n .. n+3] and the like of expert e; entries past N are not read.
__device__ __forceinline__ f32x4 row4(const float* p, int64_t ld, int e, int n, int N) {
    const float* q = p + (int64_t)e * ld + n;
    f32x4 v = {0, 0, 0, 0};
    if (together(q, n, N)) return *(const f32x4*)q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < N) v[i] = q[i];
    return v;
}

// alpha and bias of 4 columns of a matrix.
struct Scale4 {
    f32x4 alpha, bias;
    bool has_bias;
};

__device__ __forceinline__ Scale4 scale4(const ExpertMatrix& m, int e, int n, int N) {
    Scale4 s;
    if (m.ld_alpha == 0) s.alpha = f32x4{} + m.alpha[e];
    else s.alpha = row4(m.alpha, m.ld_alpha, e, n, N);
    s.has_bias = m.bias != nullptr;
    s.bias = s.has_bias ? row4(m.bias, m.ld_bias, e, n, N) : f32x4{0, 0, 0, 0};
    return s;
}

__device__ __forceinline__ f32x4 scaled4(v4i d, const Scale4& s, float xs, bool has_xs) {
    f32x4 z = s.alpha * __builtin_convertvector(d, f32x4);
    if (has_xs) z = z * xs;
    if (s.has_bias) z = z + s.bias;
    return z;
}

template <typename E>
__device__ __forceinline__ void finish4(const ExpertArgs& a, int p, int n, f32x4 v) {
    typedef E e4 __attribute__((ext_vector_type(4)));
    if (a.r) {
        const E* r = (const E*)a.r + (int64_t)p * a.ldr + n;
        if (together(r, n, a.N)) v = v + __builtin_convertvector(*(const e4*)r, f32x4);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N) v[i] += (float)r[i];
    }
    E* y = (E*)a.y + (int64_t)p * a.ldy + n;
    if (together(y, n, a.N)) {
        *(e4*)y = __builtin_convertvector(v, e4);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < a.N) y[i] = (E)v[i];
    }
}

// Columns n .. n+3 of position p, whose row has the scale xs, from the sums.
template <bool GATED>
__device__ __forceinline__ void finish(const ExpertArgs& a, int p, float xs, int n, v4i d, v4i du, const Scale4& s, const Scale4& su) {
    const bool has_xs = a.xscale != nullptr;
    f32x4 z = scaled4(d, s, xs, has_xs);
    if (a.act != ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = activate(z[i], a.act);
    }
    if (GATED) z = z * scaled4(du, su, xs, has_xs);
    if (a.y_type == T_F32) finish4<float>(a, p, n, z);
    else if (a.y_type == T_BF16) finish4<__bf16>(a, p, n, z);
    else finish4<_Float16>(a, p, n, z);
}

bool expert_rows_fits(const ExpertArgs& a, bool ternary);
hipError_t launch_expert_rows(const ExpertArgs& a, bool ternary, hipStream_t s);
bool expert_tile_takes(const ExpertArgs& a);
hipError_t launch_expert_tile(const ExpertArgs& a, bool ternary, hipStream_t s);

}  // namespace bnn
