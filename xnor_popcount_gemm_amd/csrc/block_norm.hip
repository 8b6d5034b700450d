// What lies between two linear layers of a decoder block, in one pass over
// the rows: experts' outputs joined, norm after the block, gate, residual,
// norm before the next block, INT8 quantization.
//
//     b = sum_j w_j B[place_j];  s = xs x + bs gate . post(b);  y = pre(s);
//     q = rint(fl32(y) * fl32(127 * fl32(1 / max|y|)))
//
// Bound by memory traffic: each value is read once, held in registers through
// its three or four row sums, and written once.  All arithmetic up to fl32(y)
// is in 64 bits (a 64-bit operation takes a lane as long as a 32-bit one
// here, and there are about 20 a value against 5-17 bytes moved), so codes
// and scales do not depend on the order of a sum.
//
// A row belongs to T threads (a wave, or up to 16 waves of a workgroup),
// thread t holds the 4-value groups t, t + T, ... of it.
#include "bnn_device.hpp"
#include "ffn.hpp"

namespace bnn {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

// 4 values from element e0 on of a row of D, zeros past its end.
template <typename E, typename V4>
__device__ __forceinline__ f32x4 load4(const char* row, int e0, int D, bool vec) {
    const E* p = (const E*)row + e0;
    if (vec && e0 + 4 <= D) return __builtin_convertvector(*(const V4*)p, f32x4);
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (e0 + i < D) v[i] = (float)p[i];
    return v;
}

template <typename E, typename V4>
__device__ __forceinline__ void store4(char* row, int e0, int D, bool vec, f32x4 v) {
    E* p = (E*)row + e0;
    if (vec && e0 + 4 <= D) *(V4*)p = __builtin_convertvector(v, V4);
    else
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e0 + i < D) p[i] = (E)v[i];
}

// The same for a whole row share, the type chosen outside of the loop.
template <int NI, int T>
__device__ __forceinline__ void load_row(f32x4 (&v)[NI], const char* row, int t, int D, int type, bool vec) {
    if (type == T_F32) {
#pragma unroll
        for (int i = 0; i < NI; ++i) v[i] = load4<float, f32x4>(row, 4 * (t + i * T), D, vec);
    } else if (type == T_BF16) {
#pragma unroll
        for (int i = 0; i < NI; ++i) v[i] = load4<__bf16, bf16x4>(row, 4 * (t + i * T), D, vec);
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) v[i] = load4<_Float16, f16x4>(row, 4 * (t + i * T), D, vec);
    }
}

template <int NI, int T>
__device__ __forceinline__ void store_row(const f32x4 (&v)[NI], char* row, int t, int D, int type, bool vec) {
    if (type == T_F32) {
#pragma unroll
        for (int i = 0; i < NI; ++i) store4<float, f32x4>(row, 4 * (t + i * T), D, vec, v[i]);
    } else if (type == T_BF16) {
#pragma unroll
        for (int i = 0; i < NI; ++i) store4<__bf16, bf16x4>(row, 4 * (t + i * T), D, vec, v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) store4<_Float16, f16x4>(row, 4 * (t + i * T), D, vec, v[i]);
    }
}

__device__ __forceinline__ float rounded(float v, int type) {
    return type == T_F32 ? v : type == T_BF16 ? (float)(__bf16)v : (float)(_Float16)v;
}

// Sum of a value over the T threads of a row.  Every thread of the workgroup
// calls it the same number of times; `turn` alternates the two scratch rows,
// so that one barrier a call is enough.
template <int T>
__device__ __forceinline__ double row_sum(double v, double (*red)[T / 64], int& turn) {
    v = wave_sum_f64(v);
    if (T == 64) return v;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[turn][wave] = v;
    __syncthreads();
    double s = 0;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) s += red[turn][w];
    turn ^= 1;
    return s;
}

template <int NI, int T>
__device__ __forceinline__ void norm_row(double (&v)[NI][4], int kind, const float* w, const float* b, bool vw, bool vb, float eps, int t, int D,
                                         double (*red)[T / 64], int& turn) {
    if (kind == NORM_NONE) return;
    if (kind == NORM_LAYER) {
        double s = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) s += v[i][c];
        const double mean = row_sum<T>(s, red, turn) / D;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] = 4 * (t + i * T) + c < D ? v[i][c] - mean : 0.0;
    }
    double s = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) s = fma(v[i][c], v[i][c], s);
    const double inv = 1.0 / sqrt(row_sum<T>(s, red, turn) / D + eps);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e0 = 4 * (t + i * T);
        f32x4 ww = {1, 1, 1, 1}, bb = {0, 0, 0, 0};
        if (w) ww = load4<float, f32x4>((const char*)w, e0, D, vw);
        if (b) bb = load4<float, f32x4>((const char*)b, e0, D, vb);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[i][c] = v[i][c] * inv * ww[c] + bb[c];
    }
}

__device__ __forceinline__ int code_of(float x, float inv) {
    const float r = rintf(x * inv);
    return r != r ? 0 : r > 127.f ? 127 : r < -127.f ? -127 : (int)r;
}

// T threads a row, NI groups of 4 values a thread; 256 / T rows a workgroup below 256 threads.
template <int T, int NI>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_block_norm(NormArgs a) {
    __shared__ double red[2][T < 256 ? 1 : T / 64];
    static_assert(T == 64 || T >= 256, "a row has one wave or a whole workgroup");
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    const int64_t m = (int64_t)wide_index(blockIdx.y) * ROWS + threadIdx.x / T;
    const int t = threadIdx.x % T, D = a.D;
    int64_t rows = a.M;
    if (a.used) rows = a.used[0] < rows ? a.used[0] : rows;
    if (m >= rows) return;   // a whole wave, or the whole workgroup where it shares the row
    int turn = 0;
    double (*scratch)[T / 64] = (double (*)[T / 64])red;

    double v[NI][4];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[i][c] = 0.0;
    f32x4 x[NI];
    if (a.x) load_row<NI, T>(x, a.x + m * a.ldx * type_bytes(a.x_type), t, D, a.x_type, a.vec & V_X);
    if (a.b) {
        const int n = a.place ? a.parts : 1;
        for (int j = 0; j < n; ++j) {
            const int64_t from = a.place ? a.place[m * n + j] : m;
            if ((uint64_t)from >= (uint64_t)a.b_rows) continue;
            const double w = a.place && a.weight ? a.weight[m * n + j] : 1.0;
            f32x4 b[NI];
            load_row<NI, T>(b, a.b + from * a.ldb * type_bytes(a.b_type), t, D, a.b_type, a.vec & V_B);
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) v[i][c] = fma(w, (double)b[i][c], v[i][c]);
        }
        norm_row<NI, T>(v, a.post, a.post_w, a.post_b, a.vec & V_POST_W, a.vec & V_POST_B, a.eps, t, D, scratch, turn);
        if (a.gate) {
            const char* g = (const char*)(a.gate + m * a.ld_gate);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const f32x4 gg = load4<float, f32x4>(g, 4 * (t + i * T), D, a.vec & V_GATE);
#pragma unroll
                for (int c = 0; c < 4; ++c) v[i][c] *= gg[c];
            }
        }
        const double bs = a.b_scale;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] *= bs;
    }
    if (a.x) {
        const double xs = a.x_scale;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] = fma(xs, (double)x[i][c], v[i][c]);
    }
    if (a.xo) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] = x[i][c] = rounded((float)v[i][c], a.x_type);
        store_row<NI, T>(x, a.xo + m * a.ldxo * type_bytes(a.x_type), t, D, a.x_type, a.vec & V_XO);
    }
    if (!a.y && !a.xscale) return;
    norm_row<NI, T>(v, a.pre, a.pre_w, a.pre_b, a.vec & V_PRE_W, a.vec & V_PRE_B, a.eps, t, D, scratch, turn);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[i][c] = 4 * (t + i * T) + c < D ? (float)v[i][c] : 0.f;
    if (a.y) store_row<NI, T>(x, a.y + m * a.ldy * type_bytes(a.y_type), t, D, a.y_type, a.vec & V_Y);
    if (!a.xscale) return;

    // INT8 rows
    float most = 0.f;   // NaN compares false: skipped
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) most = fabsf(x[i][c]) > most ? fabsf(x[i][c]) : most;
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) {
        const float o = __shfl_xor(most, s, 64);
        most = o > most ? o : most;
    }
    if (T > 64) {
        float* red_f = (float*)&scratch[turn][0];
        if ((threadIdx.x & 63) == 0) red_f[threadIdx.x >> 6] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < T / 64; ++w) most = red_f[w] > most ? red_f[w] : most;
        turn ^= 1;
    }
    const float inv = most > 0.f ? 1.f / most * 127.f : 0.f;   // a reciprocal and a product, each rounded
    if (t == 0) a.xscale[m] = most / 127.f;
    int32_t sum = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e0 = 4 * (t + i * T);
        uint32_t word = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int q = code_of(x[i][c], inv);   // 0 past the row's end
            sum += q;
            word |= ((uint32_t)q & 0xFFu) << (8 * c);
        }
        if (a.Xq && e0 < D) {
            int8_t* o = a.Xq + m * a.ldXq + e0;
            if ((a.vec & V_Q) && e0 + 4 <= D) *(uint32_t*)o = word;
            else
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (e0 + c < D) o[c] = (int8_t)(word >> (8 * c));
        }
        if (a.Xb && 128 * ((t + i * T) / 32) < D) {   // whole groups of 32 lanes, 4 words: all of them are written, zeros included
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                // bit p of the 4 bytes (no carries: the partial products are apart), then the 8 lanes of a word
                const uint32_t nib = (((word >> p) & 0x01010101u) * 0x01020408u) >> 24;
                const uint32_t w = or_reduce8_to_last(nib << (4 * (t & 7)));
                const int at = (t + i * T) >> 3;
                if ((t & 7) == 7 && at < a.ldXb) a.Xb[(m * 8 + p) * a.ldXb + at] = w;
            }
        }
    }
    if (a.Xb) {   // words past those
        const int done = (D + 127) / 128 * 4;
        for (int64_t i = t; i < 8 * (a.ldXb - done); i += T) a.Xb[(m * 8 + i / (a.ldXb - done)) * a.ldXb + done + i % (a.ldXb - done)] = 0u;
    }
    if (a.xsum) {
#pragma unroll
        for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s, 64);
        if (T > 64) {
            int32_t* red_i = (int32_t*)&scratch[turn][0];
            if ((threadIdx.x & 63) == 0) red_i[threadIdx.x >> 6] = sum;
            __syncthreads();
            sum = 0;
#pragma unroll
            for (int w = 0; w < T / 64; ++w) sum += red_i[w];
        }
        if (t == 0) a.xsum[m] = sum;
    }
}

template <int T, int NI>
void go(const NormArgs& a, hipStream_t s) {
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    const int64_t groups = (a.M + ROWS - 1) / ROWS;
    hipLaunchKernelGGL((k_block_norm<T, NI>), dim3(wide(groups), parts(groups)), dim3(T < 256 ? 256 : T), 0, s, a);
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
    const int groups = (a.D + 3) / 4;
    if (groups <= 64) go<64, 1>(a, s);
    else if (groups <= 128) go<64, 2>(a, s);
    else if (groups <= 256) go<256, 1>(a, s);
    else if (groups <= 512) go<256, 2>(a, s);
    else if (groups <= 1024) go<256, 4>(a, s);
    else if (groups <= 2048) go<512, 4>(a, s);
    else go<1024, 4>(a, s);
    return hipGetLastError();
}

}  // namespace bnn
