// What lies between two linear layers of a decoder block, in one pass over
// the rows: experts' outputs joined, norm after the block, gate, residual,
// norm before the next block, INT8 quantization.
//
//     b = sum_j w_j B[place_j];  s = xs x + bs gate . post(b);  y = pre(s);
//     q = rint(fl32(y) * fl32(127 * fl32(1 / max|y|)))
//
// Bound by memory traffic: each value is read once, held in registers through
// its reductions, and written once: an RMS norm with codes has two (squares,
// largest value), layer norms on both sides with planes six (two a norm, largest
// value, sum of the codes).  All arithmetic up to fl32(y)
// is in 64 bits, so codes and scales do not depend on the order of a sum; that
// costs about 10 of the 25 operations of a value.  8192 rows of 4096, fp32
// stream + two experts' rows -> stream, output, codes: 124 us, 5.15 TB/s, what a plain
// copy reaches; 16384 rows of 11008 bfloat16 -> codes, 3 bytes a value: 153 us,
// 3.5 TB/s, where the operations bound it; one row: 6.7 us, its three reductions.
// Not near a copy: rows of 8193 to 12288 values held in 64 bits, which spill 58
// registers (16384 x 11008 with a norm of the branch: 701 us, 1.8 TB/s), and
// operands that are not 4-aligned, value by value (8192 x 4097: 151 us, 48 for
// 4096).
//
// A row belongs to T threads (a wave, or up to 16 waves of a workgroup),
// thread t holds the 4-value groups t, t + T, ... of it.  Rows are read and
// written through buffer descriptors of their own length, which stand in for
// the tests of the row's end: with those, every load had a branch, and waited.
#include "bnn_device.hpp"
#include "ffn.hpp"

namespace bnn {
namespace {

// A row of `count` values of a type: loads past its end give zeros and stores
// there are dropped, without a branch (VEC: 4 values at a time, count a
// multiple of 4; otherwise one by one).
template <bool VEC>
struct Row {
    __amdgpu_buffer_rsrc_t r;

    __device__ __forceinline__ Row(const void* base, int64_t first, int count, int bytes) {   // the same in all lanes of a wave
        const char* p = (const char*)base + first * bytes;
        const uint64_t u = (uint64_t)__builtin_amdgcn_readfirstlane((int)((uint64_t)p >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint64_t)p);
        r = __builtin_amdgcn_make_buffer_rsrc((void*)u, (short)0, base ? count * bytes : 0, 0x00020000);
    }

    // 4 values from e0 on as they are stored: 16 or 8 bytes.
    __device__ __forceinline__ u32x4 load(int e0, int type) const {
        u32x4 v = {0, 0, 0, 0};
        if (type == T_F32) {
            if (VEC) return __builtin_amdgcn_raw_buffer_load_b128(r, 4 * e0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b32(r, 4 * (e0 + i), 0, 0);
        } else if (VEC) {
            const u32x2 h = __builtin_amdgcn_raw_buffer_load_b64(r, 2 * e0, 0, 0);
            v[0] = h[0]; v[1] = h[1];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i >> 1] |= (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, 2 * (e0 + i), 0, 0) << (16 * (i & 1));
        }
        return v;
    }

    __device__ __forceinline__ void store(int e0, int type, f32x4 v) const {
        if (type == T_F32) {
            if (VEC) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, 4 * e0, 0, 0);
            else
#pragma unroll
                for (int i = 0; i < 4; ++i) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[i]), r, 4 * (e0 + i), 0, 0);
        } else {
            const u32x2 h = type == T_BF16 ? __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4))
                                           : __builtin_bit_cast(u32x2, __builtin_convertvector(v, f16x4));
            if (VEC) __builtin_amdgcn_raw_buffer_store_b64(h, r, 2 * e0, 0, 0);
            else
#pragma unroll
                for (int i = 0; i < 4; ++i) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(h[i >> 1] >> (16 * (i & 1))), r, 2 * (e0 + i), 0, 0);
        }
    }

    __device__ __forceinline__ void store_bytes(int e0, uint32_t v) const {
        if (VEC) __builtin_amdgcn_raw_buffer_store_b32(v, r, e0, 0, 0);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i) __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(v >> (8 * i)), r, e0 + i, 0, 0);
    }
};

__device__ __forceinline__ f32x4 values(u32x4 v, int type) {
    if (type == T_F32) return __builtin_bit_cast(f32x4, v);
    const u32x2 h = {v[0], v[1]};
    return type == T_BF16 ? __builtin_convertvector(__builtin_bit_cast(bf16x4, h), f32x4) : __builtin_convertvector(__builtin_bit_cast(f16x4, h), f32x4);
}

// A thread's share of a row, the type chosen once.
template <int NI, int T, bool VEC>
__device__ __forceinline__ void load_row(u32x4 (&v)[NI], const Row<VEC>& row, int t, int type) {
    if (type == T_F32) {
#pragma unroll
        for (int i = 0; i < NI; ++i) v[i] = row.load(4 * (t + i * T), T_F32);
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) v[i] = row.load(4 * (t + i * T), T_BF16);
    }
}

template <int NI>
__device__ __forceinline__ void to_values(f32x4 (&x)[NI], const u32x4 (&v)[NI], int type) {
    if (type == T_F32) {
#pragma unroll
        for (int i = 0; i < NI; ++i) x[i] = values(v[i], T_F32);
    } else if (type == T_BF16) {
#pragma unroll
        for (int i = 0; i < NI; ++i) x[i] = values(v[i], T_BF16);
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) x[i] = values(v[i], T_F16);
    }
}

template <int NI, int T, bool VEC>
__device__ __forceinline__ void store_row(const f32x4 (&v)[NI], const Row<VEC>& row, int t, int type) {
    if (type == T_F32) {
#pragma unroll
        for (int i = 0; i < NI; ++i) row.store(4 * (t + i * T), T_F32, v[i]);
    } else if (type == T_BF16) {
#pragma unroll
        for (int i = 0; i < NI; ++i) row.store(4 * (t + i * T), T_BF16, v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) row.store(4 * (t + i * T), T_F16, v[i]);
    }
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

// Values are widened to 64 bits again where they are used again: held wide over
// a row sum they would take twice the registers, and registers are what limits
// the rows in flight.
template <int NI, typename H>
__device__ __forceinline__ void afresh(H (&v)[NI][4]) {
    if (sizeof(H) == 4)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) asm volatile("" : "+v"(v[i][c]));
}

// What the norm of factor * v takes off v and multiplies it with.
struct Norm {
    double mean, inv;
};

template <int NI, int T, typename H>
__device__ __forceinline__ Norm norm_of(const H (&v)[NI][4], int kind, double factor, float eps, int t, int D, double (*red)[T / 64], int& turn) {
    Norm n = {0.0, factor};
    double s = 0;
    if (kind == NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) s += v[i][c];      // zeros past the row's end
        n.mean = row_sum<T>(s, red, turn) / D;
        s = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const double d = 4 * (t + i * T) + c < D ? v[i][c] - n.mean : 0.0;
                s = fma(d, d, s);
            }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
#pragma unroll
            for (int c = 0; c < 4; ++c) s = fma((double)v[i][c], (double)v[i][c], s);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    n.inv = factor / sqrt(factor * factor * (row_sum<T>(s, red, turn) / D) + eps);
    return n;
}

// out = the norm of factor * v, with w and b; 1 and 0 without.  Values past the row's end get a weight of 0.
template <int NI, int T, bool VEC, typename H, typename O>
__device__ __forceinline__ void normed(O& out, H (&v)[NI][4], int kind, double factor, const float* w, const float* b, float eps, int t, int D, const Row<VEC>& wr,
                                       const Row<VEC>& br, double (*red)[T / 64], int& turn) {
    u32x4 ww[NI];
    if (w) load_row<NI, T, VEC>(ww, wr, t, T_F32);
    else
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) ww[i][c] = 4 * (t + i * T) + c < D ? 0x3F800000u : 0u;
    const Norm n = norm_of<NI, T>(v, kind, factor, eps, t, D, red, turn);
    afresh(v);
    if (b) {
        u32x4 bb[NI];
        load_row<NI, T, VEC>(bb, br, t, T_F32);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                out[i][c] = (v[i][c] - n.mean) * n.inv * (double)__uint_as_float(ww[i][c]) + (double)__uint_as_float(bb[i][c]);
    } else if (kind == NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) out[i][c] = (v[i][c] - n.mean) * n.inv * (double)__uint_as_float(ww[i][c]);
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {   // a group at a time, for the registers' sake
#pragma unroll
            for (int c = 0; c < 4; ++c) out[i][c] = v[i][c] * n.inv * (double)__uint_as_float(ww[i][c]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// rint(x inv) within -127 .. 127; 0 where that is NaN (the conversion gives 0 for NaN and the ends of the range for
// what passes them).
__device__ __forceinline__ int code_of(float x, float inv) {
    int q;
    asm("v_cvt_i32_f32 %0, %1" : "=v"(q) : "v"(rintf(x * inv)));
    return min(max(q, -127), 127);
}

// T threads a row, NI groups of 4 values a thread; 256 / T rows a workgroup below 256 threads.  H: what the row is
// held in, float where that loses nothing.  Values past the row's end are zeros or NaN (a norm of a row that is not
// finite): neither counts in a sum that is, nor in the largest value or a code.
template <int T, int NI, typename H, bool VEC>
__global__ __launch_bounds__(T < 256 ? 256 : T, NI <= 2 ? 6 : NI <= 4 ? 4 : 3) void k_block_norm(NormArgs a) {
    __shared__ double red[2][T < 256 ? 1 : T / 64];
    static_assert(T == 64 || T >= 256, "a row has one wave or a whole workgroup");
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    const int64_t m = (int64_t)wide_index(blockIdx.y) * ROWS + __builtin_amdgcn_readfirstlane(threadIdx.x / T);
    const int t = threadIdx.x % T, D = a.D;
    int64_t rows = a.M;
    if (a.used) rows = a.used[0] < rows ? a.used[0] : rows;
    if (m >= rows) return;   // a whole wave, or the whole workgroup where it shares the row
    int turn = 0;
    double (*scratch)[T / 64] = (double (*)[T / 64])red;
    typedef Row<VEC> R;

    u32x4 xr[NI], br[NI];
    if (a.x) load_row<NI, T, VEC>(xr, R(a.x, m * a.ldx, D, type_bytes(a.x_type)), t, a.x_type);
    if (a.b && !a.place) load_row<NI, T, VEC>(br, R(a.b, m * a.ldb, D, type_bytes(a.b_type)), t, a.b_type);
    f32x4 x[NI];
    H v[NI][4];
    if (a.b) {
        if (sizeof(H) == 4 || !a.place) {   // a row held in fp32 comes from no sum, norm or gate
            to_values(x, br, a.b_type);
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) v[i][c] = x[i][c];
        } else {
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) v[i][c] = 0;
            for (int j = 0; j < a.parts; ++j) {
                const int64_t from = a.place[m * a.parts + j];
                if ((uint64_t)from >= (uint64_t)a.b_rows) continue;
                const double w = a.weight ? a.weight[m * a.parts + j] : 1.0;
                load_row<NI, T, VEC>(br, R(a.b, from * a.ldb, D, type_bytes(a.b_type)), t, a.b_type);
                to_values(x, br, a.b_type);
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[i][c] = (H)fma(w, (double)x[i][c], (double)v[i][c]);
            }
        }
        if (sizeof(H) == 8 && a.post != NORM_NONE)
            normed<NI, T>(v, v, a.post, 1.0, a.post_w, a.post_b, a.eps, t, D, R(a.post_w, 0, D, 4), R(a.post_b, 0, D, 4), scratch, turn);
        if (sizeof(H) == 8 && a.gate) {
            u32x4 g[NI];
            load_row<NI, T, VEC>(g, R(a.gate, m * a.ld_gate, D, 4), t, T_F32);
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) v[i][c] *= (H)values(g[i], T_F32)[c];
        }
    }
    if (a.x) to_values(x, xr, a.x_type);
    const double bs = a.b_scale, xs = a.x_scale;
    double factor = 1.0;   // the stream is factor * v
    if (sizeof(H) == 4 && !a.xo) {
        // one input as it is, its factor left to the norm
        factor = a.x ? xs : bs;
        if (a.x) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) v[i][c] = x[i][c];
        }
    } else if (sizeof(H) == 4 && a.b && a.x && bs == 1.0 && xs == 1.0) {
        // a sum of two fp32 numbers rounded once (through 64 bits it is the same: 53 >= 2 * 24 + 2), without conversions to
        // 64 bits, which take four times as long as the operations
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] = (H)((float)x[i][c] + (float)v[i][c]);
    } else if (a.b && a.x) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] = (H)fma(xs, (double)x[i][c], v[i][c] * bs);
            __builtin_amdgcn_sched_barrier(0);
        }
    } else if (a.b) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] = (H)(v[i][c] * bs);
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] = (H)(xs * (double)x[i][c]);
    }
    if (a.xo) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) x[i][c] = (float)v[i][c];
        if (a.x_type == T_BF16) {
#pragma unroll
            for (int i = 0; i < NI; ++i) x[i] = __builtin_convertvector(__builtin_convertvector(x[i], bf16x4), f32x4);
        } else if (a.x_type == T_F16) {
#pragma unroll
            for (int i = 0; i < NI; ++i) x[i] = __builtin_convertvector(__builtin_convertvector(x[i], f16x4), f32x4);
        }
        store_row<NI, T, VEC>(x, R(a.xo, m * a.ldxo, D, type_bytes(a.x_type)), t, a.x_type);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] = x[i][c];
    }
    if (!a.y && !a.xscale) return;
    if (a.pre == NORM_NONE) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) x[i][c] = (float)(v[i][c] * factor);
    } else {
        normed<NI, T>(x, v, a.pre, factor, a.pre_w, a.pre_b, a.eps, t, D, R(a.pre_w, 0, D, 4), R(a.pre_b, 0, D, 4), scratch, turn);
    }
    if (a.y) store_row<NI, T, VEC>(x, R(a.y, m * a.ldy, D, type_bytes(a.y_type)), t, a.y_type);
    if (!a.xscale) return;

    // INT8 rows
    float most = 0.f;   // the larger of a value and NaN is the value
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) most = __builtin_fmaxf(most, __builtin_fabsf(x[i][c]));
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) most = fmaxf(most, __shfl_xor(most, s, 64));
    if (T > 64) {
        float* red_f = (float*)&scratch[turn][0];
        if ((threadIdx.x & 63) == 0) red_f[threadIdx.x >> 6] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < T / 64; ++w) most = fmaxf(most, red_f[w]);
        turn ^= 1;
    }
    const float inv = most > 0.f ? 1.f / most * 127.f : 0.f;   // a reciprocal and a product, each rounded
    if (t == 0) a.xscale[m] = most / 127.f;
    uint32_t word[NI];   // 4 codes each; 0 past the row's end
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        int q[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) q[c] = code_of(x[i][c], inv);
        word[i] = __builtin_amdgcn_perm((uint32_t)q[1], (uint32_t)q[0], 0x0C0C0400u) | __builtin_amdgcn_perm((uint32_t)q[3], (uint32_t)q[2], 0x04000C0Cu);
    }
    if (a.Xq) {
        const R qr(a.Xq, m * a.ldXq, D, 1);
#pragma unroll
        for (int i = 0; i < NI; ++i) qr.store_bytes(4 * (t + i * T), word[i]);
    }
    if (a.Xb) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (128 * ((t + i * T) / 32) >= D) continue;   // whole groups of 32 lanes, 4 words: all of them are written, zeros included
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                // bit p of the 4 bytes (no carries: the partial products are apart), then the 8 lanes of a word
                const uint32_t nib = (((word[i] >> p) & 0x01010101u) * 0x01020408u) >> 24;
                const uint32_t w = or_reduce8_to_last(nib << (4 * (t & 7)));
                const int at = (t + i * T) >> 3;
                if ((t & 7) == 7 && at < a.ldXb) a.Xb[(m * 8 + p) * a.ldXb + at] = w;
            }
        }
        // words past those
        const int done = (D + 127) / 128 * 4;
        for (int64_t i = t; i < 8 * (a.ldXb - done); i += T) a.Xb[(m * 8 + i / (a.ldXb - done)) * a.ldXb + done + i % (a.ldXb - done)] = 0u;
    }
    if (a.xsum) {
        int sum = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) sum = __builtin_amdgcn_sdot4((int)word[i], 0x01010101, sum, false);
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

// Whether what is held of a row are fp32 numbers: one input as it is, or the stream rounded to x's type.
bool narrow(const NormArgs& a) {
    if (a.place || a.post != NORM_NONE || a.gate) return false;
    return a.xo || !a.b || !a.x;
}

// Whether every operand can be read or written 4 values at a time.
bool by_four(const NormArgs& a) {
    const auto has = [&](const void* p, uint32_t bit) { return !p || (a.vec & bit); };
    return a.D % 4 == 0 && has(a.x, V_X) && has(a.b, V_B) && has(a.gate, V_GATE) && has(a.xo, V_XO) && has(a.y, V_Y) && has(a.Xq, V_Q) &&
           has(a.post_w, V_POST_W) && has(a.post_b, V_POST_B) && has(a.pre_w, V_PRE_W) && has(a.pre_b, V_PRE_B);
}

template <int T, int NI>
void go(const NormArgs& a, hipStream_t s) {
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    const int64_t groups = (a.M + ROWS - 1) / ROWS;
    const dim3 grid(wide(groups), parts(groups)), block(T < 256 ? 256 : T);
    if (!by_four(a))    hipLaunchKernelGGL((k_block_norm<T, NI, double, false>), grid, block, 0, s, a);
    else if (narrow(a)) hipLaunchKernelGGL((k_block_norm<T, NI, float, true>), grid, block, 0, s, a);
    else                hipLaunchKernelGGL((k_block_norm<T, NI, double, true>), grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
    const int groups = (a.D + 3) / 4;
    // few threads a row, so that many rows are in flight (8192 rows of 4096: 79 us with 256 threads, 84 with 512,
    // 184 with 1024), but registers for the row (16384 of 11008: 183 us with 512 threads, 271 with 768, at that stage)
    if (groups <= 64) go<64, 1>(a, s);
    else if (groups <= 128) go<64, 2>(a, s);
    else if (groups <= 256) go<256, 1>(a, s);
    else if (groups <= 512) go<256, 2>(a, s);
    else if (groups <= 1024) go<256, 4>(a, s);
    else if (groups <= 2048) go<512, 4>(a, s);
    else if (groups <= 6 * 512) go<512, 6>(a, s);
    else go<1024, 4>(a, s);
    return hipGetLastError();
}

}  // namespace bnn
