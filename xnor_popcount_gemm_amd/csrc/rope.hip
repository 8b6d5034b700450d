// Norm and rotation of queries and keys, and the append of keys and values to
// the cache, in one pass over the fused QKV rows.
//
//     y = x * rsqrt(mean(x^2) + eps) * w ;  (a, b) -> (a c - b s, b c + a s)
//
// Bound by memory traffic: each value is read once and written once (about 8
// operations a value).  A lane holds one unit of 8 values of a head in two
// pieces of 4: in the half layout 4 values and their partners rot/2 further,
// in the interleaved layout 8 neighbours.  Either way both members of a pair
// are in one lane, the unit needs the same 4 cosines and 4 sines, and no
// values cross lanes but the sum of squares (a butterfly over the head's
// lanes).  A workgroup owns one token: the lookup of its sequence and slot is
// done once, the cosines and sines stay in registers over its heads.  8190
// tokens of 48 heads of 128: 58 us, 5.2 TB/s, what a plain copy reaches; one
// token: 4.5 us, the latency of its dependent reads.
#include "bnn_device.hpp"
#include "kv_launch.hpp"

namespace bnn {
namespace {

template <typename S> struct Src;
template <> struct Src<float> {
    static __device__ __forceinline__ f32x4 load(const char* p) { return *(const f32x4*)p; }
};
template <> struct Src<Bf16> {
    static __device__ __forceinline__ f32x4 load(const char* p) { return __builtin_convertvector(*(const bf16x4*)p, f32x4); }
};
template <> struct Src<F16> {
    static __device__ __forceinline__ f32x4 load(const char* p) { return __builtin_convertvector(*(const f16x4*)p, f32x4); }
};

// LPR: lanes per head (a power of two >= dim / 8).
template <typename T, typename S, int LPR, bool INTER>
__global__ __launch_bounds__(256) void k_qk_norm_rope(KvCache c, KvBatch b, RopeArgs a) {
    constexpr int ESZ = sizeof(S) == 4 ? 4 : 2;
    constexpr int HEADS = 256 / LPR;   // heads in flight per workgroup
    const int row = wide_index(blockIdx.y), tid = threadIdx.x;
    const int seq = row_sequence(b, row, tid & 63);
    if (seq < 0 || row >= b.rows) return;
    const Seq sq = sequence(c, b, seq);
    const int64_t slot = (int64_t)sq.ctx + (row - sq.row0);
    const bool fits = slot < sq.total;
    uint32_t place = 0;
    const int32_t page = fits ? slot_page(c, seq, (uint32_t)slot, place) : -1;

    const int u = tid % LPR, dim = c.dim, rot = a.rot, half = rot >> 1;
    const bool live = u < dim / 8, turn = 8 * u < rot;
    int e0 = 8 * u, e1 = e0 + 4;
    if (!INTER && turn) { e0 = 4 * u; e1 = e0 + half; }
    const int32_t position = a.positions[row];
    f32x4 cs = {1, 1, 1, 1}, sn = {0, 0, 0, 0};
    if (turn) {
        if ((uint32_t)position < (uint32_t)a.max_pos) {
            const float* t = a.turns + (int64_t)position * rot;
            cs = *(const f32x4*)(t + 4 * u);
            sn = *(const f32x4*)(t + half + 4 * u);
        } else {
            cs = sn = f32x4{} + __builtin_nanf("");
        }
    }
    const int all = a.heads + 2 * c.kv_heads;
    for (int h = tid / LPR; h < all; h += HEADS) {
        const bool isq = h < a.heads, isk = !isq && h < a.heads + c.kv_heads;
        const int hh = isq ? h : isk ? h - a.heads : h - a.heads - c.kv_heads;
        const char* src = isq ? a.q + row * a.q_row + hh * a.q_head
                        : isk ? a.k + row * a.k_row + hh * a.k_head : a.v + row * a.v_row + hh * a.v_head;
        char* dst = isq ? a.qo + row * a.qo_row + hh * a.qo_head
                  : isk ? c.K + page * c.k_page + place * c.k_slot + hh * c.k_head
                        : c.V + page * c.v_page + place * c.v_slot + hh * c.v_head;
        f32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
        if (live) {
            x = Src<S>::load(src + e0 * ESZ);
            y = Src<S>::load(src + e1 * ESZ);
        }
        const float* w = isq ? a.qw : isk ? a.kw : nullptr;
        if (w) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
            for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor(ss, m, 64);
            const float inv = 1.0f / sqrtf(ss / dim + a.eps);
            if (live) {
                x = x * inv * *(const f32x4*)(w + e0);
                y = y * inv * *(const f32x4*)(w + e1);
            }
        }
        if (turn && (isq || isk)) {
            f32x4 p = x, q = y;
            if (INTER) {
                p = f32x4{x[0], x[2], y[0], y[2]};
                q = f32x4{x[1], x[3], y[1], y[3]};
            }
            const f32x4 r = p * cs - q * sn, t = q * cs + p * sn;
            x = INTER ? f32x4{r[0], t[0], r[1], t[1]} : r;
            y = INTER ? f32x4{r[2], t[2], r[3], t[3]} : t;
        }
        if (live && (isq || page >= 0)) {
            *(typename T::vec4*)(dst + 2 * e0) = __builtin_convertvector(x, typename T::vec4);
            *(typename T::vec4*)(dst + 2 * e1) = __builtin_convertvector(y, typename T::vec4);
        }
        if (isk && u == 0 && fits) {
            const int64_t at = ((int64_t)seq * c.kv_heads + hh) * a.ld_slots + slot;
            if (a.pos) a.pos[at] = position;
            if (a.score) a.score[at] = 0.f;
        }
    }
}

template <typename T, typename S, int LPR>
void launch_one(const KvCache& c, const KvBatch& b, const RopeArgs& a, bool inter, hipStream_t s) {
    const dim3 grid(wide(b.rows), parts(b.rows));
    if (inter) hipLaunchKernelGGL((k_qk_norm_rope<T, S, LPR, true>), grid, dim3(256), 0, s, c, b, a);
    else       hipLaunchKernelGGL((k_qk_norm_rope<T, S, LPR, false>), grid, dim3(256), 0, s, c, b, a);
}

template <typename T, typename S>
void launch_dim(const KvCache& c, const KvBatch& b, const RopeArgs& a, bool inter, hipStream_t s) {
    if (c.dim <= 64) launch_one<T, S, 8>(c, b, a, inter, s);
    else if (c.dim <= 128) launch_one<T, S, 16>(c, b, a, inter, s);
    else launch_one<T, S, 32>(c, b, a, inter, s);
}

}  // namespace

hipError_t launch_qk_norm_rope(const KvCache& c, const KvBatch& b, const RopeArgs& a, int32_t dtype, int32_t src_dtype,
                               bool inter, hipStream_t s) {
    if (dtype == KV_BF16) {
        if (src_dtype == KV_F32) launch_dim<Bf16, float>(c, b, a, inter, s);
        else launch_dim<Bf16, Bf16>(c, b, a, inter, s);
    } else {
        if (src_dtype == KV_F32) launch_dim<F16, float>(c, b, a, inter, s);
        else launch_dim<F16, F16>(c, b, a, inter, s);
    }
    return hipGetLastError();
}

}  // namespace bnn
