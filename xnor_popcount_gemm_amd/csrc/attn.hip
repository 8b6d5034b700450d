// Attention of a step's new tokens (a tree of drafts, a causal run, or one
// token) over the cache.
//
//     s_j = scale <q, k_j> ;  out = sum_j exp(s_j - lse) v_j ;  lse = ln sum_j exp(s_j)
//
// One wave per (row, query head).  A step takes 64 slots: each lane computes
// one slot's product with q (from LDS), the wave updates its running maximum
// and sum, then the lanes share out the head's dimensions and add the 64
// weighted rows of V.
#include <math.h>

#include "bnn_device.hpp"
#include "kv_launch.hpp"

namespace bnn {
namespace {

template <typename T, typename O, int D>
__global__ __launch_bounds__(64) void k_tree_attention(KvCache c, KvBatch b, AttnArgs a) {
    __shared__ float qs[D];
    const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
    const int seq = row_sequence(b, row, lane);
    if (seq < 0) return;
    const Seq sq = sequence(c, b, seq);
    const int node = row - sq.row0;
    if (node >= b.max_nodes) return;
    const typename T::elem* q = (const typename T::elem*)(a.q + row * a.q_row + h * a.q_head);
    for (int d = lane; d < D; d += 64) qs[d] = (float)q[d];
    __syncthreads();
    const int kh = h / a.group;
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int s0 = 0; s0 < sq.total; s0 += 64) {
        const int slot = s0 + lane;
        bool sees = slot < sq.ctx;
        if (!sees && slot < sq.total) {
            const int j = slot - sq.ctx;
            sees = a.mask ? packed_bit(a.mask + row * a.ld_mask, a.ld_mask, j) : j <= node;
        }
        int64_t vo = -1;
        float x = -INFINITY;
        if (sees) {
            uint32_t place;
            const int32_t pg = slot_page(c, seq, slot, place);
            float dot = 0.f;
            if (pg >= 0) {
                vo = pg * c.v_page + place * c.v_slot + kh * c.v_head;
                const typename T::vec8* k = (const typename T::vec8*)(c.K + pg * c.k_page + place * c.k_slot + kh * c.k_head);
                for (int i = 0; i < D / 8; ++i) {
                    const typename T::vec8 v = k[i];
#pragma unroll
                    for (int j = 0; j < 8; ++j) dot = fmaf((float)v[j], qs[8 * i + j], dot);
                }
            }
            x = dot * a.scale;
        }
        float mx = x;
        for (int t = 32; t; t >>= 1) mx = fmaxf(mx, __shfl_xor(mx, t, 64));
        const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
        const float p = sees ? expf(x - ms) : 0.f, al = expf(m - ms);
        float ps = p;
        for (int t = 32; t; t >>= 1) ps += __shfl_xor(ps, t, 64);
        l = l * al + ps;
        m = mn;
#pragma unroll
        for (int i = 0; i < D / 64 + (D % 64 != 0); ++i) o[i] *= al;
        const uint64_t seen = __ballot(sees);
        for (uint64_t left = seen; left; left &= left - 1) {
            const int j = __ffsll((unsigned long long)left) - 1;
            const float pj = __shfl(p, j, 64);
            const int64_t vj = __shfl(vo, j, 64);
            if (vj < 0) continue;
            const typename T::elem* v = (const typename T::elem*)(c.V + vj);
#pragma unroll
            for (int i = 0; i < D / 64 + (D % 64 != 0); ++i)
                if (lane + 64 * i < D) o[i] = fmaf(pj, (float)v[lane + 64 * i], o[i]);
        }
    }
    O* out = (O*)(a.out + row * a.o_row + h * a.o_head);
#pragma unroll
    for (int i = 0; i < D / 64 + (D % 64 != 0); ++i)
        if (lane + 64 * i < D) out[lane + 64 * i] = (O)(l == 0.f ? 0.f : o[i] / l);
    if (a.lse && lane == 0) a.lse[row * a.ld_lse + h] = m + logf(l);
}

template <typename T, typename O>
void launch_dim(const KvCache& c, const KvBatch& b, const AttnArgs& a, hipStream_t s) {
    const dim3 grid(b.rows, a.heads);
    if (c.dim == 64) hipLaunchKernelGGL((k_tree_attention<T, O, 64>), grid, dim3(64), 0, s, c, b, a);
    else if (c.dim == 96) hipLaunchKernelGGL((k_tree_attention<T, O, 96>), grid, dim3(64), 0, s, c, b, a);
    else if (c.dim == 128) hipLaunchKernelGGL((k_tree_attention<T, O, 128>), grid, dim3(64), 0, s, c, b, a);
    else hipLaunchKernelGGL((k_tree_attention<T, O, 256>), grid, dim3(64), 0, s, c, b, a);
}

}  // namespace

int64_t tree_attention_work(int32_t, int32_t, const KvBatch&, int32_t) { return 0; }

hipError_t launch_tree_attention(const KvCache& c, const KvBatch& b, const AttnArgs& a, int32_t dtype, int32_t out_dtype,
                                 hipStream_t s) {
    if (dtype == KV_BF16) {
        if (out_dtype == KV_F32) launch_dim<Bf16, float>(c, b, a, s);
        else launch_dim<Bf16, __bf16>(c, b, a, s);
    } else {
        if (out_dtype == KV_F32) launch_dim<F16, float>(c, b, a, s);
        else launch_dim<F16, _Float16>(c, b, a, s);
    }
    return hipGetLastError();
}

}  // namespace bnn
