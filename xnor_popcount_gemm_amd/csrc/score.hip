// The attention weight each cached slot received from the accepted new
// tokens, added to its running sum:
//
//     out_j = in_j + sum over accepted rows i that see j and the group's heads g
//             of exp(scale <q_ig, k_j> - lse_ig)
//
// One thread per slot of a (sequence, key head).
#include <math.h>

#include "bnn_device.hpp"
#include "kv_launch.hpp"

namespace bnn {
namespace {

template <typename T, int D>
__global__ __launch_bounds__(256) void k_cache_score_add(KvCache c, KvBatch b, ScoreArgs a) {
    const int seq = blockIdx.z, kh = blockIdx.y;
    const Seq sq = sequence(c, b, seq);
    const int nodes = sq.nodes < b.max_nodes ? sq.nodes : b.max_nodes;
    const int64_t head = ((int64_t)seq * c.kv_heads + kh) * a.ld_slots;
    if (a.out != a.in)   // slots that hold no token: copied
        for (int64_t i = sq.total + blockIdx.x * 256 + threadIdx.x; i < a.ld_slots; i += gridDim.x * 256)
            a.out[head + i] = a.in[head + i];
    for (int slot = blockIdx.x * 256 + threadIdx.x; slot < sq.total; slot += gridDim.x * 256) {
        uint32_t place;
        const int32_t pg = slot_page(c, seq, slot, place);
        const typename T::vec8* k = (const typename T::vec8*)(c.K + pg * c.k_page + place * c.k_slot + kh * c.k_head);
        float sum = 0.f;
        for (int i = 0; i < nodes; ++i) {
            if (a.accept && !packed_bit(a.accept + seq * a.ld_accept, a.ld_accept, i)) continue;
            const int64_t row = sq.row0 + i;
            const int j = slot - sq.ctx;
            const bool sees = j < 0 || (a.mask ? packed_bit(a.mask + row * a.ld_mask, a.ld_mask, j) : j <= i);
            if (!sees) continue;
            for (int g = 0; g < a.group; ++g) {
                const int h = kh * a.group + g;
                const typename T::vec8* q = (const typename T::vec8*)(a.q + row * a.q_row + h * a.q_head);
                float dot = 0.f;
                if (pg >= 0)
                    for (int e = 0; e < D / 8; ++e) {
                        const typename T::vec8 x = q[e], y = k[e];
#pragma unroll
                        for (int t = 0; t < 8; ++t) dot = fmaf((float)x[t], (float)y[t], dot);
                    }
                const float lse = a.lse[row * a.ld_lse + h];
                if (lse != -INFINITY) sum += expf(dot * a.scale - lse);
            }
        }
        a.out[head + slot] = a.in[head + slot] + sum;
    }
}

template <typename T>
void launch_dim(const KvCache& c, const KvBatch& b, const ScoreArgs& a, hipStream_t s) {
    const int64_t slots = (int64_t)b.max_ctx + b.max_nodes;
    const dim3 grid((unsigned)((slots + 255) / 256 > 0 ? (slots + 255) / 256 : 1), c.kv_heads, b.B);
    if (c.dim == 64) hipLaunchKernelGGL((k_cache_score_add<T, 64>), grid, dim3(256), 0, s, c, b, a);
    else if (c.dim == 96) hipLaunchKernelGGL((k_cache_score_add<T, 96>), grid, dim3(256), 0, s, c, b, a);
    else if (c.dim == 128) hipLaunchKernelGGL((k_cache_score_add<T, 128>), grid, dim3(256), 0, s, c, b, a);
    else hipLaunchKernelGGL((k_cache_score_add<T, 256>), grid, dim3(256), 0, s, c, b, a);
}

}  // namespace

hipError_t launch_cache_score_add(const KvCache& c, const KvBatch& b, const ScoreArgs& a, int32_t dtype, hipStream_t s) {
    if (dtype == KV_BF16) launch_dim<Bf16>(c, b, a, s);
    else launch_dim<F16>(c, b, a, s);
    return hipGetLastError();
}

}  // namespace bnn
