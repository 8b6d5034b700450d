// Layout of 1-bit and ternary matrices for the grouped products, once per
// model: the packed planes (rows of k, 32 to a word) become the fragments that
// the matrix cores take, 1 KiB to a wave's load.  See bnn_expert_pack in
// include/bnn.h for the layout; what it buys the products: a weight costs 3
// operations to 4 weights to expand (shift, mask, byte permute) instead of 7
// from the planes, one stream of whole 128-byte lines, and no row or k bounds.
// Bound by memory traffic, and run once.
#include "ffn.hpp"

namespace bnn {
namespace {

// A thread writes one lane's 16 bytes.
template <bool TERN>
__global__ __launch_bounds__(256) void k_expert_pack(const uint32_t* __restrict__ Wp, const uint32_t* __restrict__ Zp, int64_t ldWp, int64_t w_expert,
                                                     int64_t pieces, int N, int K, int frags, int chunks, uint4* __restrict__ out) {
    const int64_t at = ((int64_t)wide_index(blockIdx.y)) * 256 + threadIdx.x;
    if (at >= pieces) return;
    const int lane = (int)(at & 63), g = lane >> 4;
    int64_t rest = at >> 6;
    const int c = (int)(rest % chunks);
    rest /= chunks;
    const int f = (int)(rest % frags);
    const int64_t e = rest / frags;
    const int n = 16 * f + (lane & 15);
    uint32_t w[4] = {0, 0, 0, 0};
    if (n < N) {
        const uint32_t* sp = Wp + e * w_expert + n * ldWp;
        const uint32_t* zp = TERN ? Zp + e * w_expert + n * ldWp : nullptr;
#pragma unroll
        for (int s = 0; s < chunk_k(TERN) / 64; ++s) {
            const int k0 = chunk_k(TERN) * c + 64 * s + 16 * g;
            if (k0 >= K) continue;
            const uint32_t left = K - k0 >= 16 ? 0xFFFFu : (1u << (K - k0)) - 1u;
            const uint32_t sg = (sp[k0 >> 5] >> (k0 & 31)) & left;
            const uint32_t nz = TERN ? (zp[k0 >> 5] >> (k0 & 31)) & left : 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int d = i >> 2, j = i & 3;
                if (TERN) w[s] |= (((nz >> i) & 1u) | (((nz & sg) >> i) & 1u) << 1) << (8 * j + 2 * d);
                else w[s >> 1] |= ((sg >> i) & 1u) << (8 * j + 4 * (s & 1) + d);
            }
        }
    }
    out[at] = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace

hipError_t launch_expert_pack(const uint32_t* Wp, const uint32_t* Zp, int64_t ldWp, int64_t w_expert, int64_t experts, int64_t N, int64_t K, void* out,
                              hipStream_t s) {
    const int frags = (int)((N + 15) / 16), ck = chunk_k(Zp != nullptr), chunks = (int)((K + ck - 1) / ck);
    const int64_t pieces = experts * frags * chunks * 64, groups = (pieces + 255) / 256;
    const dim3 grid(wide(groups), parts(groups));
    if (Zp) hipLaunchKernelGGL((k_expert_pack<true>), grid, dim3(256), 0, s, Wp, Zp, ldWp, w_expert, pieces, (int)N, (int)K, frags, chunks, (uint4*)out);
    else    hipLaunchKernelGGL((k_expert_pack<false>), grid, dim3(256), 0, s, Wp, Zp, ldWp, w_expert, pieces, (int)N, (int)K, frags, chunks, (uint4*)out);
    return hipGetLastError();
}

}  // namespace bnn
