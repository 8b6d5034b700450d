// Host-side launchers of the feed-forward kernels (internal to libbnn).
// ffn_api.hip validates every argument before calling these.
#pragma once

#include "kv.hpp"

namespace bnn {

enum : int32_t { T_BF16 = 1, T_F16 = 2, T_F32 = 3 };
__host__ __device__ inline int type_bytes(int32_t t) { return t == T_F32 ? 4 : 2; }

enum : int32_t { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };

// Strides in elements.
struct NormArgs {
    int64_t M;
    int32_t D;
    const int32_t* used;
    const char* x; int64_t ldx; int32_t x_type;
    const char* b; int64_t ldb; int32_t b_type; int32_t b_rows;
    const int32_t* place; const float* weight; int32_t parts;
    int32_t post; const float* post_w; const float* post_b;
    const float* gate; int64_t ld_gate;
    float x_scale, b_scale;
    int32_t pre; const float* pre_w; const float* pre_b;
    float eps;
    char* xo; int64_t ldxo;
    char* y; int64_t ldy; int32_t y_type;
    int8_t* Xq; int64_t ldXq;
    uint32_t* Xb; int64_t ldXb;
    int32_t* xsum; float* xscale;
    uint32_t vec;   // operands that are read or written 4 values at a time (V_*)
};
enum : uint32_t { V_X = 1, V_B = 2, V_GATE = 4, V_XO = 8, V_Y = 16, V_Q = 32, V_POST_W = 64, V_POST_B = 128, V_PRE_W = 256, V_PRE_B = 512 };

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s);

struct RouteArgs {
    const char* logits; int64_t ld; int32_t type;
    int32_t rows, experts, top;
    const int32_t* used;
    int32_t sigmoid;
    const float* bias;
    int32_t renorm; float scale;
    int32_t* expert; float* weight;
    int32_t* offsets; int32_t* order; int32_t* place;
    int32_t* work;
};

int64_t expert_route_work(int64_t rows, int64_t experts, int64_t top);   // bytes
hipError_t launch_expert_route(const RouteArgs& a, hipStream_t s);

// k of a lane's 16 bytes over its 64-k steps: 4 steps of ternary weights, 8 of binary ones.
__host__ __device__ constexpr int chunk_k(bool ternary) { return ternary ? 256 : 512; }

hipError_t launch_expert_pack(const uint32_t* Wp, const uint32_t* Zp, int64_t ldWp, int64_t w_expert, int64_t experts, int64_t N, int64_t K,
                              void* out, hipStream_t s);

struct ExpertMatrix {
    const uint4* W;
    const float* alpha; int64_t ld_alpha;
    const float* bias; int64_t ld_bias;
};

struct ExpertArgs {
    const int8_t* Xq; int64_t ldXq;
    const float* xscale;
    int32_t rows;
    const int32_t* order; FastDiv per_row;
    const int32_t* offsets;
    int32_t experts, positions, N, K;
    ExpertMatrix m, u;
    int32_t act;
    const char* r; int64_t ldr;
    char* y; int64_t ldy; int32_t y_type;
};

bool expert_linear_fits(const ExpertArgs& a, bool ternary);   // a launch takes the grid
hipError_t launch_expert_linear(const ExpertArgs& a, bool ternary, hipStream_t s);

}  // namespace bnn
