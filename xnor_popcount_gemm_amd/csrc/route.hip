// The router: every row's experts and their weights, and the (row, choice)
// pairs sorted by expert.
//
//     choose   top-k of the logits (or of score + bias, in 64 bits)
//     offsets  offsets[e] = pairs of the experts before e
//     order    the pairs of e at offsets[e] .., in their own order
//
// A wave owns a row: lane l holds the logits of experts l, l + 64, ..., and a
// round of the choice is a maximum over the wave in registers and a ballot for
// the lowest index.  The sort is a stable count: ranks within 64 neighbouring pairs by comparing the
// experts' bits across the wave (a ballot a bit), the waves of a tile and the
// tiles of a workgroup by counts in LDS, the workgroups by counts in the
// workspace.  No atomic decides a position, so the order is the same on every
// run.  A few rows are chosen and sorted by one workgroup in one launch.
//
// Bound by latency for few rows (1 x 8: 5.3 us, 200 x 64 with a bias: 7.4 and
// 5.4 in two kernels), by the rounds of the choice for many (16384 x 128, 8 of
// them: 18.6, and 8.3 for counts and places; 99 us in all with butterflies over
// 64-bit keys and a thread that walked the workgroups' counts one by one).
#include "bnn_device.hpp"
#include "ffn.hpp"

namespace bnn {
namespace {

constexpr int MAX_EXPERTS = 1024;
constexpr int THREADS = 1024, WAVES = THREADS / 64;
constexpr int MAX_PARTS = 256;       // workgroups that share the rows; with fewer a workgroup has at most 16
constexpr int ONE_PART_ROWS = 32;    // rows that one workgroup takes in one launch

// Keys in the order of an unsigned integer, in two words; 0 for what is never
// chosen (-inf, NaN), which no other value's first word is.
struct Key {
    uint32_t hi, lo;
};
__device__ __forceinline__ Key key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 as +0: they are equal
    return {x > -__builtin_inff() ? (u >> 31 ? ~u : u | 0x80000000u) : 0u, 0u};
}
__device__ __forceinline__ Key key_of(double x) {
    uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    u = x > -__builtin_inf() ? (u >> 63 ? ~u : u | 0x8000000000000000ull) : 0ull;
    return {(uint32_t)(u >> 32), (uint32_t)u};
}

// Over the wave, in registers (row shifts, then the rows' last lanes on to the next ones); the result is in lane 63.
template <typename Op>
__device__ __forceinline__ uint32_t wave_fold(uint32_t v, Op op) {   // 0 must change nothing
#define BNN_FOLD(ctrl, rows) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, false))
    BNN_FOLD(0x111, 0xF);
    BNN_FOLD(0x112, 0xF);
    BNN_FOLD(0x114, 0xF);
    BNN_FOLD(0x118, 0xF);
    BNN_FOLD(0x142, 0xA);
    BNN_FOLD(0x143, 0xC);
#undef BNN_FOLD
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    return wave_fold(v, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
}
__device__ __forceinline__ float wave_sum(float v) {
    return __uint_as_float(wave_fold(__float_as_uint(v), [](uint32_t x, uint32_t y) { return __float_as_uint(__uint_as_float(x) + __uint_as_float(y)); }));
}

__device__ __forceinline__ float logit_at(const char* row, int e, int type) {
    if (type == T_F32) return ((const float*)row)[e];
    return type == T_BF16 ? (float)((const __bf16*)row)[e] : (float)((const _Float16*)row)[e];
}

// The experts of one row, by one wave; each is also counted in `count` (LDS).
template <int PER>
__device__ void choose(const RouteArgs& a, int row, int lane, uint32_t* count) {
    const char* lr = a.logits + (int64_t)row * a.ld * type_bytes(a.type);
    float l[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < a.experts ? logit_at(lr, e, a.type) : -__builtin_inff();
        if (l[i] != l[i]) l[i] = -__builtin_inff();
    }
    Key key[PER], plain[PER];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        plain[i] = key_of(l[i]);
        top = plain[i].hi > top ? plain[i].hi : top;
    }
    top = wave_max(top);
    const float most = top == 0 ? 0.f : __uint_as_float(top >> 31 ? top & 0x7FFFFFFFu : ~top);   // the largest logit
    float total = 0.f;
    if (a.bias) {
        double s[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            s[i] = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - (double)most);
            sum += s[i];
        }
        if (!a.sigmoid) sum = wave_sum_f64(sum);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 64 * i;
            const double v = a.sigmoid || sum == 0.0 ? s[i] : s[i] / sum;
            key[i] = e < a.experts && l[i] > -__builtin_inff() ? key_of(v + (double)a.bias[e]) : Key{0, 0};
        }
        total = (float)sum;
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = plain[i];
        if (!a.sigmoid) {
#pragma unroll
            for (int i = 0; i < PER; ++i) total += expf(l[i] - most);
            total = wave_sum(total);
        }
    }
    int mine = -1;   // lane j keeps choice j
    for (int j = 0; j < a.top; ++j) {
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) hi = key[i].hi > hi ? key[i].hi : hi;
        hi = wave_max(hi);
        if (hi == 0) break;   // the same in all lanes
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < PER; ++i) lo = key[i].hi == hi && key[i].lo > lo ? key[i].lo : lo;
            lo = wave_max(lo);
        }
        int at = -1;   // the lowest index that has the largest key
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) {
            const uint64_t has = __ballot(key[i].hi == hi && key[i].lo == lo);
            at = has ? 64 * i + __ffsll((unsigned long long)has) - 1 : at;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (at == lane + 64 * i) key[i].hi = 0;
        if (lane == j) mine = at;
    }
    float w = 0.f;
    if (mine >= 0) {
        const float lg = logit_at(lr, mine, a.type);
        const float ex = expf(a.sigmoid ? -fabsf(lg) : lg - most);
        // a sigmoid by exp(-|l|): exp(-l) overflows at -88.7, where the score is still a number
        w = a.sigmoid ? (lg < 0.f ? ex : 1.f) / (1.f + ex) : ex / total;
        atomicAdd(&count[mine], 1u);
    }
    if (a.renorm) {
        const float sum = wave_sum(w);
        w = sum == 0.f ? 0.f : w / sum;
    }
    if (lane < a.top) {
        a.expert[(int64_t)row * a.top + lane] = mine;
        a.weight[(int64_t)row * a.top + lane] = w * a.scale;
    }
}

__device__ void choose_row(const RouteArgs& a, int row, int lane, uint32_t* count) {
    if (a.experts <= 64) choose<1>(a, row, lane, count);
    else if (a.experts <= 128) choose<2>(a, row, lane, count);
    else if (a.experts <= 256) choose<4>(a, row, lane, count);
    else choose<16>(a, row, lane, count);
}

__device__ __forceinline__ int used_rows(const RouteArgs& a) {
    if (!a.used) return a.rows;
    const int u = a.used[0];
    return u < 0 ? 0 : u < a.rows ? u : a.rows;
}

// The rows of part p of n.
__device__ __forceinline__ int first_row(int rows, int p, int n) { return (int)((int64_t)rows * p / n); }

// Exclusive prefix sums over the experts, thread e's value in `v` (0 past the
// experts); `red` holds a word per wave.
__device__ __forceinline__ uint32_t scan_experts(uint32_t v, uint32_t* red, uint32_t& all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(s, d, 64);
        if (lane >= d) s += o;
    }
    if (lane == 63) red[wave] = s;
    __syncthreads();
    uint32_t before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        if (w < wave) before += red[w];
        all += red[w];
    }
    __syncthreads();
    return before + s - v;
}

// Positions of the pairs of rows lo .. hi-1; base[e] (LDS) is the next
// position of expert e.  part: 16 counters of 16 bits for each expert.
__device__ void place_rows(const RouteArgs& a, int lo, int hi, uint32_t* base, uint16_t (*part)[MAX_EXPERTS]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t first = (int64_t)lo * a.top, last = (int64_t)hi * a.top;
    int bits = 0;
    while ((1 << bits) < a.experts) ++bits;
    for (int64_t p0 = first; p0 < last; p0 += THREADS) {
        for (int i = tid; i < WAVES * a.experts; i += THREADS) part[i / a.experts][i % a.experts] = 0;
        __syncthreads();
        const int64_t p = p0 + tid;
        const int e = p < last ? a.expert[p] : -1;
        uint64_t same = __ballot(e >= 0);
        for (int b = 0; b < bits; ++b) {
            const bool on = (e >> b) & 1;
            const uint64_t m = __ballot(on);
            same &= on ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (e >= 0 && rank == 0) part[wave][e] = (uint16_t)__popcll(same);
        __syncthreads();
        if (tid < a.experts) {   // where each wave's pairs of the expert begin; counts become starts, below 2^10
            uint32_t run = 0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const uint32_t n = part[w][tid];
                part[w][tid] = (uint16_t)run;
                run += n;
            }
            base[MAX_EXPERTS + tid] = run;
        }
        __syncthreads();
        if (e >= 0) {
            const uint32_t at = base[e] + part[wave][e] + rank;
            a.order[at] = (int32_t)p;
            a.place[p] = (int32_t)at;
        } else if (p < last) {
            a.place[p] = -1;
        }
        __syncthreads();
        if (tid < a.experts) base[tid] += base[MAX_EXPERTS + tid];
    }
}

// Choice and, with one workgroup, the order too; with more, each writes how
// many pairs of each expert its rows have.
__global__ __launch_bounds__(THREADS) void k_route(RouteArgs a) {
    __shared__ uint32_t base[2 * MAX_EXPERTS], red[WAVES];
    __shared__ uint16_t part[WAVES][MAX_EXPERTS];
    const int tid = threadIdx.x, rows = used_rows(a);
    const int lo = first_row(rows, blockIdx.x, gridDim.x), hi = first_row(rows, blockIdx.x + 1, gridDim.x);
    if (tid < a.experts) base[tid] = 0;
    __syncthreads();
    for (int r = lo + (tid >> 6); r < hi; r += WAVES) choose_row(a, r, tid & 63, base);
    __syncthreads();
    if (gridDim.x > 1) {
        if (tid < a.experts) a.work[(int64_t)blockIdx.x * a.experts + tid] = (int32_t)base[tid];
        return;
    }
    uint32_t all;
    const uint32_t at = scan_experts(tid < a.experts ? base[tid] : 0, red, all);
    if (tid < a.experts) {
        base[tid] = at;
        a.offsets[tid] = (int32_t)at;
        if (tid == a.experts - 1) a.offsets[a.experts] = (int32_t)all;
    }
    __syncthreads();
    place_rows(a, lo, hi, base, part);
}

__global__ __launch_bounds__(THREADS) void k_route_place(RouteArgs a) {
    __shared__ uint32_t base[2 * MAX_EXPERTS], red[WAVES];
    __shared__ uint16_t part[WAVES][MAX_EXPERTS];
    const int tid = threadIdx.x, rows = used_rows(a);
    // pairs of each expert in all workgroups and in those before this one: a slice of the workgroups to each group of
    // threads as long as the experts, 8 counts in flight
    __shared__ uint32_t sums[2][MAX_EXPERTS];
    if (tid < a.experts) sums[0][tid] = sums[1][tid] = 0;
    __syncthreads();
    const int slices = THREADS / a.experts, slice = tid / a.experts, e = tid - slice * a.experts;
    if (slice < slices) {
        uint32_t own = 0, ahead = 0;
        for (int g = slice; g < (int)gridDim.x; g += 8 * slices) {
            uint32_t n[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int h = g + u * slices;
                n[u] = h < (int)gridDim.x ? (uint32_t)a.work[(int64_t)h * a.experts + e] : 0u;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                own += n[u];
                if (g + u * slices < (int)blockIdx.x) ahead += n[u];
            }
        }
        atomicAdd(&sums[0][e], own);   // whole numbers: in any order the same
        atomicAdd(&sums[1][e], ahead);
    }
    __syncthreads();
    const uint32_t mine = tid < a.experts ? sums[0][tid] : 0, before = tid < a.experts ? sums[1][tid] : 0;
    uint32_t all;
    const uint32_t at = scan_experts(mine, red, all);
    if (tid < a.experts) {
        base[tid] = at + before;
        if (blockIdx.x == 0) {
            a.offsets[tid] = (int32_t)at;
            if (tid == a.experts - 1) a.offsets[a.experts] = (int32_t)all;
        }
    }
    __syncthreads();
    place_rows(a, first_row(rows, blockIdx.x, gridDim.x), first_row(rows, blockIdx.x + 1, gridDim.x), base, part);
}

int route_parts(int64_t rows) {
    if (rows <= ONE_PART_ROWS) return 1;
    const int64_t n = (rows + WAVES - 1) / WAVES;
    return (int)(n < MAX_PARTS ? n : MAX_PARTS);
}

}  // namespace

int64_t expert_route_work(int64_t rows, int64_t experts, int64_t) {
    const int n = route_parts(rows);
    return n > 1 ? (int64_t)n * experts * 4 : 0;
}

hipError_t launch_expert_route(const RouteArgs& a, hipStream_t s) {
    const int n = route_parts(a.rows);
    hipLaunchKernelGGL(k_route, dim3(n), dim3(THREADS), 0, s, a);
    if (n > 1) hipLaunchKernelGGL(k_route_place, dim3(n), dim3(THREADS), 0, s, a);
    return hipGetLastError();
}

}  // namespace bnn
