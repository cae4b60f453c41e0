// Routing of tokens to experts.  With x the router's logits of one token,
//     s_e = softmax(x)_e or 1 / (1 + exp(-x_e)),   c_e = s_e + b_e,
// the token's experts are the `top` largest c, in descending order and the lower
// index first among equals, out of the `top_groups` groups of E / groups
// neighbouring experts whose group_top (1 or 2) largest c sum highest.  Their
// weights are scale * s, or scale * s over the sum of the chosen s.
//
// Scores next to each other decide what is chosen, so c is compared in 64 bits;
// without a bias (and without sums of two scores) the logits themselves are
// compared, whose order is that of the scores.  The weights are formed in fp32
// from the logits of the chosen.  A logit (or c) of -inf or NaN is never chosen;
// of +inf the softmax is its limit.
//
// L lanes hold a token, V experts each, in the experts' order, so the lowest
// index among equals is that of the lowest lane.  Each of the `top` rounds takes
// the largest of the lanes' maxima (4 exchanges within 16 lanes) and only then
// does the lane that held it look for its next.  Four tokens to a wave (L = 16)
// take a quarter of the rounds' instructions; a wave to a token (L = 64) is
// quicker where there are few tokens.
#pragma once

#include "common.hpp"
#include "dense_gemm.h"
#include "ragged.hpp"

namespace dg {

constexpr int ROUTE_MAX_EXPERTS = 1024, ROUTE_MAX_TOP = 32;
constexpr int ROUTE_CHUNK = 64;    // tokens whose experts are counted together, at most
constexpr int ROUTE_SUPER = 256;   // chunks whose counts are added up for the others

struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    int32_t* offsets;    // the plan: all three, or none
    int32_t* order;
    int32_t* position;
    uint8_t* counts;     // chunks x count_ld: tokens of a chunk that chose an expert
    int32_t* supers;     // supers x experts: sums over ROUTE_SUPER chunks
    int64_t ld;
    int tokens, experts, top;
    int groups, group_size, lanes_per_group;  // lanes of a token that hold a group
    int top_groups, group_top;
    int sigmoid, renormalize;
    float scale;
    int chunk, chunks, count_ld;
};

template <typename K>
__device__ __forceinline__ K key_low();
template <>
__device__ __forceinline__ float key_low<float>() { return -__builtin_inff(); }
template <>
__device__ __forceinline__ double key_low<double>() { return -__builtin_inf(); }

// x of the lane that CTRL of the data-parallel primitives names.
template <int CTRL>
__device__ __forceinline__ float dpp(float x)
{
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double x)
{
    return __hiloint2double(__builtin_amdgcn_mov_dpp(__double2hiint(x), CTRL, 0xf, 0xf, true),
                            __builtin_amdgcn_mov_dpp(__double2loint(x), CTRL, 0xf, 0xf, true));
}

__device__ __forceinline__ float max_of(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double max_of(double a, double b) { return fmax(a, b); }

// op over the lane's L lanes, in every one of them (L = 16 or 64; the same tree
// of exchanges in each lane, so the same result).
template <int L, typename K, class F>
__device__ __forceinline__ K lanes_reduce(K x, F op)
{
    x = op(x, dpp<0xB1>(x));   // quad_perm 1, 0, 3, 2
    x = op(x, dpp<0x4E>(x));   // quad_perm 2, 3, 0, 1
    x = op(x, dpp<0x141>(x));  // row_half_mirror
    x = op(x, dpp<0x140>(x));  // row_mirror
    if constexpr (L == 64) {
        x = op(x, __shfl_xor(x, 16));
        x = op(x, __shfl_xor(x, 32));
    }
    return x;
}
template <int L, typename K>
__device__ __forceinline__ K lanes_max(K x)
{
    return lanes_reduce<L>(x, [](K a, K b) { return max_of(a, b); });
}
template <int L, typename K>
__device__ __forceinline__ K lanes_sum(K x)
{
    return lanes_reduce<L>(x, [](K a, K b) { return a + b; });
}

// Lowest of the lane's L lanes where `yes` (none: some lane beyond them).
template <int L>
__device__ __forceinline__ int first_lane(bool yes, int lane)
{
    const uint64_t m = __ballot(yes);
    if constexpr (L == 64) return m ? __builtin_ctzll(m) : 64;
    const uint32_t mine = (uint32_t)(m >> (lane & 48)) & 0xFFFFu;
    return (lane & 48) + (mine ? __builtin_ctz(mine) : 64);
}

// What a wave's lanes wrote to LDS is there for its other lanes.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// e^(x - m) with m >= x, 1 where both are infinite.
__device__ __forceinline__ float exp_below(float x, float m) { return x == m ? 1.0f : expf(x - m); }
__device__ __forceinline__ double exp_below(double x, double m) { return x == m ? 1.0 : exp(x - m); }

// A token's chosen logit as a score: softmax over all (e^(x - m) / sum), or with
// renormalised weights a number in proportion to it, of which the largest is
// about 1 (m the largest chosen logit): e^(x - m); e^(x - m) / (1 + e^x) for the
// sigmoid of logits below zero, whose own value may be too small for fp32.
__device__ __forceinline__ float chosen_score(const RouteArgs& p, float x, float m)
{
    if (!p.sigmoid) return exp_below(x, m);
    if (!p.renormalize || x > 0.0f) return 1.0f / (1.0f + expf(-x));
    return expf(x - fminf(m, 0.0f)) / (1.0f + expf(x));
}

// Tokens t0 .. of the workgroup's pass, one per L lanes: chooses their experts
// into picked[token of the pass][j] and writes ids and weights.
template <typename X, int L, int V, typename K>
__device__ __forceinline__ void route_token(const RouteArgs& p, int t, bool live,
                                            int32_t* picked)
{
    const int lane = threadIdx.x & 63, sub = lane & (L - 1);
    const X* row = static_cast<const X*>(p.logits) + (int64_t)(live ? t : 0) * p.ld;
    // the lane's experts
    const int group = sub / p.lanes_per_group, part = sub % p.lanes_per_group;
    const int e0 = group * p.group_size + part * V;
    int count = group < p.groups && live ? p.group_size - part * V : 0;
    count = count < 0 ? 0 : count > V ? V : count;
    float x[V];
    if (count == V && V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            if constexpr (sizeof(X) == 4) {
                const f32x4 v = *reinterpret_cast<const f32x4_a4*>(row + e0 + i);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (i + q < V) x[i + q] = v[q];
            } else {
                const u16x4 v = *reinterpret_cast<const u16x4_a2*>(row + e0 + i);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (i + q < V) x[i + q] = to_f32((bf16_t)v[q]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < count ? to_f32(row[e0 + i]) : -__builtin_inff();
    }
    // NaN is as little a choice as -inf
    float most = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = x[i] > -__builtin_inff() ? x[i] : -__builtin_inff();
        most = fmaxf(most, x[i]);
    }
    most = lanes_max<L>(most);
    float total = 1.0f;
    if (!p.sigmoid && !p.renormalize) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) s += x[i] > -__builtin_inff() ? exp_below(x[i], most) : 0.0f;
        total = lanes_sum<L>(s);
    }
    K c[V];
    if constexpr (sizeof(K) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = x[i];
    } else {
        double sum = 1.0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            c[i] = p.sigmoid ? 1.0 / (1.0 + exp(-(double)x[i]))
                   : x[i] > -__builtin_inff() ? exp_below((double)x[i], (double)most) : 0.0;
        if (!p.sigmoid) {
            sum = 0.0;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += c[i];
            sum = lanes_sum<L>(sum);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (!p.sigmoid) c[i] /= sum;
            if (p.bias) c[i] += i < count ? (double)p.bias[e0 + i] : 0.0;
            c[i] = x[i] > -__builtin_inff() && c[i] > key_low<K>() ? c[i] : key_low<K>();
        }
    }
    if (p.groups > 1) {
        K a = key_low<K>(), b = key_low<K>();  // the group's two largest
#pragma unroll
        for (int i = 0; i < V; ++i) {
            b = max_of(b, c[i] < a ? c[i] : a);
            a = max_of(a, c[i]);
        }
        for (int d = 1; d < p.lanes_per_group; d *= 2) {
            const K a2 = __shfl_xor(a, d), b2 = __shfl_xor(b, d);
            b = max_of(a < a2 ? a : a2, max_of(b, b2));
            a = max_of(a, a2);
        }
        K score = p.group_top > 1 && b > key_low<K>() ? a + b : a;
        bool kept = false;
        for (int j = 0; j < p.top_groups; ++j) {
            const K best = lanes_max<L>(kept ? key_low<K>() : score);
            const int first = first_lane<L>(!kept && score == best, lane);
            kept |= group == (first & (L - 1)) / p.lanes_per_group && first < 64;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = kept ? c[i] : key_low<K>();
    }
    // the lane's largest and where it is
    K best;
    int at;
    auto look = [&]() __attribute__((always_inline)) {
        best = c[0];
        at = 0;
#pragma unroll
        for (int i = 1; i < V; ++i) {
            at = c[i] > best ? i : at;
            best = max_of(best, c[i]);
        }
    };
    look();
    for (int j = 0; j < p.top; ++j) {
        const K m = lanes_max<L>(best);
        const int first = first_lane<L>(best == m, lane);
        if (lane == first) {
            const bool any = m > key_low<K>();
            picked[j] = any ? e0 + at : -1;
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] = any && i == at ? key_low<K>() : c[i];
            look();
        }
    }
    wave_sync();
    // the weights, one per lane
    const int e = sub < p.top ? picked[sub] : -1;
    const float xe = e >= 0 ? to_f32(row[e]) : -__builtin_inff();
    const float m = p.renormalize ? lanes_max<L>(xe) : most;
    float w = e >= 0 ? chosen_score(p, xe, m) : 0.0f;
    if (p.renormalize) total = lanes_sum<L>(w);
    if (live && sub < p.top) {
        const int64_t o = (int64_t)t * p.top + sub;
        p.ids[o] = e;
        p.weights[o] = e >= 0 ? w / total * p.scale : 0.0f;
    }
}

// Which of a chunk's tokens chose an expert, as bits.
struct ChosenBits {
    uint32_t w[ROUTE_MAX_EXPERTS][2];
};
__device__ __forceinline__ void clear_bits(ChosenBits& b, int experts)
{
    for (int e = threadIdx.x; e < experts; e += blockDim.x) b.w[e][0] = b.w[e][1] = 0;
}
__device__ __forceinline__ int count_bits(const ChosenBits& b, int e)
{
    return __popc(b.w[e][0]) + __popc(b.w[e][1]);
}
// ... of those before token t of the chunk.
__device__ __forceinline__ int rank_bits(const ChosenBits& b, int e, int t)
{
    const uint32_t below = (1u << (t & 31)) - 1u;
    return t < 32 ? __popc(b.w[e][0] & below) : __popc(b.w[e][0]) + __popc(b.w[e][1] & below);
}

// Exclusive sum of n[0 .. experts) in place, the total to *total; ends with a
// barrier.  Every thread of the workgroup takes part.
__device__ __forceinline__ void scan_experts(int* n, int experts, int* wave_sum, int* total)
{
    const int lane = threadIdx.x & 63, waves = blockDim.x / 64, wave = threadIdx.x >> 6;
    int carry = 0;
    for (int base = 0; base < experts; base += blockDim.x) {
        const int e = base + threadIdx.x;
        const int x = e < experts ? n[e] : 0, incl = wave_scan(x);
        if (lane == 63) wave_sum[wave] = incl;
        __syncthreads();
        int before = carry;
        for (int w = 0; w < waves; ++w) {
            const int s = wave_sum[w];
            before += w < wave ? s : 0;
            carry += s;
        }
        if (e < experts) n[e] = before + incl - x;
        __syncthreads();
    }
    if (threadIdx.x == 0) *total = carry;
    __syncthreads();
}

// Rows of the chunk's assignments: expert e's begin at start[e].
__device__ __forceinline__ void place_rows(const RouteArgs& p, int t0, int tokens, const ChosenBits& bits,
                                           const int* start)
{
    for (int i = threadIdx.x; i < tokens * p.top; i += blockDim.x) {
        const int64_t a = (int64_t)t0 * p.top + i;
        const int e = p.ids[a];
        const int r = e >= 0 ? start[e] + rank_bits(bits, e, i / p.top) : -1;
        p.position[a] = r;
        if (e >= 0) p.order[r] = (int32_t)a;
    }
}

// Chooses the experts of `chunk` tokens per workgroup.  PLAN: counts them by
// expert for route_place, or (a single workgroup) makes the plan at once.
template <typename X, int L, int V, typename K>
__global__ __launch_bounds__(1024) void route_kernel(RouteArgs p)
{
    const int threads = blockDim.x, pass = threads / L;  // tokens at a time
    __shared__ int32_t picked[1024 / L][ROUTE_MAX_TOP];
    __shared__ ChosenBits bits;
    __shared__ int start[ROUTE_MAX_EXPERTS];
    __shared__ int wave_sum[16], total;
    const bool plan = p.order != nullptr;
    const int t0 = blockIdx.x * p.chunk;
    const int tokens = p.tokens - t0 < p.chunk ? p.tokens - t0 : p.chunk;
    if (plan) {
        clear_bits(bits, p.experts);
        __syncthreads();
    }
    const int slot = threadIdx.x / L, sub = threadIdx.x & (L - 1);
    for (int i = slot; i - slot < tokens; i += pass) {
        route_token<X, L, V, K>(p, t0 + i, i < tokens, picked[slot]);
        if (plan && i < tokens && sub < p.top) {
            const int e = picked[slot][sub];
            if (e >= 0) atomicOr(&bits.w[e][i >> 5], 1u << (i & 31));
        }
        wave_sync();
    }
    if (!plan) return;
    __syncthreads();
    if (gridDim.x > 1) {
        for (int e = threadIdx.x; e < p.count_ld; e += threads)
            p.counts[(int64_t)blockIdx.x * p.count_ld + e] = e < p.experts ? count_bits(bits, e) : 0;
        return;
    }
    for (int e = threadIdx.x; e < p.experts; e += threads) start[e] = count_bits(bits, e);
    __syncthreads();
    scan_experts(start, p.experts, wave_sum, &total);
    place_rows(p, t0, tokens, bits, start);
    for (int e = threadIdx.x; e <= p.experts; e += threads)
        p.offsets[e] = e < p.experts ? start[e] : total;
    for (int r = total + threadIdx.x; r < p.tokens * p.top; r += threads) p.order[r] = -1;
}

}  // namespace dg
