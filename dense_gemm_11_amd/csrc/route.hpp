// Routing of tokens to experts.  With x the router's logits of one token,
//     s_e = softmax(x)_e or 1 / (1 + exp(-x_e)),   c_e = s_e + b_e,
// the token's experts are the `top` largest c, in descending order and the lower
// index first among equals, out of the `top_groups` groups of E / groups
// neighbouring experts whose group_top (1 or 2) largest c sum highest.  Their
// weights are scale * s, or scale * s over the sum of the chosen s.
//
// Scores next to each other decide what is chosen, so c is compared in 64 bits;
// without a bias the logits themselves are compared, whose order is that of the
// scores.  The weights are formed in fp32 from the logits of the chosen.  A logit
// (or c) of -inf or NaN is never chosen; of +inf the softmax is its limit.
//
// L lanes hold a token, V experts each, in the experts' order.  Each of the `top`
// rounds takes the largest of the lanes' maxima (4 exchanges within 16 lanes) and
// strikes it out.  Four tokens to a wave (L = 16) share the rounds' instructions,
// which are what bounds the launch: 16384 tokens of 256 experts, in groups and with
// a bias, top 8, take 957 vector instructions a wave and 14.7 us in a trace (the
// bytes alone would take 3.5), and the plan 6.1; the whole call, from a graph, 17 us on
// the same logits again and 19 to 20 on others each time.
//
// route_quick does so on 32-bit integers in the order of the values with the
// expert's place in their low bits, so that no two are equal, striking out takes a
// compare and a select for each, and every lane knows the expert.  bf16 logits
// leave 16 bits free; of others the places take the last 8 or so.  Where two
// neighbours among the chosen (or the last of them and the next) are closer than
// what is cut off, or scores closer than their fp32 errors, the token's candidates,
// one to a lane, are compared for certain (route_rank).  A token for which that is
// not enough (three so close, sums of groups, softmax scores with a bias that 32
// bits cannot tell apart) is chosen for again in 64 bits by a wave of its own once
// its workgroup is done with the others (route_exact): 3 to 4 us more for a launch
// with a few of them.  Where all tokens are such, fp32 logits that are all equal as
// in a router that begins at zero, a workgroup's 16 waves take them in rounds, up
// to eight: 96 tokens of 64 experts 6.3 -> 16.1 us, with a bias 7.0 -> 22.3; 16384 of
// 256, top 8, 15.1 -> 29.0 and 16.0 -> 40.5 (equal bf16 logits without a bias cost
// nothing more: their keys hold all of the value).
#pragma once

#include "common.hpp"
#include "dense_gemm.h"
#include "ragged.hpp"

namespace dg {

constexpr int ROUTE_MAX_EXPERTS = 1024, ROUTE_MAX_TOP = 32;
constexpr int ROUTE_CHUNK = 64;    // tokens whose experts are counted together, at most
constexpr int ROUTE_ONE = 128;     // ... by a single workgroup, which makes the plan
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

// x of one lane.
template <int LANE>
__device__ __forceinline__ float lane_of(float x)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), LANE));
}
template <int LANE>
__device__ __forceinline__ double lane_of(double x)
{
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(x), LANE),
                            __builtin_amdgcn_readlane(__double2loint(x), LANE));
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
    if constexpr (L == 64) x = op(op(lane_of<0>(x), lane_of<16>(x)), op(lane_of<32>(x), lane_of<48>(x)));
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

// V values from x, `count` of them (V: as vectors), the others `rest`.
template <int V, typename X>
__device__ __forceinline__ void load_part(float (&v)[V], const X* x, int count, float rest)
{
    if (count == V && V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            if constexpr (sizeof(X) == 4) {
                const f32x4 r = *reinterpret_cast<const f32x4_a4*>(x + i);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (i + q < V) v[i + q] = r[q];
            } else {
                const u16x4 r = *reinterpret_cast<const u16x4_a2*>(x + i);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (i + q < V) v[i + q] = to_f32((bf16_t)r[q]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < count ? to_f32(x[i]) : rest;
    }
}

// A lane's part of a token: V experts from e0, `count` of them, and their logits
// (-inf beyond, and for NaN, which is as little a choice).
template <typename X, int L, int V>
struct TokenPart {
    int e0, count, group;
    float x[V];

    __device__ __forceinline__ TokenPart(const RouteArgs& p, int group_lanes, int t, bool live)
    {
        const int sub = threadIdx.x & (L - 1);
        const int log = __builtin_ctz(group_lanes), part = sub & (group_lanes - 1);
        group = sub >> log;
        e0 = group * p.group_size + part * V;
        count = group < p.groups && live ? p.group_size - part * V : 0;
        count = count < 0 ? 0 : count > V ? V : count;
        load_part(x, static_cast<const X*>(p.logits) + (int64_t)(live ? t : 0) * p.ld + (count > 0 ? e0 : 0),
                  count, -__builtin_inff());
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = fmaxf(x[i], -__builtin_inff());
    }
    // The expert in place n = V * lane + i of the token's lanes.
    __device__ static __forceinline__ int expert_at(const RouteArgs& p, int group_lanes, int n)
    {
        const int lane = n / V, log = __builtin_ctz(group_lanes);
        return (lane >> log) * p.group_size + (lane & (group_lanes - 1)) * V + n % V;
    }
    // The token's largest logit, and the sum of e^(x - most) where weights need it.
    __device__ __forceinline__ void sums(const RouteArgs& p, float& most, float& total) const;
};

// An unsigned integer in the order of x, and back.  Below LEAST: -inf, or nothing.
__device__ __forceinline__ uint32_t order_key(float x)
{
    const int i = __float_as_int(x);
    return (uint32_t)i ^ ((uint32_t)(i >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k ^ (~(uint32_t)((int)k >> 31) | 0x80000000u));
}
constexpr uint32_t LEAST = 0x00800000u;

__device__ __forceinline__ uint32_t least_of(uint32_t a, uint32_t b) { return a < b ? a : b; }
__device__ __forceinline__ uint32_t most_of(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xf, 0xf, true);
}

// op (least_of or most_of) over the lane's L lanes.
template <int L, class F>
__device__ __forceinline__ uint32_t lanes_pick(uint32_t k, F op)
{
    k = op(k, dpp<0xB1>(k));
    k = op(k, dpp<0x4E>(k));
    k = op(k, dpp<0x141>(k));
    k = op(k, dpp<0x140>(k));
    if constexpr (L == 64)
        k = op(op((uint32_t)__builtin_amdgcn_readlane((int)k, 0), (uint32_t)__builtin_amdgcn_readlane((int)k, 16)),
               op((uint32_t)__builtin_amdgcn_readlane((int)k, 32), (uint32_t)__builtin_amdgcn_readlane((int)k, 48)));
    return k;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_most(uint32_t k)
{
    return lanes_pick<L>(k, [](uint32_t a, uint32_t b) { return most_of(a, b); });
}

// The second of three where a >= b are two of them: of a, b and c.
__device__ __forceinline__ uint32_t second_of(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("v_med3_u32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// The lane's L lanes' part of a mask over the wave.
template <int L>
__device__ __forceinline__ uint64_t lanes_mask(uint64_t m, int lane)
{
    return L == 64 ? m : m >> (lane & 48) & 0xFFFFu;
}

// The largest two of a group's keys, from its lanes' (a >= b).
__device__ __forceinline__ void group_two(int lanes, uint32_t& a, uint32_t& b)
{
    auto join = [&](uint32_t a2, uint32_t b2) __attribute__((always_inline)) {
        b = most_of(least_of(a, a2), most_of(b, b2));
        a = most_of(a, a2);
    };
    if (lanes > 1) join(dpp<0xB1>(a), dpp<0xB1>(b));
    if (lanes > 2) join(dpp<0x4E>(a), dpp<0x4E>(b));
    if (lanes > 4) join(dpp<0x141>(a), dpp<0x141>(b));
    if (lanes > 8) join(dpp<0x140>(a), dpp<0x140>(b));
    if (lanes > 16) join(__shfl_xor(a, 16), __shfl_xor(b, 16));
    if (lanes > 32) join(__shfl_xor(a, 32), __shfl_xor(b, 32));
}

__device__ __forceinline__ float quick_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }
// 1 / (1 + e^-x)
__device__ __forceinline__ float quick_sigmoid(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + quick_exp(-x));
}
__device__ __forceinline__ float quick_exp_below(float x, float m) { return x == m ? 1.0f : quick_exp(x - m); }

template <typename X, int L, int V>
__device__ __forceinline__ void TokenPart<X, L, V>::sums(const RouteArgs& p, float& most, float& total) const
{
    most = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) most = x[i] > most ? x[i] : most;
    most = key_value(lanes_most<L>(order_key(most)));
    total = 1.0f;
    if (!p.sigmoid && !p.renormalize) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) s += x[i] > -__builtin_inff() ? quick_exp_below(x[i], most) : 0.0f;
        total = lanes_sum<L>(s);
    }
}

// A token's chosen logit as a score: softmax over all (e^(x - m) / sum), or with
// renormalised weights a number in proportion to it, of which the largest is
// about 1 (m the largest chosen logit): e^(x - m); e^(x - m) / (1 + e^x) for the
// sigmoid of logits below zero, whose own value may be too small for fp32.
__device__ __forceinline__ float chosen_score(const RouteArgs& p, float x, float m)
{
    if (!p.sigmoid) return quick_exp_below(x, m);
    if (!p.renormalize || x > 0.0f) return quick_sigmoid(x);
    return quick_exp(x - fminf(m, 0.0f)) * __builtin_amdgcn_rcpf(1.0f + quick_exp(x));
}

// How far a token's choice is certain.
enum : int { ROUTE_SURE = 0, ROUTE_RANK = 1, ROUTE_AGAIN = 2 };

// (see route_quick)
__device__ __forceinline__ float near_softmax(float share) { return 1.0f + 60.0f * share; }

// Chooses a token's experts: the j-th of them, and the one after the last, to lane
// j of its L lanes (-1: none), and returns how certain that is, in every lane.
// share: one over a softmax's sum, the largest p, where there is a bias.
// BIAS: by scores with a bias, which it forms in fp32.  In units u of 2^-24 a
// sigmoid is off by 4 at most and the sum c with the bias by |c| more, so two
// choices may be in the wrong order up to 8 + 2 |c| apart.  A softmax is off by
// |x - m| e^(x - m) <= 0.37 for its argument and 4 p for its exponential and
// products, and its sum by 49 of itself at most (of which 38 are additions), which
// shifts two choices against each other by 49 of the largest p: 0.8 + 57 p + 2 |c|.
// Sums of two choices are off by the choices' errors and by |c| + |c'| more (which
// may be large where the sum is not), two of them by twice the above + 8 |c|;
// without a bias, of exponentials or sigmoids up to 1, by 2 (2 4.4 + 2) < 26.
// `near` is a little more than the part that does not depend on c.
template <typename X, int L, int V, bool BIAS>
__device__ __forceinline__ int route_quick(const RouteArgs& p, const TokenPart<X, L, V>& in, float most,
                                           int& expert, float& share)
{
    constexpr int BITS = sizeof(X) == 2 && !BIAS ? 16 : __builtin_ctz(L * V);
    constexpr uint32_t PLACES = (1u << BITS) - 1u;
    constexpr bool WHOLE = BITS == 16;  // nothing of the value is cut off
    const int lane = threadIdx.x & 63, sub = lane & (L - 1);
    float near = BIAS ? 10.0f : 13.0f;
    bool again = false;
    uint32_t c[V];
    if constexpr (BIAS) {
        float s[V], b[V];
        load_part(b, p.bias + (in.count > 0 ? in.e0 : 0), in.count, 0.0f);
        if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = quick_sigmoid(in.x[i]);
        } else {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[i] = in.x[i] > -__builtin_inff() ? quick_exp_below(in.x[i], most) : 0.0f;
                sum += s[i];
            }
            share = sum = 1.0f / lanes_sum<L>(sum);
            near = near_softmax(share);
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] *= sum;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // (0 + -0 is 0; a NaN becomes -inf)
            const float v = in.x[i] > -__builtin_inff() ? s[i] + b[i] : -__builtin_inff();
            c[i] = order_key(fmaxf(v, -__builtin_inff()));
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = order_key(in.x[i] + 0.0f);  // -0 is 0
    }
    if (p.groups > 1) {
        uint32_t a = c[0], b = 0;
#pragma unroll
        for (int i = 1; i < V; ++i) {
            b = second_of(a, b, c[i]);
            a = most_of(a, c[i]);
        }
        group_two(p.lanes_per_group, a, b);
        const bool sums = p.group_top > 1;
        uint32_t score = a;
        float size = 0.0f;  // of the largest choice in a sum
        if (sums && a >= LEAST) {
            // (without a bias: of the two logits' scores, a softmax's up to its sum)
            float f = key_value(a), g = key_value(b);
            if constexpr (!BIAS) {
                f = p.sigmoid ? quick_sigmoid(f) : quick_exp_below(f, most);
                g = p.sigmoid ? quick_sigmoid(g) : quick_exp_below(g, most);
            }
            // (two live choices stay a live sum, however low: below the lowest number
            // sums are as good as equal)
            score = order_key(b >= LEAST ? fmaxf(f + g, -0x1.fffffep127f) : f);
            if constexpr (BIAS) size = fmaxf(fabsf(f), b >= LEAST ? fabsf(g) : 0.0f);
        }
        bool kept = false;
        uint32_t m = 0;
        for (int j = 0; j < p.top_groups; ++j) {
            m = lanes_most<L>(kept ? 0u : score);
            kept |= score == m && m >= LEAST;
        }
        // equal scores went in together; where that is too many, and where rounded
        // ones are as good as equal, 64 bits or the groups' order decide
        again = __popcll(lanes_mask<L>(__ballot(kept), lane)) > p.top_groups * p.lanes_per_group;
        if (BIAS || sums) {
            const uint32_t next = lanes_most<L>(kept ? 0u : score);
            const float hi = key_value(m), lo = key_value(next);
            if constexpr (BIAS) size = sums ? lanes_max<L>(size) : fmaxf(fabsf(hi), fabsf(lo));
            again |= next >= LEAST && !(hi - lo > 0x1p-24f * (2.0f * near + 9.0f * size));
        }
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = kept ? c[i] : 0u;
    }
    // the places, and the keys' distance below each choice: those not below it wrap
    // round to large numbers, so the least is the next choice's
    const uint32_t place = PLACES - V * sub;
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = (c[i] & ~PLACES) + (place - i);
    uint32_t m = 0, mine = 0;  // this choice, lane j's
    bool rank = false;
    auto next = [&]() __attribute__((always_inline)) {
        uint32_t d = m - 1u - c[0];
#pragma unroll
        for (int i = 1; i < V; ++i) d = least_of(d, m - 1u - c[i]);
        m = m - 1u - lanes_pick<L>(d, [](uint32_t a, uint32_t b) { return least_of(a, b); });
    };
    // whether hi, at the least, is above lo at the most
    auto sure = [&](uint32_t hi, uint32_t lo) __attribute__((always_inline)) {
        if constexpr (BIAS) {
            const float a = key_value(hi & ~PLACES), b = key_value(lo | PLACES);
            return a - b > 0x1p-24f * (near + 3.0f * fmaxf(fabsf(a), fabsf(b)));
        } else return (hi & ~PLACES) > (lo | PLACES);
    };
    for (int j = 0; j < p.top; ++j) {
        next();
        mine = sub == j ? m : mine;
    }
    if constexpr (!WHOLE) {
        const uint32_t last = m;
        next();
        mine = sub == p.top ? m : mine;
        // each lane's choice against the one before, of the lane before
        const uint32_t before = L == 16 ? dpp<0x111>(mine) : dpp<0x138>(mine);  // row_shr, wave_shr: 1
        const bool meet = sub > 0 && sub <= p.top && mine >= LEAST && !sure(before, mine);
        rank = lanes_mask<L>(__ballot(meet), lane) != 0;
        if (__any(rank)) {
            next();  // has to be below the last for certain
            again |= rank && m >= LEAST && !sure(last, m);
        }
    }
    expert = mine < LEAST ? -1 : TokenPart<X, L, V>::expert_at(p, p.lanes_per_group, PLACES - (mine & PLACES));
    return again ? ROUTE_AGAIN : rank ? ROUTE_RANK : ROUTE_SURE;
}

// Puts the candidates of lanes 0 .. top (one more than are chosen) in their order,
// of logits or of sigmoids with a bias in 64 bits, or of softmax scores with a bias
// in all of their 32; c: the lane's.  `tight` where another one is as near as `off`.
template <int L>
__device__ __forceinline__ int route_rank(const RouteArgs& p, int expert, double c, double off,
                                          int32_t* picked, bool& tight)
{
    const int lane = threadIdx.x & 63, sub = lane & (L - 1);
    const bool in = sub <= p.top && expert >= 0;
    c = in ? c : key_low<double>();
    const int e = in ? expert : 0x7FFFFFFF;
    int before = 0;  // candidates ahead of the lane's
    auto meet = [&](double c2, int e2) __attribute__((always_inline)) {
        before += c2 > c || (c2 == c && e2 < e);
        tight |= fabs(c2 - c) <= off && e2 != e;
    };
    if constexpr (L == 16) {
        static_for<15>([&](auto q_c) __attribute__((always_inline)) {
            constexpr int ROR = 0x121 + decltype(q_c)::value;  // row_ror: 1 to 15
            meet(dpp<ROR>(c), __builtin_amdgcn_mov_dpp(e, ROR, 0xf, 0xf, true));
        });
    } else {
        for (int q = 0; q <= p.top; ++q)
            meet(__hiloint2double(__builtin_amdgcn_readlane(__double2hiint(c), q),
                                  __builtin_amdgcn_readlane(__double2loint(c), q)),
                 __builtin_amdgcn_readlane(e, q));
    }
    if (sub < p.top) picked[sub] = -1;
    wave_sync();
    if (in && before < p.top) picked[before] = expert;
    wave_sync();
    return sub < p.top ? picked[sub] : -1;
}

// The same, certain of every case: scores with a bias and groups' sums in 64 bits,
// the lowest number first among equals.
template <typename X, int L, int V, bool BIAS>
__device__ __forceinline__ void route_exact(const RouteArgs& p, int group_lanes,
                                            const TokenPart<X, L, V>& in, float most, int32_t* picked)
{
    using K = std::conditional_t<BIAS, double, float>;
    const int lane = threadIdx.x & 63;
    // 1 / (1 + e^-x), or e^(x - most)
    auto score_of = [&](float x) __attribute__((always_inline)) -> double {
        return p.sigmoid ? 1.0 / (1.0 + exp(-(double)x))
               : x > -__builtin_inff() ? exp_below((double)x, (double)most) : 0.0;
    };
    K c[V];
    if constexpr (BIAS) {
        float b[V];
        load_part(b, p.bias + (in.count > 0 ? in.e0 : 0), in.count, 0.0f);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = score_of(in.x[i]);
            sum += c[i];
        }
        if (!p.sigmoid) sum = lanes_sum<L>(sum);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (!p.sigmoid) c[i] /= sum;
            c[i] += b[i];
            c[i] = in.x[i] > -__builtin_inff() && c[i] > key_low<K>() ? c[i] : key_low<K>();
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = in.x[i];
    }
    if (p.groups > 1) {
        K a = key_low<K>(), b = key_low<K>();  // the group's two largest
#pragma unroll
        for (int i = 0; i < V; ++i) {
            b = max_of(b, c[i] < a ? c[i] : a);
            a = max_of(a, c[i]);
        }
        for (int d = 1; d < group_lanes; d *= 2) {
            const K a2 = __shfl_xor(a, d), b2 = __shfl_xor(b, d);
            b = max_of(a < a2 ? a : a2, max_of(b, b2));
            a = max_of(a, a2);
        }
        double score = a;
        if (p.group_top > 1 && a > key_low<K>()) {
            // (without a bias: of logits' scores, a softmax's up to its sum)
            score = BIAS ? (double)a : score_of((float)a);
            if (b > key_low<K>()) score += BIAS ? (double)b : score_of((float)b);
        }
        bool kept = false;
        for (int j = 0; j < p.top_groups; ++j) {
            const double best = lanes_max<L>(kept ? key_low<double>() : score);
            const int first = first_lane<L>(!kept && score == best, lane);
            kept |= in.group == (first & (L - 1)) / group_lanes && first < 64;
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
            picked[j] = any ? in.e0 + at : -1;
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] = any && i == at ? key_low<K>() : c[i];
            look();
        }
    }
}

// Which of a chunk's tokens chose an expert, as bits.
struct __attribute__((aligned(16))) ChosenBits {
    uint32_t w[ROUTE_MAX_EXPERTS][ROUTE_ONE / 32];
};
__device__ __forceinline__ void clear_bits(ChosenBits& b, int experts)
{
    for (int e = threadIdx.x; e < experts; e += blockDim.x) *reinterpret_cast<u32x4*>(b.w[e]) = u32x4{};
}
__device__ __forceinline__ int count_bits(const ChosenBits& b, int e)
{
    const u32x4 w = *reinterpret_cast<const u32x4*>(b.w[e]);
    return __popc(w[0]) + __popc(w[1]) + __popc(w[2]) + __popc(w[3]);
}
// ... of those before token t of the chunk.
__device__ __forceinline__ int rank_bits(const ChosenBits& b, int e, int t)
{
    const u32x4 w = *reinterpret_cast<const u32x4*>(b.w[e]);
    const uint32_t below = (1u << (t & 31)) - 1u;
    int n = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) n += __popc(t >= 32 * (q + 1) ? w[q] : t >= 32 * q ? w[q] & below : 0u);
    return n;
}

// Writes ids and weights of token t (i of its chunk), lane j of its L lanes those of
// choice j, `expert`, and notes them in `bits` for a plan.
template <typename X, int L>
__device__ __forceinline__ void route_finish(const RouteArgs& p, int t, int i, bool live, float most,
                                             float total, int expert, ChosenBits& bits)
{
    const int sub = threadIdx.x & (L - 1);
    const int e = live && sub < p.top ? expert : -1;
    const float x = e >= 0 ? to_f32(static_cast<const X*>(p.logits)[(int64_t)t * p.ld + e]) : -__builtin_inff();
    const float m = p.renormalize ? lanes_max<L>(x) : most;
    const float w = e >= 0 ? chosen_score(p, x, m) : 0.0f;
    if (p.renormalize) total = lanes_sum<L>(w);
    if (!live || sub >= p.top) return;
    const int64_t o = (int64_t)t * p.top + sub;
    p.ids[o] = e;
    p.weights[o] = e >= 0 ? w * __builtin_amdgcn_rcpf(total) * p.scale : 0.0f;
    if (p.order && e >= 0) atomicOr(&bits.w[e][i >> 5], 1u << (i & 31));
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

// The row of the chunk's assignment i, of expert e, whose rows begin at start[e].
__device__ __forceinline__ void place_row(const RouteArgs& p, int t0, int i, int e, const ChosenBits& bits,
                                          const int* start)
{
    const int64_t a = (int64_t)t0 * p.top + i;
    const int r = e >= 0 ? start[e] + rank_bits(bits, e, i / p.top) : -1;
    p.position[a] = r;
    if (e >= 0) p.order[r] = (int32_t)a;
}

// Chooses the experts of `chunk` tokens per workgroup.  With a plan: counts them by
// expert for route_place, or (a single workgroup) makes the plan at once.
template <typename X, int L, int V, bool BIAS>
__global__ __launch_bounds__(1024) void route_kernel(RouteArgs p)
{
    constexpr int VX = V * L >= 4 * 64 ? V * L / 64 : V * L >= 2 * 64 ? 2 : 1;  // a wave to a token
    const int threads = blockDim.x, pass = threads / L;                         // tokens at a time
    __shared__ int32_t picked[1024 / L][ROUTE_MAX_TOP];
    __shared__ ChosenBits bits;
    __shared__ int start[ROUTE_MAX_EXPERTS];
    __shared__ int wave_sum[16], total_rows;
    __shared__ int again[ROUTE_ONE], again_count;
    const bool plan = p.order != nullptr;
    const int t0 = blockIdx.x * p.chunk;
    const int tokens = p.tokens - t0 < p.chunk ? p.tokens - t0 : p.chunk;
    if (threadIdx.x == 0) again_count = 0;
    if (plan) clear_bits(bits, p.experts);
    const int lane = threadIdx.x & 63, slot = threadIdx.x / L;
    // (a wave without a token left stays for the first pass alone, which has a barrier)
    const int wave_slot = __builtin_amdgcn_readfirstlane(slot);
    for (int i = slot; i - slot < (i == slot ? tokens : tokens - wave_slot); i += pass) {
        bool live = i < tokens;
        const TokenPart<X, L, V> in(p, p.lanes_per_group, t0 + i, live);
        float most, total;
        in.sums(p, most, total);
        int expert;
        float share = 0.0f;
        int certain = route_quick<X, L, V, BIAS>(p, in, most, expert, share);
        if (__any(certain == ROUTE_RANK)) {
            double c = 0.0, off = -1.0;
            if (live && expert >= 0) {
                const float x = to_f32(static_cast<const X*>(p.logits)[(int64_t)(t0 + i) * p.ld + expert]);
                if constexpr (BIAS) {
                    const float b = p.bias[expert];
                    if (p.sigmoid) {
                        c = 1.0 / (1.0 + exp(-(double)x)) + b;
                    } else {
                        const float v = quick_exp_below(x, most) * share + b;
                        c = v;
                        off = 0x1p-24f * (near_softmax(share) + 3.0f * fabsf(v));
                    }
                } else {
                    c = x;
                }
            }
            bool tight = false;
            const int ranked = route_rank<L>(p, expert, c, off, picked[slot], tight);
            if (BIAS && certain == ROUTE_RANK && lanes_mask<L>(__ballot(tight), lane) != 0)
                certain = ROUTE_AGAIN;
            expert = certain == ROUTE_RANK ? ranked : expert;
        }
        // (the first logits were asked for before the workgroup meets)
        if (i == slot) __syncthreads();
        if (certain == ROUTE_AGAIN && live) {
            if ((lane & (L - 1)) == 0) again[atomicAdd(&again_count, 1)] = i;
            live = false;
        }
        route_finish<X, L>(p, t0 + i, i, live, most, total, expert, bits);
    }
    __syncthreads();  // (no tokens: the first)
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int q = wave; q < again_count; q += threads / 64) {
        const int i = __builtin_amdgcn_readfirstlane(again[q]), group_lanes = p.lanes_per_group * (64 / L);
        const TokenPart<X, 64, VX> in(p, group_lanes, t0 + i, true);
        float most, total;
        in.sums(p, most, total);
        route_exact<X, 64, VX, BIAS>(p, group_lanes, in, most, picked[wave]);
        wave_sync();
        route_finish<X, 64>(p, t0 + i, i, true, most, total, lane < p.top ? picked[wave][lane] : -1, bits);
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
    scan_experts(start, p.experts, wave_sum, &total_rows);
    for (int i = threadIdx.x; i < tokens * p.top; i += threads)
        place_row(p, t0, i, p.ids[(int64_t)t0 * p.top + i], bits, start);
    for (int e = threadIdx.x; e <= p.experts; e += threads)
        p.offsets[e] = e < p.experts ? start[e] : total_rows;
    for (int r = total_rows + threadIdx.x; r < p.tokens * p.top; r += threads) p.order[r] = -1;
}

}  // namespace dg
