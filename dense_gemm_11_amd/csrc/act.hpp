// Product with bias, activation, gate and residual in its epilogue, for ragged
// groups of rows or one dense matrix:
//     Z = alpha s_g A op(B_g) + bias_g
//     D = act(Z) + R                      (RAG_ACT)
//     D = act(Z[:, :N]) * Z[:, N:] + R    (RAG_GATE: op(B_g) is K x 2N)
// and the gradient of what follows the product.
//
// A gated output needs a gate's column and its partner N columns on.  Both are in
// one workgroup's tile: its columns are, for each wave, a run of N's columns and
// the same run N further, so the wave that holds a gate's accumulators holds the
// partner's, D is written once and Z only if it is asked for (without the fusion:
// Z written and read again, 4 N elements a row beside the N of D).
//
// The products bound it as they do without all this: 384 rows of 64 experts of
// 4096 x 2 1792 bf16 read their matrices at 5.7 TB/s (286 us), 16384 rows of 8 of
// 4096 x 2 14336 take 3.17 ms (1.2 PFLOP/s; even groups 3.09, silu 1 % of it, gelu 2),
// two of 2048 x 2 1024 a launch and a trip to memory (6.0 us).
#pragma once

#include "common.hpp"
#include "ragged.hpp"

namespace dg {

enum : int { EPI_ACT_SILU = 3, EPI_ACT_GELU_TANH = 4 };

struct ActArgs : RaggedArgs {
    const void* z_bias;   // D's type, or null: groups of the products' columns
    int64_t stride_bias;
    void* Z;              // D's type, or null
    const void* R;        // D's type, or null
    int64_t ldz, ldr;
};

// s(x) = 1 / (1 + e^-x) and 1 - s(x), both from e^-|x|, which cannot overflow.
// PRECISE: to fp32's last places, else by the hardware's exponential and
// reciprocal (an error of 2^-22 or so before D's rounding to bf16).
template <bool PRECISE>
__device__ __forceinline__ void sigmoids(float x, float& s, float& rest)
{
    const float ax = fabsf(x);
    const float e = PRECISE ? expf(-ax) : __builtin_amdgcn_exp2f(ax * -1.44269504088896341f);
    const float up = PRECISE ? 1.0f / (1.0f + e) : __builtin_amdgcn_rcpf(1.0f + e);
    s = x < 0.0f ? e * up : up;
    rest = x < 0.0f ? up : e * up;
}

// The normal distribution's Phi(x).  The fast form takes the tail Phi(-|x|) as
// e^(-a^2) / 2 times a polynomial in 1 / (1 + 0.36 a), a = |x| / sqrt 2, so it keeps
// its relative accuracy where 1 - erf would cancel.  The polynomial is a weighted
// minimax fit to e^(a^2) erfc(a) on [0, 9.4], which is as far as e^(-a^2) is a normal
// number: the tail is off by 4e-6 of itself at most, and by 4e-8 absolutely, and
// by the roundings of a^2 (formula 7.1.26's five terms, which bound the absolute
// error alone, were off by 1.6e-3 of the tail at x = -5 and 2e-2 at -10).
template <bool PRECISE>
__device__ __forceinline__ float normal_cdf(float x)
{
    if constexpr (PRECISE) return 0.5f * erfcf(x * -0.70710678118654752f);
    const float a = fabsf(x) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.36f * a);
    const float poly =
        t * (0.2022218704f +
             t * (0.2163794935f +
                  t * (0.1087818071f +
                       t * (0.4258081019f +
                            t * (-0.3520432115f + t * (0.5619213581f + t * -0.1630693525f))))));
    const float tail = 0.5f * poly * __builtin_amdgcn_exp2f(-(a * a) * 1.44269504088896341f);
    return x < 0.0f ? tail : 1.0f - tail;
}

// 2 sqrt(2 / pi): gelu by tanh is x s(TANH_C (x + 0.044715 x^3)).
constexpr float TANH_C = 1.59576912160573080f, TANH_K = 0.044715f;

// What s is taken of: x for silu (and not the cubic by a factor of 0, which makes a
// NaN of an infinite x), and its slope, with the square kept finite.
__device__ __forceinline__ float sigmoid_argument(float x, int act)
{
    return act == EPI_ACT_SILU ? x : TANH_C * (x + TANH_K * x * x * x);
}
__device__ __forceinline__ float argument_slope(float x, int act)
{
    return act == EPI_ACT_SILU ? 1.0f : TANH_C * (1.0f + 3.0f * TANH_K * fminf(x * x, 3e38f));
}

// act(x); act is uniform across a launch.
template <bool PRECISE>
__device__ __forceinline__ f32x4 act_value4(f32x4 x, int act)
{
    f32x4 r = x;
    if (act == EPI_ACT_SILU || act == EPI_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float s, rest;
            sigmoids<PRECISE>(sigmoid_argument(x[i], act), s, rest);
            r[i] = x[i] * s;
        }
    } else if (act == EPI_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = x[i] * normal_cdf<PRECISE>(x[i]);
    } else if (act == EPI_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = x[i] <= 0.0f ? 0.0f : x[i];  // (a NaN stays)
    }
    return r;
}

// act(x) and act'(x).
template <bool PRECISE>
__device__ __forceinline__ void act_slope(float x, int act, float& value, float& slope)
{
    value = x;
    slope = 1.0f;
    if (act == EPI_ACT_SILU || act == EPI_ACT_GELU_TANH) {
        float s, rest;
        sigmoids<PRECISE>(sigmoid_argument(x, act), s, rest);
        value = x * s;
        slope = s + value * rest * argument_slope(x, act);  // (far out value * rest is 0)
    } else if (act == EPI_ACT_GELU) {
        const float phi = normal_cdf<PRECISE>(x), q = -0.5f * x * x;
        const float e = PRECISE ? expf(q) : __builtin_amdgcn_exp2f(q * 1.44269504088896341f);
        value = x * phi;
        slope = phi + x * (e * 0.39894228040143268f);
    } else if (act == EPI_ACT_RELU) {
        slope = x > 0.0f ? 1.0f : 0.0f;
        value = x <= 0.0f ? 0.0f : x;
    }
}

// The workgroup's tile among the groups', or among one matrix's without offsets.
template <int BM>
__device__ __forceinline__ bool find_act_tile(const RaggedArgs& p, int tiles_n, RowTile& t)
{
    if (p.offsets) return find_row_tile<BM>(p, blockIdx.x, tiles_n, t);
    t.tiles_m = (p.M + BM - 1) / BM;
    const int tiles = t.tiles_m * tiles_n;
    if ((int)blockIdx.x >= tiles) return false;
    t.group = t.start = t.first = 0;
    t.size = p.M;
    t.in_group = block_cyclic(blockIdx.x, tiles);
    return true;
}

// Narrow p to the workgroup's group, as narrow_to_group does for the products
// alone, and (tm, tn) to its tile.  False when the workgroup has none.
template <int BM, typename T, typename OutT>
__device__ __forceinline__ bool narrow_act(ActArgs& p, int& tm, int& tn)
{
    RowTile t;
    if (!find_act_tile<BM>(p, p.tiles_n, t)) return false;
    p.M = t.size;
    p.tiles_m = t.tiles_m;
    tile_of(p, t.in_group, tm, tn);
    p.A = static_cast<const T*>(p.A) + (int64_t)t.start * p.lda;
    p.B = static_cast<const T*>(p.B) + (int64_t)t.group * p.stride_b;
    p.D = reinterpret_cast<float*>(reinterpret_cast<OutT*>(p.D) + (int64_t)t.start * p.ldd);
    if (p.Z) p.Z = static_cast<OutT*>(p.Z) + (int64_t)t.start * p.ldz;
    if (p.R) p.R = static_cast<const OutT*>(p.R) + (int64_t)t.start * p.ldr;
    if (p.z_bias) p.z_bias = static_cast<const OutT*>(p.z_bias) + (int64_t)t.group * p.stride_bias;
    p.alpha = group_alpha(p, t.group, t.size);
    return true;
}

// Four values from or to x: those from `skip` up to n, the others 0 or left.
template <typename OutT>
__device__ __forceinline__ f32x4 load_four(const OutT* x, int n, int skip = 0)
{
    f32x4 v;
    if (n >= 4 && skip <= 0) {
        if constexpr (sizeof(OutT) == 2) {
            const u16x4 h = *reinterpret_cast<const u16x4_a2*>(x);
            v = f32x4{to_f32(h[0]), to_f32(h[1]), to_f32(h[2]), to_f32(h[3])};
        } else {
            v = *reinterpret_cast<const f32x4_a4*>(x);
        }
    } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s] = s >= skip && s < n ? to_f32(x[s]) : 0.0f;
    }
    return v;
}
template <typename OutT>
__device__ __forceinline__ void store_four(OutT* x, f32x4 v, int n, int skip = 0)
{
    if (n >= 4 && skip <= 0) {
        if constexpr (sizeof(OutT) == 2)
            *reinterpret_cast<bf16x4_a2*>(x) = __builtin_convertvector(v, bf16x4);
        else
            *reinterpret_cast<f32x4_a4*>(x) = v;
    } else {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if (s >= skip && s < n) x[s] = from_f32<OutT>(v[s]);
    }
}

// Outputs (row, col .. col+3), those from `skip` up to n of them, from the
// products' sums g and, gated, u of the partner columns: bias, Z, activation,
// gate, residual, D.
template <bool GATE, typename OutT>
__device__ __forceinline__ void act_outputs(const ActArgs& p, int row, int col, int n, f32x4 g, f32x4 u,
                                            f32x4 bias_g, f32x4 bias_u, int skip = 0)
{
    constexpr bool PRECISE = sizeof(OutT) == 4;
    g = p.alpha * g + bias_g;
    if constexpr (GATE) u = p.alpha * u + bias_u;
    if (p.Z) {
        OutT* z = static_cast<OutT*>(p.Z) + (int64_t)row * p.ldz + col;
        store_four(z, g, n, skip);
        if constexpr (GATE) store_four(z + p.N, u, n, skip);
    }
    f32x4 d = act_value4<PRECISE>(g, p.act);
    if constexpr (GATE) d *= u;
    if (p.R) d += load_four(static_cast<const OutT*>(p.R) + (int64_t)row * p.ldr + col, n, skip);
    store_four(reinterpret_cast<OutT*>(p.D) + (int64_t)row * p.ldd + col, d, n, skip);
}
// Bias of columns col .. col+3 (0 without one, and beyond `n`).
template <typename OutT>
__device__ __forceinline__ f32x4 act_bias(const ActArgs& p, int col, int n)
{
    return p.z_bias && n > 0 ? load_four(static_cast<const OutT*>(p.z_bias) + col, n) : f32x4{};
}

}  // namespace dg
