// Low-rank adapters of many requests beside a shared product:
//     D = alpha * (X op(W) + s_a (X op(down_a)) op(up_a)) + beta * C
// where a is the adapter of the row's segment (none: the shared product
// alone), op(down_a) is K x R and op(up_a) R x N with a small rank R.
//
// Two launches.  The streaming kernel forms T = s_a X op(down_a), rows x R, in
// fp32 (R padded to whole fragments with zeros); the shared product then runs
// as it does alone, and its epilogue adds T op(up_a) to the accumulators
// (lora_fragment; the streaming kernel adds lora_row to its sums), so D is
// written once and rounded once.  Where all rows of an output tile share an
// adapter, T and up are more of the product's K instead: T's terms and up_a
// go through LDS behind the last step of X and W.
// The second product costs 2 M R N operations beside 2 M K N.  T stays fp32
// in memory; as bf16 MFMA operands it goes in as a sum of bf16 terms (each of
// what the ones before leave), two where D is bf16 and three where D is fp32.
// One term's rounding, up to 2^-8 of the low-rank part, would be as large as that
// of a bf16 D itself; two keep 16 bits, which an fp32 D shows (487 rows of
// 4608x1152, rank 4: 1.3e-6 off the 64-bit result, 0.6e-6 with fp32 T), three 24.
#pragma once

#include "common.hpp"
#include "mfma_gemm.hpp"
#include "ragged.hpp"

namespace dg {

// T is padded to whole fragments of rank along k: LORA_PAD columns.
constexpr int LORA_PAD = 16;

// Ranks that RAG_LORA_ONE (stream.hpp) takes at most.
constexpr int LORA_ONE_RANK = 32;

// VEC consecutive k of one row (or column) with every index clamped into
// [0, K) and zero past K.  `x` points at the row; ks: elements between k.
template <typename T>
__device__ __forceinline__ u32x4 clamped_chunk(const T* x, int64_t ks, int k, int K)
{
    constexpr int VEC = 16 / sizeof(T);
    T e[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) e[v] = x[(int64_t)(k + v < K ? k + v : K - 1) * ks];
#pragma unroll
    for (int v = 0; v < VEC; ++v) e[v] = k + v < K ? e[v] : T(0);
    return pack_chunk<T>(e);
}

// Terms of T that make up one MFMA operand of KIND's type beside a D of bf16
// (OUT_BF16) or fp32.
template <typename T, bool OUT_BF16>
constexpr int LORA_TERMS = sizeof(T) == 4 ? 1 : OUT_BF16 ? 2 : 3;

// fp32 values as MFMA operand terms: bf16 as a sum of N, fp32 as itself.  An
// infinite or NaN term takes zeros behind it, so an infinity stays one.
template <int N>
__device__ __forceinline__ void split_terms(const float (&t)[8], u32x4 (&v)[N])
{
    float rest[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) rest[e] = t[e];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        bf16x8 h;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[e] = (__bf16)rest[e];
            const float hf = (float)h[e];
            rest[e] = fabsf(hf) <= 3.402823466e38f ? rest[e] - hf : 0.0f;
        }
        v[n] = __builtin_bit_cast(u32x4, h);
    }
}
__device__ __forceinline__ void split_terms(const float (&t)[4], u32x4 (&v)[1])
{
    v[0] = u32x4{__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]),
                 __float_as_uint(t[3])};
}

// T as bf16 operand terms in memory: row r holds p.terms (2 or 3) runs of
// rank_pad columns, one per term.  Four columns of it.
__device__ __forceinline__ void store_terms(const RaggedArgs& p, int64_t row, int col, const f32x4& t)
{
    const float e[8] = {t[0], t[1], t[2], t[3]};
    u32x4 v[3];
    split_terms(e, v);
    uint16_t* d = p.t_terms + row * p.terms * p.rank_pad + col;
#pragma unroll
    for (int n = 0; n < 3; ++n)
        if (n < p.terms) *reinterpret_cast<uint2*>(d + n * p.rank_pad) = uint2{v[n][0], v[n][1]};
}

// ... one column.
__device__ __forceinline__ void store_term(const RaggedArgs& p, int64_t row, int col, float t)
{
    const float e[8] = {t};
    u32x4 v[3];
    split_terms(e, v);
    uint16_t* d = p.t_terms + row * p.terms * p.rank_pad + col;
#pragma unroll
    for (int n = 0; n < 3; ++n)
        if (n < p.terms) d[n * p.rank_pad] = (uint16_t)v[n][0];
}

// adapter[r] = the adapter of row m0 + r for the BM rows of a tile, or -1;
// ends with a barrier.  (Where segments overlap, one of theirs.)
template <int BM, int THREADS>
__device__ __forceinline__ void map_adapters(const RaggedArgs& p, int m0, int tid, int* adapter)
{
    const int lane = tid & 63;
    for (int r = tid; r < BM; r += THREADS) adapter[r] = -1;
    __syncthreads();
    for (int s0 = tid - lane; s0 < p.groups; s0 += THREADS) {
        int lo = 0, n = 0, a = -1;
        if (s0 + lane < p.groups) {
            group_span(p, s0 + lane, lo, n);
            a = p.ids ? p.ids[s0 + lane] : s0 + lane;
        }
        const int first = lo > m0 ? lo - m0 : 0;
        const int end = lo + n < m0 + BM ? lo + n - m0 : BM;
        uint64_t live = __ballot(n > 0 && first < end && a >= 0 && a < p.adapters);
        for (; live != 0; live &= live - 1) {
            const int src = __builtin_ctzll(live);
            const int e = __builtin_amdgcn_readlane(end, src), v = __builtin_amdgcn_readlane(a, src);
            for (int r = __builtin_amdgcn_readlane(first, src) + lane; r < e; r += 64) adapter[r] = v;
        }
    }
    __syncthreads();
}

// The adapter of every row of [m0, m_end), or TILE_NONE where no row has one,
// or TILE_MIXED (also where `whole` is false).  Every lane of the wave takes
// part.
enum : int { TILE_NONE = -1, TILE_MIXED = -2 };
__device__ __forceinline__ int tile_adapter(const RaggedArgs& p, int m0, int m_end, int lane, bool whole)
{
    int found = TILE_NONE;
    for (int s0 = 0; s0 < p.groups; s0 += 64) {
        int lo = 0, n = 0, a = -1;
        if (s0 + lane < p.groups) {
            group_span(p, s0 + lane, lo, n);
            a = p.ids ? p.ids[s0 + lane] : s0 + lane;
        }
        const bool here = a >= 0 && a < p.adapters && n > 0 && lo < m_end && lo + n > m0;
        const uint64_t all = __ballot(here && lo <= m0 && lo + n >= m_end);
        if (all != 0 && whole) return __builtin_amdgcn_readlane(a, __builtin_ctzll(all));
        if (__ballot(here) != 0) found = TILE_MIXED;
    }
    return found;
}

template <int BYTES>
struct RawLoad;
template <>
struct RawLoad<4> {
    typedef uint32_t T __attribute__((ext_vector_type(1), aligned(2)));
};
template <>
struct RawLoad<8> {
    typedef uint32_t T __attribute__((ext_vector_type(2), aligned(2)));
};
template <>
struct RawLoad<16> {
    typedef uint32_t T __attribute__((ext_vector_type(4), aligned(2)));
};

// Ranks k .. k + 4 V - 1 of a row's T, summed over the slices of K.  Up to four
// slices, read at once.
template <int V>
__device__ __forceinline__ void load_t(const RaggedArgs& p, int row, int k, f32x4 (&t)[V])
{
    const float* src = p.t + (int64_t)row * p.rank_pad + k;
    const int64_t slice = (int64_t)p.rows * p.rank_pad;
    if (p.splits == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) t[v] = reinterpret_cast<const f32x4*>(src)[v];
        return;
    }
    f32x4 q[4][V];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int v = 0; v < V; ++v)
            q[s][v] = reinterpret_cast<const f32x4*>(src + (s < p.splits ? s : 0) * slice)[v];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        t[v] = q[0][v] + q[1][v];
#pragma unroll
        for (int s = 2; s < 4; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) t[v][e] += s < p.splits ? q[s][v][e] : 0.0f;
    }
}

// A row's T op(up_a), four columns from `col` (`inside`: of a tile that lies
// inside the matrix, the same for every lane), in fp32 (T is not rounded on
// this path), eight ranks at a time: get_t(r, t) gives ranks r .. r + 7.
template <typename T, class F>
__device__ __forceinline__ f32x4 lora_row(const RaggedArgs& p, int col, int a, bool inside, F get_t)
{
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    const T* up = static_cast<const T*>(p.up) + (int64_t)a * p.stride_up;
    for (int r = 0; r < p.rank; r += 8) {
        f32x4 t[2];
        get_t(r, t);
        T u[4][8];
        if (inside && p.up_kc && r + 8 <= p.rank) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                u32x4_elem<T> c[sizeof(T) / 2];
#pragma unroll
                for (int h = 0; h < (int)sizeof(T) / 2; ++h)
                    c[h] = reinterpret_cast<const u32x4_elem<T>*>(up + (col + s) * p.ld_up + r)[h];
                __builtin_memcpy(u[s], c, sizeof(u[s]));
            }
        } else if (inside && !p.up_kc) {
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                using C = typename RawLoad<4 * sizeof(T)>::T;
                const C c = *reinterpret_cast<const C*>(
                    up + (int64_t)(r + v < p.rank ? r + v : p.rank - 1) * p.ld_up + col);
                T e[4];
                __builtin_memcpy(e, &c, sizeof(e));
#pragma unroll
                for (int s = 0; s < 4; ++s) u[s][v] = e[s];
            }
        } else {
            const int64_t kr = p.up_kc ? 1 : p.ld_up, kc = p.up_kc ? p.ld_up : 1;
#pragma unroll
            for (int v = 0; v < 8; ++v)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    u[s][v] = up[(r + v < p.rank ? r + v : p.rank - 1) * kr +
                                 (col + s < p.N ? col + s : p.N - 1) * kc];
        }
#pragma unroll
        for (int v = 0; v < 8; ++v)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                sum[s] += r + v < p.rank ? t[v / 4][v % 4] * to_f32(u[s][v]) : 0.0f;
    }
    return sum;
}

// T op(up_a) of a fragment of 32 rows from `row0` (of a tile whose rows start
// at m_tile and have the adapters adapter[]) and NQ fragments of 32 columns
// from `col0`, added to the sums a lane holds of them: row l % 32, four columns
// each in sum[q][vg] (the epilogue's copies of the accumulators: adding to the
// accumulators themselves, in code with branches, makes the compiler copy and
// spill them).
//
// The fragment takes its rows' adapters one after another, into a product of
// its own that only the adapter's rows add: whatever an adapter holds
// (infinities, NaN) reaches no other row.  The loads are free of branches
// (clamped and zeroed instead), and the first adapter's are issued ahead of
// T's, so a fragment of one adapter waits for memory once per 32 ranks.
template <int KIND, bool OUT_BF16, int NQ, int VG>
__device__ __forceinline__ void lora_fragment(const RaggedArgs& p, const int* adapter, int m_tile,
                                              int row0, int col0, int lane, f32x4 (&sum)[NQ][VG])
{
    using T = typename MfmaShape<KIND>::T;
    using Acc = typename AccType<KIND>::type;
    constexpr int FM = MfmaShape<KIND>::FM, VEC = 16 / sizeof(T), KSTEP = 64 / FM * VEC;
    constexpr int NK = 2;  // fragment steps of rank at once
    constexpr int TERMS = LORA_TERMS<T, OUT_BF16>;
    static_assert(FM == 32 && VG == 4, "accumulator layout");
    int row = row0 + lane % FM;
    const int mine = row < p.M ? adapter[row - m_tile] : -1;
    const uint64_t some = __ballot(mine >= 0);
    if (some == 0) return;
    if (row >= p.M) row = p.M - 1;
    const int kl = VEC * (lane / FM);
    for (int r0 = 0; r0 < p.rank; r0 += NK * KSTEP) {
        u32x4 b[NQ][NK];
        auto load_up = [&](int a) __attribute__((always_inline)) {
            const T* up = static_cast<const T*>(p.up) + (int64_t)a * p.stride_up;
            int64_t at[NQ];
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int col = col0 + q * FM + lane % FM;
                at[q] = (int64_t)(col < p.N ? col : p.N - 1) * (p.up_kc ? p.ld_up : 1);
            }
            if (p.up_kc && p.rank % VEC == 0) {
#pragma unroll
                for (int q = 0; q < NQ; ++q)
#pragma unroll
                    for (int kk = 0; kk < NK; ++kk) {
                        const int k = r0 + kk * KSTEP + kl;
                        const u32x4 v = *reinterpret_cast<const u32x4_elem<T>*>(
                            up + at[q] + (k < p.rank ? k : 0));
                        b[q][kk] = k < p.rank ? v : u32x4{0, 0, 0, 0};
                    }
            } else {
#pragma unroll
                for (int q = 0; q < NQ; ++q)
#pragma unroll
                    for (int kk = 0; kk < NK; ++kk)
                        b[q][kk] = clamped_chunk<T>(up + at[q], p.up_kc ? 1 : p.ld_up,
                                                    r0 + kk * KSTEP + kl, p.rank);
            }
        };
        int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(some));
        load_up(a);
        // the rows' T as operand terms
        u32x4 terms[NK][TERMS];
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
            const int k = r0 + kk * KSTEP + kl;
            f32x4 q[VEC / 4];
            load_t(p, row, k < p.rank_pad ? k : 0, q);
            float t[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) t[e] = k < p.rank_pad ? q[e / 4][e % 4] : 0.0f;
            split_terms(t, terms[kk]);
        }
        for (uint64_t left = some;;) {
            left &= ~__ballot(mine == a);
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                Acc v = {};
#pragma unroll
                for (int kk = 0; kk < NK; ++kk)
#pragma unroll
                    for (int n = 0; n < TERMS; ++n) mfma_step<KIND>(b[q][kk], terms[kk][n], v);
#pragma unroll
                for (int e = 0; e < 4 * VG; ++e) sum[q][e / 4][e % 4] += mine == a ? v[e] : 0.0f;
            }
            if (left == 0) break;
            a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
            load_up(a);
        }
    }
}

// 16x16 products of 16-byte k-chunks: lane l holds row (a) or column (b) l % 16
// at k-chunk l / 16; the result has row l % 16, columns 4 (l / 16) .. + 3.
template <typename T>
__device__ __forceinline__ void mfma16(const u32x4& a, const u32x4& b, f32x4& acc)
{
    if constexpr (sizeof(T) == 2) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b),
                                                      __builtin_bit_cast(bf16x8, a), acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b[e]), __uint_as_float(a[e]),
                                                       acc, 0, 0, 0);
    }
}

}  // namespace dg
