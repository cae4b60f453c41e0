// Low-rank adapters of many requests beside a shared product:
//     D = alpha * (X op(W) + s_a (X op(down_a)) op(up_a)) + beta * C
// where a is the adapter of the row's segment (none: the shared product
// alone), op(down_a) is K x R and op(up_a) R x N with a small rank R.
//
// Two launches.  lora_shrink_kernel forms T = s_a X op(down_a), rows x R, in
// fp32 (R padded to whole fragments with zeros); the shared product then runs
// as it does alone, and between its mainloop and its epilogue each wave adds
// T op(up_a) for its own rows to its accumulators (lora_expand), so D is
// written once and rounded once.  The second product costs 2 M R N operations
// beside 2 M K N.  T stays fp32 in memory; as bf16 MFMA operands it goes in
// as two terms, T = hi + lo with lo = bf16(T - hi), which keeps 16 of its
// bits: as one bf16 term its rounding (2^-9 of the low-rank part) would be as
// large as that of D itself.
#pragma once

#include "common.hpp"
#include "mfma_gemm.hpp"
#include "ragged.hpp"

namespace dg {

// T is padded to whole fragments of rank along k: LORA_PAD columns.
constexpr int LORA_PAD = 16;

// VEC consecutive k (from k) of column / row mn of a matrix stored with k
// contiguous (KC: element (mn, k) at mn*ld + k) or mn contiguous (at
// k*ld + mn); zero where k >= K or !ok.
template <typename T>
__device__ __forceinline__ u32x4 load_k_chunk(const T* x, int64_t ld, bool kc, int64_t mn, bool ok,
                                              int k, int K)
{
    constexpr int VEC = 16 / sizeof(T);
    if (kc && ok && k + VEC <= K) return *reinterpret_cast<const u32x4_elem<T>*>(x + mn * ld + k);
    T e[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j)
        e[j] = ok && k + j < K ? (kc ? x[mn * ld + k + j] : x[(int64_t)(k + j) * ld + mn]) : T(0);
    return pack_chunk<T>(e);
}

// fp32 values as MFMA operand terms: bf16 as hi + lo, fp32 as itself.  An
// infinite or NaN hi takes a zero lo, so an infinity stays one.
__device__ __forceinline__ void split_terms(const float (&t)[8], u32x4& hi, u32x4& lo)
{
    bf16x8 h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        h[e] = (__bf16)t[e];
        const float hf = (float)h[e];
        l[e] = (__bf16)(fabsf(hf) <= 3.402823466e38f ? t[e] - hf : 0.0f);
    }
    hi = __builtin_bit_cast(u32x4, h);
    lo = __builtin_bit_cast(u32x4, l);
}
__device__ __forceinline__ void split_terms(const float (&t)[4], u32x4& hi, u32x4&)
{
    hi = u32x4{__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]),
               __float_as_uint(t[3])};
}

// First segment that may hold row m0 or a later one: the number of segments
// that end at or before it (offsets do not decrease).
__device__ __forceinline__ int first_segment(const RaggedArgs& p, int m0, int lane)
{
    int s = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 64) {
        const uint64_t before = __ballot(g0 + lane < p.groups && p.offsets[g0 + lane + 1] <= m0);
        s += __builtin_popcountll(before);
        if (~before != 0) break;
    }
    return s;
}

// Adds T op(up_a) to the accumulators of a wave whose block starts at row m0
// and column n0 (MF x NF fragments of FM x FM; lane l holds row l % FM of
// each).  Segments are taken one after another; the product of a segment's
// adapter with the fragment's rows goes into a temporary, and only lanes whose
// row lies in the segment add it, so nothing an adapter holds (infinities,
// NaN) reaches another segment's rows.
template <int KIND, int MF, int NF, typename Acc>
__device__ __forceinline__ void lora_expand(const RaggedArgs& p, int m0, int n0, int lane,
                                            Acc (&acc)[MF][NF])
{
    using T = typename MfmaShape<KIND>::T;
    constexpr int FM = MfmaShape<KIND>::FM, ACC = MfmaShape<KIND>::ACC;
    constexpr int VEC = 16 / sizeof(T), KSTEP = 64 / FM * VEC;
    constexpr int NK = 4;  // fragment steps of rank held at once
    const int m_end = m0 + MF * FM < p.M ? m0 + MF * FM : p.M;
    if (m0 >= m_end || n0 >= p.N) return;
    const int kl = VEC * (lane / FM);
    for (int s = first_segment(p, m0, lane); s < p.groups; ++s) {
        int start, size;
        group_span(p, s, start, size);
        if (start >= m_end) break;
        const int end = start + size;
        const int a = p.ids ? p.ids[s] : s;
        if (size == 0 || end <= m0 || a < 0 || a >= p.adapters) continue;
        const T* up = static_cast<const T*>(p.up) + (int64_t)a * p.stride_up;
        for (int r0 = 0; r0 < p.rank; r0 += NK * KSTEP) {
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                const int rf = m0 + i * FM;  // the fragment's first row
                if (rf >= end || rf + FM <= start) continue;
                const int row = rf + lane % FM;
                const bool mine = row >= start && row < end;
                u32x4 hi[NK], lo[NK];
#pragma unroll
                for (int kk = 0; kk < NK; ++kk) {
                    const int k = r0 + kk * KSTEP + kl;
                    float t[VEC] = {};
                    if (mine && k < p.rank_pad) {
                        const float* src = p.t + (int64_t)row * p.rank_pad + k;
                        for (int sp = 0; sp < p.splits; ++sp, src += (int64_t)p.rows * p.rank_pad)
#pragma unroll
                            for (int v = 0; v < VEC / 4; ++v) {
                                const f32x4 q = reinterpret_cast<const f32x4*>(src)[v];
#pragma unroll
                                for (int e = 0; e < 4; ++e) t[4 * v + e] += q[e];
                            }
                    }
                    split_terms(t, hi[kk], lo[kk]);
                }
#pragma unroll
                for (int j = 0; j < NF; ++j) {
                    const int col = n0 + j * FM + lane % FM;
                    Acc tmp = {};
#pragma unroll
                    for (int kk = 0; kk < NK; ++kk) {
                        if (r0 + kk * KSTEP >= p.rank) break;
                        const u32x4 b = load_k_chunk<T>(up, p.ld_up, p.up_kc, col, col < p.N,
                                                        r0 + kk * KSTEP + kl, p.rank);
                        mfma_step<KIND>(b, hi[kk], tmp);
                        if constexpr (sizeof(T) == 2) mfma_step<KIND>(b, lo[kk], tmp);
                    }
                    if (mine)
#pragma unroll
                        for (int v = 0; v < ACC; ++v) acc[i][j][v] += tmp[v];
                }
            }
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

// T = s_a X op(down_a): one block of 16*RF rows of one segment per workgroup
// (blockIdx.x), a slice of K per blockIdx.y (its own partial sums of T) and
// 16*NF columns of rank per blockIdx.z.  The eight waves split the slice's K
// in runs of 4 chunk rows (256 contiguous bytes of each row of X and, where k
// is contiguous, of down), load fragments straight from memory into the MFMA
// lane layout and add their sums through LDS in wave order.
constexpr int SHRINK_WAVES = 8;
template <typename T, int RF, int NF, bool KC>
__global__ __launch_bounds__(64 * SHRINK_WAVES) void lora_shrink_kernel(
    RaggedArgs p, const void* down_v, int64_t ld_down, int64_t stride_down, int k_slice, float* t_out)
{
    constexpr int VEC = 16 / sizeof(T), KB = 4 * VEC, U = 4;
    RowTile t;
    if (!find_row_tile<16 * RF>(p, blockIdx.x, 1, t)) return;
    const int a = p.ids ? p.ids[t.group] : t.group;
    if (a < 0 || a >= p.adapters) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r0 = t.in_group * 16 * RF;  // first row within the segment
    const int c0 = blockIdx.z * 16 * NF;  // first column of rank
    const int k_lo = blockIdx.y * k_slice;
    const int k_hi = k_lo + k_slice < p.K ? k_lo + k_slice : p.K;
    const T* X = static_cast<const T*>(p.A) + (int64_t)t.start * p.lda;
    const T* down = static_cast<const T*>(down_v) + (int64_t)a * stride_down;
    f32x4 acc[RF][NF] = {};
    for (int kw = k_lo + wave * U * KB; kw < k_hi; kw += SHRINK_WAVES * U * KB) {
        u32x4 xa[U][RF], xb[U][NF];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = kw + u * KB + VEC * (lane / 16);
#pragma unroll
            for (int i = 0; i < RF; ++i) {
                const int row = r0 + i * 16 + lane % 16;
                xa[u][i] = load_k_chunk<T>(X, p.lda, true, row, row < t.size, k, k_hi);
            }
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                const int col = c0 + j * 16 + lane % 16;
                xb[u][j] = load_k_chunk<T>(down, ld_down, KC, col, col < p.rank, k, k_hi);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < RF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j) mfma16<T>(xa[u][i], xb[u][j], acc[i][j]);
    }
    __shared__ f32x4 part[SHRINK_WAVES][RF * NF][64];
#pragma unroll
    for (int i = 0; i < RF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) part[wave][i * NF + j][lane] = acc[i][j];
    __syncthreads();
    const float scale = p.scales ? p.scales[a] : 1.0f;
    float* out = t_out + (int64_t)blockIdx.y * p.rows * p.rank_pad;
    for (int f = wave; f < RF * NF; f += SHRINK_WAVES) {
        const int row = r0 + f / NF * 16 + lane % 16;
        const int col = c0 + f % NF * 16 + 4 * (lane / 16);
        if (row >= t.size || col >= p.rank_pad) continue;
        f32x4 sum = part[0][f][lane];
#pragma unroll
        for (int w = 1; w < SHRINK_WAVES; ++w) sum += part[w][f][lane];
        *reinterpret_cast<f32x4*>(out + (int64_t)(t.start + row) * p.rank_pad + col) = scale * sum;
    }
}

}  // namespace dg
