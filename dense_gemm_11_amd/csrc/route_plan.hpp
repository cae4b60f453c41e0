// The launches behind a routing's (route.hpp): the plan from the experts' counts,
// and the gradient.
#pragma once

#include "act.hpp"
#include "route.hpp"

namespace dg {

// The counts of chunks [lo, hi), four experts to a thread, added to n[] where
// the chunk is below `below` and to all[].
__device__ __forceinline__ void add_counts(const RouteArgs& p, int lo, int hi, int below, int* n, int* all)
{
    // (with few experts no more than 16 parts: they meet in one sum each)
    const int quads = p.count_ld / 4, segs = quads > 64 ? 1024 / quads : 16;
    const int q = threadIdx.x % quads, seg = threadIdx.x / quads;
    if (seg >= segs) return;
    // even and odd bytes as 16-bit sums: at most ROUTE_SUPER * ROUTE_CHUNK each
    static_assert(ROUTE_SUPER * ROUTE_CHUNK < 65536, "16-bit sums");
    uint32_t b0 = 0, b1 = 0, a0 = 0, a1 = 0;
    const uint32_t* c = reinterpret_cast<const uint32_t*>(p.counts) + q;
#pragma unroll 8
    for (int i = lo + seg; i < hi; i += segs) {
        const uint32_t v = c[(int64_t)i * quads], even = v & 0xFF00FFu, odd = (v >> 8) & 0xFF00FFu;
        a0 += even;
        a1 += odd;
        b0 += i < below ? even : 0;
        b1 += i < below ? odd : 0;
    }
    const uint32_t b[2] = {b0, b1}, a[2] = {a0, a1};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int e = 4 * q + s;
        if (e >= p.experts) break;
        if (n) atomicAdd(&n[e], (int)(b[s & 1] >> (16 * (s >> 1)) & 0xFFFFu));
        if (all) atomicAdd(&all[e], (int)(a[s & 1] >> (16 * (s >> 1)) & 0xFFFFu));
    }
}

// Sums of ROUTE_SUPER chunks' counts.
__global__ __launch_bounds__(1024) void route_super(RouteArgs p)
{
    __shared__ int all[ROUTE_MAX_EXPERTS];
    for (int e = threadIdx.x; e < p.experts; e += 1024) all[e] = 0;
    __syncthreads();
    const int lo = blockIdx.x * ROUTE_SUPER, hi = lo + ROUTE_SUPER;
    add_counts(p, lo, hi < p.chunks ? hi : p.chunks, 0, nullptr, all);
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += 1024)
        p.supers[(int64_t)blockIdx.x * p.experts + e] = all[e];
}

// The plan, a chunk per workgroup.  Where its rows begin follows from the counts
// of the chunks before it and of all chunks, which every workgroup adds up for
// itself (a byte per expert and chunk: 64 KiB from L2 for 16384 tokens of 256
// experts, 6 us in all) rather than wait for a launch that does.
__global__ __launch_bounds__(1024) void route_place(RouteArgs p)
{
    __shared__ ChosenBits bits;
    __shared__ int start[ROUTE_MAX_EXPERTS], all[ROUTE_MAX_EXPERTS];
    __shared__ int wave_sum[16], total;
    const int b = blockIdx.x, t0 = b * p.chunk;
    const int tokens = p.tokens - t0 < p.chunk ? p.tokens - t0 : p.chunk;
    // the chunk's assignments, up to two to a thread, asked for before all else
    constexpr int OWN = ROUTE_CHUNK * ROUTE_MAX_TOP / 1024;
    int own[OWN];
#pragma unroll
    for (int q = 0; q < OWN; ++q) {
        const int i = threadIdx.x + 1024 * q;
        own[q] = i < tokens * p.top ? p.ids[(int64_t)t0 * p.top + i] : -1;
    }
    clear_bits(bits, p.experts);
    for (int e = threadIdx.x; e < p.experts; e += 1024) start[e] = all[e] = 0;
    __syncthreads();
    const int super = b / ROUTE_SUPER, supers = (p.chunks + ROUTE_SUPER - 1) / ROUTE_SUPER;
    if (supers == 1) {
        add_counts(p, 0, p.chunks, b, start, all);
    } else {
        add_counts(p, super * ROUTE_SUPER, b, b, start, nullptr);
        const int segs = p.experts > 512 ? 1 : 1024 / p.experts;
        const int e = threadIdx.x % p.experts, seg = threadIdx.x / p.experts;
        if (seg < segs) {
            int before = 0, sum = 0;
            for (int s = seg; s < supers; s += segs) {
                const int n = p.supers[(int64_t)s * p.experts + e];
                sum += n;
                before += s < super ? n : 0;
            }
            atomicAdd(&start[e], before);
            atomicAdd(&all[e], sum);
        }
    }
#pragma unroll
    for (int q = 0; q < OWN; ++q) {
        const int t = ((int)threadIdx.x + 1024 * q) / p.top;
        if (own[q] >= 0) atomicOr(&bits.w[own[q]][t >> 5], 1u << (t & 31));
    }
    __syncthreads();
    scan_experts(all, p.experts, wave_sum, &total);
    for (int e = threadIdx.x; e < p.experts; e += 1024) start[e] += all[e];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < OWN; ++q) {
        const int i = threadIdx.x + 1024 * q;
        if (i < tokens * p.top) place_row(p, t0, i, own[q], bits, start);
    }
    if (b == 0)
        for (int e = threadIdx.x; e <= p.experts; e += 1024)
            p.offsets[e] = e < p.experts ? all[e] : total;
    for (int64_t r = (int64_t)total + b * 1024 + threadIdx.x; r < (int64_t)p.tokens * p.top;
         r += (int64_t)gridDim.x * 1024)
        p.order[r] = -1;
}

// The weights' gradient carried back to the logits, L lanes to a token:
//   softmax          dx_e = scale p_e (g_e - sum_j g_j p_j)
//   ... renormalised dx_j = scale q_j (g_j - sum_l g_l q_l), q_j = p_j / sum_l p_l
//   sigmoid          dx_j = scale s_j (1 - s_j) g_j
//   ... renormalised dx_j = scale q_j (1 - s_j) (g_j - sum_l g_l q_l)
// with g_e = 0 for experts that were not chosen.  What the chosen get goes
// through LDS to the lanes that write the row, NQ quads of neighbouring experts
// each.  DENSE, the first form, needs every logit, which its lanes hold (read three
// times over instead, 16384 rows of 256 fp32 took 14.9 us; 8.3).  Bound by reading
// and writing the logits, of the other forms only by writing.
struct RouteGradArgs {
    const void* logits;
    const int32_t* ids;
    const float* dweights;
    void* dlogits;
    int64_t ld, ldd;
    int tokens, experts, top, row;  // row: experts padded to whole quads
    int sigmoid, renormalize;
    float scale;
};

template <typename X, int L, int NQ, bool DENSE>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs p)
{
    extern __shared__ f32x4 quads[];  // a row of experts per token
    const int lane = threadIdx.x & 63, sub = lane & (L - 1), slot = threadIdx.x / L;
    const int t = blockIdx.x * (256 / L) + slot;
    if (t >= p.tokens) return;  // (no exchange below leaves a token's L lanes)
    const X* row = static_cast<const X*>(p.logits) + (int64_t)t * p.ld;
    X* out = static_cast<X*>(p.dlogits) + (int64_t)t * p.ldd;
    f32x4* mine = quads + slot * (p.row / 4);
    const float low = -__builtin_inff();
    float x[DENSE ? NQ : 1][4];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int e = 4 * (sub + i * L);
        if (e < p.experts) mine[e / 4] = f32x4{};
        if constexpr (DENSE) {
            load_part<4>(x[i], row + (e < p.experts ? e : 0), e + 4 <= p.experts ? 4 : p.experts - e, low);
#pragma unroll
            for (int q = 0; q < 4; ++q) x[i][q] = fmaxf(x[i][q], low);  // a NaN is as -inf
        }
    }
    const int e = sub < p.top ? p.ids[(int64_t)t * p.top + sub] : -1;
    const bool live = e >= 0 && e < p.experts;
    const float xe = live ? fmaxf(to_f32(row[e]), low) : low;
    const float g = live ? p.dweights[(int64_t)t * p.top + sub] : 0.0f;
    float m = xe, total = 1.0f;
    if constexpr (DENSE) {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) m = fmaxf(m, x[i][q]);
    }
    m = lanes_max<L>(m);
    if constexpr (DENSE) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                x[i][q] = x[i][q] > low ? quick_exp_below(x[i][q], m) : 0.0f;
                s += x[i][q];
            }
        total = lanes_sum<L>(s);
    }
    // p_j, or in proportion to it (chosen_score), and q_j
    float q = xe > low ? quick_exp_below(xe, m) : 0.0f, rest = 1.0f;
    if (p.sigmoid && xe > low) {
        const float tail = quick_exp(-fabsf(xe));
        const float up = __builtin_amdgcn_rcpf(1.0f + tail), dn = tail * up;  // the larger of s and 1 - s
        rest = xe > 0.0f ? dn : up;
        q = xe > 0.0f ? up : p.renormalize ? quick_exp(xe - fminf(m, 0.0f)) * up : dn;
    }
    if (p.renormalize) total = lanes_sum<L>(q);
    const float share = total > 0.0f ? __builtin_amdgcn_rcpf(total) : 0.0f;
    q *= share;
    const float mean = DENSE || p.renormalize ? lanes_sum<L>(q * g) : 0.0f;
    const float d = p.scale * q * rest * (p.renormalize ? g - mean : g);
    // an expert named more than once gets the sum
    float sum = 0.0f;
    for (int j = 0; j < p.top; ++j) {
        const int from = (lane & ~(L - 1)) + j;
        const int ej = __shfl(live ? e : -1, from);
        const float dj = __shfl(d, from);
        sum += live && ej == e ? dj : 0.0f;
    }
    wave_sync();
    if (live) reinterpret_cast<float*>(mine)[e] = sum;
    wave_sync();
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int at = 4 * (sub + i * L);
        if (at >= p.experts) break;
        f32x4 v = mine[at / 4];
        if constexpr (DENSE)
#pragma unroll
            for (int s = 0; s < 4; ++s) v[s] -= p.scale * (x[i][s] * share) * mean;
        store_four(out + at, v, p.experts - at);
    }
}

}  // namespace dg
