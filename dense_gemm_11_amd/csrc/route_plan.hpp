// The launches behind a routing's (route.hpp): the plan from the experts' counts,
// and the gradient.
#pragma once

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
// experts) rather than wait for a launch that does.
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
// through LDS to the lanes that write the row.  Bound by reading and writing the
// logits (only writing where nothing but the chosen count).
struct RouteGradArgs {
    const void* logits;
    const int32_t* ids;
    const float* dweights;
    void* dlogits;
    int64_t ld, ldd;
    int tokens, experts, top;
    int sigmoid, renormalize;
    float scale;
};

template <typename X, int L>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs p)
{
    extern __shared__ float chosen[];  // a row of experts per token
    const int lane = threadIdx.x & 63, sub = lane & (L - 1), slot = threadIdx.x / L;
    const int t = blockIdx.x * (256 / L) + slot;
    if (t >= p.tokens) return;  // (whole waves are not needed: nothing below crosses the L lanes)
    const X* row = static_cast<const X*>(p.logits) + (int64_t)t * p.ld;
    X* out = static_cast<X*>(p.dlogits) + (int64_t)t * p.ldd;
    float* mine = chosen + slot * p.experts;
    const int E = p.experts;
    for (int e = sub; e < E; e += L) mine[e] = 0.0f;
    const bool dense = !p.sigmoid && !p.renormalize;
    const float low = -__builtin_inff();
    const int e = sub < p.top ? p.ids[(int64_t)t * p.top + sub] : -1;
    const bool live = e >= 0 && e < E;
    float x = live ? to_f32(row[e]) : low;
    x = x > low ? x : low;
    float g = live ? p.dweights[(int64_t)t * p.top + sub] : 0.0f;
    float m, total = 1.0f;
    if (dense) {
        m = low;
        for (int i = sub; i < E; i += L) m = fmaxf(m, to_f32(row[i]));
        m = lanes_max<L>(m);
        float s = 0.0f;
        for (int i = sub; i < E; i += L) {
            const float v = to_f32(row[i]);
            s += v > low ? exp_below(v, m) : 0.0f;
        }
        total = lanes_sum<L>(s);
        total = total > 0.0f ? total : 1.0f;
    } else {
        m = lanes_max<L>(x);
    }
    // p_j, or in proportion to it (chosen_score), and q_j
    float q = x > low ? exp_below(x, p.sigmoid ? fminf(m, 0.0f) : m) : 0.0f, rest = 1.0f;
    if (p.sigmoid && x > low) {
        const float up = 1.0f / (1.0f + expf(-fabsf(x)));  // the larger of s and 1 - s
        const float dn = expf(-fabsf(x)) * up;
        rest = x > 0.0f ? dn : up;
        q = x > 0.0f ? up : p.renormalize ? expf(x - fminf(m, 0.0f)) * up : dn;
    }
    if (p.renormalize) {
        total = lanes_sum<L>(q);
        total = total > 0.0f ? total : 1.0f;
    }
    q /= total;
    const float mean = p.renormalize || dense ? lanes_sum<L>(q * g) : 0.0f;
    float d = p.scale * q * rest * (p.renormalize ? g - mean : g);
    // an expert named more than once gets the sum
    float sum = 0.0f;
    for (int j = 0; j < p.top; ++j) {
        const int from = (lane & ~(L - 1)) + j;
        const int ej = __shfl(live ? e : -1, from);
        const float dj = __shfl(d, from);
        sum += live && ej == e ? dj : 0.0f;
    }
    wave_sync();
    if (live) mine[e] = sum;
    wave_sync();
    for (int i = sub; i < E; i += L) {
        float v = mine[i];
        if (dense) {
            const float xi = to_f32(row[i]);
            if (xi > low) v -= p.scale * (exp_below(xi, m) / total) * mean;
        }
        out[i] = from_f32<X>(v);
    }
}

}  // namespace dg
