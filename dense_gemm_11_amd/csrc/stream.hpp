// Products of few rows with matrices that are read once: tiles of 16 to 64
// rows, for experts or requests with a handful of rows each.  Such a call is
// bound by the bytes of B, so the kernel is built around keeping them in
// flight rather than around reuse:
//
//  * one workgroup of eight waves per tile of 16*RF rows and 16*NF columns,
//    the waves splitting K into eight runs, so even a call of a few tiles has
//    every wave of a compute unit loading;
//  * operands go from memory straight into the registers of the 16x16 MFMA
//    layout, U fragment steps at a time in two batches (one loading while the
//    other is multiplied); nothing is staged, so no barrier is met until the
//    waves' sums are added;
//  * a k-contiguous B gives each lane 16 consecutive bytes along k; an
//    n-contiguous one NF consecutive columns of each of VEC rows of k, turned
//    into fragments of every NF-th column by byte permutes (for fp32 they
//    already are);
//  * rows past the group's and the ragged last columns are not masked on the
//    way in: the lane reads the group's last row again, and the last tile of
//    a row starts at column N - BN instead, and what is read twice is not
//    stored.  Only K's ragged end, and matrices smaller than a tile, take
//    element-wise loads.
//
// The eight sums are added through LDS in wave order, so results are
// reproducible, and rounded once.
#pragma once

#include "lora.hpp"
#include "ragged.hpp"

namespace dg {

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

// RF x NF fragments of 16x16, U fragment steps of K per batch.
template <typename T_, bool KC_, int RF_, int NF_, int U_>
struct StreamConfig {
    using T = T_;
    static constexpr bool KC = KC_;
    static constexpr int RF = RF_, NF = NF_, U = U_;
    static constexpr int WAVES = 8, THREADS = 64 * WAVES;
    static constexpr int ES = sizeof(T), VEC = 16 / ES, KSTEP = 4 * VEC;
    static constexpr int BM = 16 * RF, BN = 16 * NF;
    // rows of fragments whose sums are exchanged at once (64 KiB of LDS at most)
    static constexpr int PF = RF * NF <= 8 ? RF : 8 / NF;
    static constexpr int PASSES = RF / PF;
    static constexpr int SLOTS = PF * NF;               // 16x16 blocks per pass
    static constexpr int ITEMS = SLOTS * 64;            // 16-byte pieces of them
    static constexpr int IPT = (ITEMS + THREADS - 1) / THREADS;
    static_assert(RF % PF == 0 && NF <= 8, "exchange");
    static_assert(KC || NF * ES >= 4, "an n-contiguous row piece of at least 4 bytes");
    // Column within the tile of fragment j's column c.
    __device__ static constexpr int column(int j, int c) { return KC ? j * 16 + c : NF * c + j; }
    // Slot q of lane l holds four adjacent columns of row l % 16, from this one:
    // a lane's accumulators cover columns column(j, 4 (l / 16) + v).
    __device__ static constexpr int slot_column(int q, int l)
    {
        return KC ? q * 16 + 4 * (l / 16) : 4 * NF * (l / 16) + 4 * q;
    }
};

// One batch of operand registers.
template <class S>
struct StreamBatch {
    u32x4 a[S::U][S::RF];
    uint32_t b[S::U][S::NF * 4];
};

// Fragment j of step u of a batch as the MFMA operand.
template <class S>
__device__ __forceinline__ u32x4 stream_b(const StreamBatch<S>& x, int u, int j)
{
    u32x4 r;
    if constexpr (S::KC) {
#pragma unroll
        for (int q = 0; q < 4; ++q) r[q] = x.b[u][4 * j + q];
    } else if constexpr (S::ES == 4) {   // row k: words NF*k .. of the columns
#pragma unroll
        for (int q = 0; q < 4; ++q) r[q] = x.b[u][S::NF * q + j];
    } else {                             // row k: words NF/2*k .., two columns each
        constexpr int W = S::NF / 2;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            r[q] = __builtin_amdgcn_perm(x.b[u][W * (2 * q + 1) + j / 2], x.b[u][W * (2 * q) + j / 2],
                                         j % 2 ? 0x07060302u : 0x05040100u);
    }
    return r;
}

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

// t[0..8) . up[0..8) of four adjacent columns from `col`, added to sum: ranks
// r .. r+7 of adapter `up` (clamped to the matrix; ranks past the last add
// nothing).
template <typename T>
__device__ __forceinline__ void lora_dot8(const RaggedArgs& p, const T* up, int col, int r,
                                          const float (&t)[8], f32x4& sum)
{
    T u[4][8];
    const bool whole = r + 8 <= p.rank;
    if (p.up_kc) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const T* row = up + (int64_t)(col + s < p.N ? col + s : p.N - 1) * p.ld_up;
            if (whole) {
#pragma unroll
                for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
                    constexpr int VEC = 16 / sizeof(T);
                    const u32x4 c = *reinterpret_cast<const u32x4_elem<T>*>(row + r + h * VEC);
                    T e[VEC];
                    __builtin_memcpy(e, &c, 16);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) u[s][h * VEC + v] = e[v];
                }
            } else {
#pragma unroll
                for (int v = 0; v < 8; ++v) u[s][v] = row[r + v < p.rank ? r + v : p.rank - 1];
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            const T* row = up + (int64_t)(r + v < p.rank ? r + v : p.rank - 1) * p.ld_up;
            if (col + 4 <= p.N) {
                const typename RawLoad<4 * sizeof(T)>::T c =
                    *reinterpret_cast<const typename RawLoad<4 * sizeof(T)>::T*>(row + col);
                T e[4];
                __builtin_memcpy(e, &c, 4 * sizeof(T));
#pragma unroll
                for (int s = 0; s < 4; ++s) u[s][v] = e[s];
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s) u[s][v] = row[col + s < p.N ? col + s : p.N - 1];
            }
        }
    }
#pragma unroll
    for (int v = 0; v < 8; ++v)
        if (r + v < p.rank)
#pragma unroll
            for (int s = 0; s < 4; ++s) sum[s] += t[v] * to_f32(u[s][v]);
}

// T op(up_a) of row `row`, four columns from `col`, in fp32 (T is not
// rounded on this path).
template <typename T>
__device__ __forceinline__ f32x4 lora_row(const RaggedArgs& p, int row, int col, int a)
{
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    const T* up = static_cast<const T*>(p.up) + (int64_t)a * p.stride_up;
    const float* src = p.t + (int64_t)row * p.rank_pad;
    for (int r = 0; r < p.rank; r += 8) {
        float t[8] = {};
        for (int sp = 0; sp < p.splits; ++sp) {
            const f32x4* q =
                reinterpret_cast<const f32x4*>(src + (int64_t)sp * p.rows * p.rank_pad + r);
            const f32x4 q0 = q[0], q1 = q[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                t[e] += q0[e];
                t[4 + e] += q1[e];
            }
        }
        lora_dot8<T>(p, up, col, r, t, sum);
    }
    return sum;
}

template <class S, typename OutT, int RAG>
__global__ __launch_bounds__(S::THREADS) void stream_kernel(RaggedArgs p)
{
    using T = typename S::T;
    constexpr int RF = S::RF, NF = S::NF, U = S::U, KSTEP = S::KSTEP, VEC = S::VEC, ES = S::ES;
    __shared__ f32x4 part[S::WAVES][S::SLOTS][64];
    __shared__ int adapter[RAG == RAG_LORA ? S::BM : 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn, start = 0, size = p.M, g = 0;
    if constexpr (RAG == RAG_ROWS) {
        RowTile t;
        if (!find_row_tile<S::BM>(p, blockIdx.x, p.tiles_n, t)) return;
        g = t.group;
        start = t.start;
        size = t.size;
        p.tiles_m = t.tiles_m;
        tile_of(p, t.in_group, tm, tn);
        if (p.scales) p.alpha *= p.scales[g];
    } else {
        tile_coords(p, tm, tn);
    }
    const int r0 = tm * S::BM, n0 = tn * S::BN;  // r0 within the group
    // the last tile of a row moves back to end at column N
    const int nb = n0 + S::BN <= p.N ? n0 : (p.N >= S::BN ? p.N - S::BN : 0);
    const T* A = static_cast<const T*>(p.A) + (int64_t)(start + r0) * p.lda;
    const T* B = static_cast<const T*>(p.B) + (int64_t)g * p.stride_b +
                 (S::KC ? (int64_t)nb * p.ldb : nb);
    const int rows = size - r0;  // of the group, from the tile's first

    f32x4 acc[RF][NF] = {};
    auto multiply = [&](const StreamBatch<S>& x, int u) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const u32x4 b = stream_b<S>(x, u, j);
#pragma unroll
            for (int i = 0; i < RF; ++i) mfma16<T>(x.a[u][i], b, acc[i][j]);
        }
    };
    auto arow = [&](int i) { const int r = i * 16 + lane % 16; return r < rows ? r : rows - 1; };
    // whole fragment steps of K, split evenly over the waves
    const bool narrow = p.N < S::BN;
    const int steps = narrow ? 0 : p.K / KSTEP;
    uint32_t off_a[RF], off_b[S::KC ? NF : 1];
#pragma unroll
    for (int i = 0; i < RF; ++i)
        off_a[i] = (uint32_t)(((int64_t)arow(i) * p.lda + VEC * (lane / 16)) * ES);
    if constexpr (S::KC) {
#pragma unroll
        for (int j = 0; j < NF; ++j)
            off_b[j] = (uint32_t)(((int64_t)(j * 16 + lane % 16) * p.ldb + VEC * (lane / 16)) * ES);
    } else {
        off_b[0] = (uint32_t)(((int64_t)VEC * (lane / 16) * p.ldb + NF * (lane % 16)) * ES);
    }
    auto load = [&](StreamBatch<S>& x, int u, int step) __attribute__((always_inline)) {
        const int k = step * KSTEP;
        const char* a = reinterpret_cast<const char*>(A + k);
#pragma unroll
        for (int i = 0; i < RF; ++i)
            x.a[u][i] = *reinterpret_cast<const u32x4_elem<T>*>(a + off_a[i]);
        if constexpr (S::KC) {
            const char* b = reinterpret_cast<const char*>(B + k);
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                const u32x4 v = *reinterpret_cast<const u32x4_elem<T>*>(b + off_b[j]);
#pragma unroll
                for (int q = 0; q < 4; ++q) x.b[u][4 * j + q] = v[q];
            }
        } else {
            constexpr int W = NF * ES / 4, PW = W > 4 ? 4 : W;  // words per row of k, per load
            using V = typename RawLoad<4 * PW>::T;
#pragma unroll
            for (int r = 0; r < VEC; ++r) {
                const char* b = reinterpret_cast<const char*>(B + (int64_t)(k + r) * p.ldb);
#pragma unroll
                for (int h = 0; h < W / PW; ++h) {
                    const V v = *reinterpret_cast<const V*>(b + off_b[0] + h * 16);
#pragma unroll
                    for (int q = 0; q < PW; ++q) x.b[u][W * r + PW * h + q] = v[q];
                }
            }
        }
    };
    const int s_lo = (int)((int64_t)steps * wave / S::WAVES);
    const int s_hi = (int)((int64_t)steps * (wave + 1) / S::WAVES);
    const int batches = (s_hi - s_lo) / U, rest = (s_hi - s_lo) % U;
    StreamBatch<S> x0, x1;
    // the steps that fill no batch first, with the first batch behind them
    int s = s_lo + rest;
    static_for<U - 1>([&](auto u) __attribute__((always_inline)) {
        if (decltype(u)::value < rest) load(x1, decltype(u)::value, s_lo + decltype(u)::value);
    });
    if (batches > 0)
        static_for<U>([&](auto u) __attribute__((always_inline)) {
            load(x0, decltype(u)::value, s + decltype(u)::value);
        });

    // the low-rank part of this thread's outputs, while the batches load
    f32x4 low[RAG == RAG_LORA ? S::PASSES * S::IPT : 1];
    if constexpr (RAG == RAG_LORA) {
        for (int r = tid; r < S::BM; r += S::THREADS) adapter[r] = -1;
        __syncthreads();
        for (int sg = tid; sg < p.groups; sg += S::THREADS) {
            int lo, n;
            group_span(p, sg, lo, n);
            const int hi = lo + n < r0 + S::BM ? lo + n : r0 + S::BM;
            const int a = p.ids ? p.ids[sg] : sg;
            if (a >= 0 && a < p.adapters)
                for (int r = lo > r0 ? lo : r0; r < hi; ++r) adapter[r - r0] = a;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < S::PASSES * S::IPT; ++q) {
            const int item = tid + (q % S::IPT) * S::THREADS, slot = item / 64, l = item & 63;
            const int row = ((q / S::IPT) * S::PF + slot / NF) * 16 + l % 16;
            const int col = nb + S::slot_column(slot % NF, l);
            low[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (item < S::ITEMS && row < rows && col < p.N && adapter[row] >= 0)
                low[q] = lora_row<T>(p, r0 + row, col, adapter[row]);
        }
    }

    static_for<U - 1>([&](auto u) __attribute__((always_inline)) {
        if (decltype(u)::value < rest) multiply(x1, decltype(u)::value);
    });
    auto turn = [&](StreamBatch<S>& next, const StreamBatch<S>& cur, bool more)
                    __attribute__((always_inline)) {
        s += U;
        if (more)
            static_for<U>([&](auto u) __attribute__((always_inline)) {
                load(next, decltype(u)::value, s + decltype(u)::value);
            });
        static_for<U>([&](auto u) __attribute__((always_inline)) {
            multiply(cur, decltype(u)::value);
        });
    };
    int b = 0;
    for (; b + 2 <= batches; b += 2) {
        turn(x1, x0, true);
        turn(x0, x1, b + 2 < batches);
    }
    if (b < batches) turn(x1, x0, false);
    // K's ragged end, and every step of a matrix narrower than the tile
    const int all = (p.K + KSTEP - 1) / KSTEP;
    for (int t = steps + (S::WAVES - 1 - wave); t < all; t += S::WAVES) {
        const int k = t * KSTEP + VEC * (lane / 16);
        u32x4 fa[RF];
#pragma unroll
        for (int i = 0; i < RF; ++i)
            fa[i] = clamped_chunk<T>(A + (int64_t)arow(i) * p.lda, 1, k, p.K);
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            int c = S::column(j, lane % 16);
            if (nb + c >= p.N) c = p.N - 1 - nb;
            const u32x4 fb = clamped_chunk<T>(B + (S::KC ? (int64_t)c * p.ldb : c),
                                              S::KC ? 1 : p.ldb, k, p.K);
#pragma unroll
            for (int i = 0; i < RF; ++i) mfma16<T>(fa[i], fb, acc[i][j]);
        }
    }

    // add the waves' sums, PF rows of fragments at a time
    static_for<S::PASSES>([&](auto pass_c) __attribute__((always_inline)) {
        constexpr int pass = decltype(pass_c)::value;
        if constexpr (pass > 0) __syncthreads();
        static_for<S::SLOTS>([&](auto q_c) __attribute__((always_inline)) {
            constexpr int slot = decltype(q_c)::value, i = pass * S::PF + slot / NF, q = slot % NF;
            f32x4 v;
            if constexpr (S::KC) v = acc[i][q];
            else
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][(4 * q + e) % NF][(4 * q + e) / NF];
            part[wave][slot][lane] = v;
        });
        __syncthreads();
#pragma unroll
        for (int h = 0; h < S::IPT; ++h) {
            const int item = tid + h * S::THREADS, slot = item / 64, l = item & 63;
            if (item >= S::ITEMS) break;
            const int row = (pass * S::PF + slot / NF) * 16 + l % 16;
            const int col = nb + S::slot_column(slot % NF, l);
            if (row >= rows || col >= p.N) continue;
            f32x4 v = part[0][slot][l];
#pragma unroll
            for (int w = 1; w < S::WAVES; ++w) v += part[w][slot][l];
            if constexpr (RAG == RAG_LORA) v += low[pass * S::IPT + h];
            v *= p.alpha;
            const int64_t at = start + r0 + row;
            OutT* d = reinterpret_cast<OutT*>(p.D) + at * p.ldd + col;
            const OutT* c = reinterpret_cast<const OutT*>(p.C) + at * p.ldc + col;
            if (col >= n0 && col + 4 <= p.N) {
                if (p.beta != 0.0f) {
                    OutT e[4];
                    const typename RawLoad<4 * sizeof(OutT)>::T w =
                        *reinterpret_cast<const typename RawLoad<4 * sizeof(OutT)>::T*>(c);
                    __builtin_memcpy(e, &w, sizeof(e));
#pragma unroll
                    for (int s4 = 0; s4 < 4; ++s4) v[s4] += p.beta * to_f32(e[s4]);
                }
                OutT e[4];
#pragma unroll
                for (int s4 = 0; s4 < 4; ++s4) e[s4] = from_f32<OutT>(v[s4]);
                typename RawLoad<4 * sizeof(OutT)>::T w;
                __builtin_memcpy(&w, e, sizeof(e));
                *reinterpret_cast<typename RawLoad<4 * sizeof(OutT)>::T*>(d) = w;
            } else {
#pragma unroll
                for (int s4 = 0; s4 < 4; ++s4) {
                    if (col + s4 < n0 || col + s4 >= p.N) continue;
                    float o = v[s4];
                    if (p.beta != 0.0f) o += p.beta * to_f32(c[s4]);
                    d[s4] = from_f32<OutT>(o);
                }
            }
        }
    });
}

}  // namespace dg
