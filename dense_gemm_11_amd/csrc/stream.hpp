// Products of few rows with matrices that are read once: tiles of 16 to 64
// rows, for experts or requests with a handful of rows each.  Such a call is
// bound by the bytes of B, so the kernel is built around keeping them in
// flight rather than around reuse:
//
//  * one workgroup of eight waves per tile of 16*RF rows and 16*NF columns,
//    the waves splitting K into eight runs, so even a call of a few tiles has
//    every wave of a compute unit loading;
//  * operands go from memory straight into registers, four fragment steps of
//    K at a time and, where the registers hold them, two such batches in flight; nothing is staged, so no
//    barrier is met until the waves' sums are added;
//  * the memory pipeline looks up the lines of four consecutive lanes at a
//    time, so a k-contiguous operand is not read in the MFMA's lane order (16
//    rows side by side: a line per lane; 64 rows of a 4096x4096 product took
//    24 us) but 64 bytes of one row per four lanes, 256 of each of four rows
//    per load, and four loads are then transposed within each four lanes
//    (quad_turn);
//  * an n-contiguous B gives each lane NF consecutive columns of each of VEC
//    rows of k, turned into fragments of every NF-th column by byte permutes
//    (for fp32 they already are);
//  * rows past the group's and columns past N are not masked on the way in:
//    the lane reads the last row or column again (the last tile of an
//    n-contiguous B starts at column N - BN instead), and what is read twice
//    is not stored.  Only K's ragged end, and an n-contiguous B narrower than
//    a tile and of no multiple of NF columns, take element-wise loads.
//
// The eight sums are added through LDS in wave order, so results are
// reproducible, and rounded once.
//
// RAG_SHRINK forms the adapters' first product, T = s_a X op(down_a): the row
// groups are the segments, B is their adapter's matrix and N its rank.
// blockIdx.y takes a slice of K each, whose sums go to a part of T of their
// own.  RAG_LORA_ONE is RAG_LORA that forms its rows' T itself: every
// workgroup reads the adapters' down again (from L2), which for one tile of
// rows and one or two adapters costs less than a launch and T's way through
// memory (one token, 2048x2048, rank 8: 12.6 -> 10.31 us).
#pragma once

#include "lora.hpp"
#include "ragged.hpp"

namespace dg {

// RF x NF fragments of 16x16.
template <typename T_, bool KC_, int RF_, int NF_>
struct StreamConfig {
    using T = T_;
    static constexpr bool KC = KC_;
    static constexpr int RF = RF_, NF = NF_;
    static constexpr int WAVES = 8, THREADS = 64 * WAVES;
    static constexpr int ES = sizeof(T), VEC = 16 / ES, KSTEP = 4 * VEC;
    static constexpr int BM = 16 * RF, BN = 16 * NF;
    // rows of fragments whose sums are exchanged at once (64 KiB of LDS at most)
    static constexpr int PF = RF * NF <= 8 ? RF : 8 / NF;
    static constexpr int PASSES = RF / PF;
    static constexpr int SLOTS = PF * NF;               // 16x16 blocks per pass
    static constexpr int ITEMS = SLOTS * 64;            // 16-byte pieces of them
    static constexpr int IPT = (ITEMS + THREADS - 1) / THREADS;
    // a second batch in flight where the registers hold it
    static constexpr bool TWO = (RF + NF) * 36 - (KC ? 0 : 4 * NF) + 4 * RF * NF < 240;
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

// Four fragment steps of operand registers.  Step j of lane group g = lane / 16
// covers the VEC k from VEC * (4 g + j) of the batch's 4 KSTEP: any assignment
// serves that is the same for both operands, and with this one the chunks of
// four consecutive lanes are consecutive in memory.
template <class S>
struct StreamBatch {
    u32x4 a[S::RF][4];
    u32x4 b[S::KC ? S::NF : 1][4];                       // k-contiguous B
    uint32_t r[S::KC ? 1 : 4][S::KC ? 1 : S::NF * 4];    // rows of the other
};

// x[s] of lane 4 q + j to x[j] of lane 4 q + s, for every q: two rounds of
// exchanges between register and lane numbers that differ in one bit.
__device__ __forceinline__ void quad_turn(u32x4 (&x)[4], int lane)
{
    const bool odd = lane & 1, high = lane & 2;
    auto swap = [](u32x4& lo, u32x4& hi, bool upper, auto perm) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t l = lo[e], h = hi[e];
            const uint32_t from_h = __builtin_amdgcn_mov_dpp(h, decltype(perm)::value, 0xf, 0xf, true);
            const uint32_t from_l = __builtin_amdgcn_mov_dpp(l, decltype(perm)::value, 0xf, 0xf, true);
            lo[e] = upper ? from_h : l;
            hi[e] = upper ? h : from_l;
        }
    };
    using X1 = std::integral_constant<int, 0xB1>;  // quad_perm 1, 0, 3, 2
    using X2 = std::integral_constant<int, 0x4E>;  // quad_perm 2, 3, 0, 1
    swap(x[0], x[1], odd, X1{});
    swap(x[2], x[3], odd, X1{});
    swap(x[0], x[2], high, X2{});
    swap(x[1], x[3], high, X2{});
}

// Fragment j of the rows of k in r as the MFMA operand.
template <class S>
__device__ __forceinline__ u32x4 rows_fragment(const uint32_t (&x)[S::NF * 4], int j)
{
    u32x4 r;
    if constexpr (S::ES == 4) {          // row k: words NF*k .. of the columns
#pragma unroll
        for (int q = 0; q < 4; ++q) r[q] = x[S::NF * q + j];
    } else {                             // row k: words NF/2*k .., two columns each
        constexpr int W = S::NF / 2;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            r[q] = __builtin_amdgcn_perm(x[W * (2 * q + 1) + j / 2], x[W * (2 * q) + j / 2],
                                         j % 2 ? 0x07060302u : 0x05040100u);
    }
    return r;
}

// This wave's part of a tile's product, added to acc: `rows` rows of A (at least
// one) and `cols` columns of B, from the tile's first, by all of K.  meanwhile()
// runs once, while the first loads are under way.
template <class S, class F>
__device__ __forceinline__ void stream_product(const typename S::T* A, int64_t lda, int rows,
                                               const typename S::T* B, int64_t ldb, int cols, int K,
                                               int wave, int lane, f32x4 (&acc)[S::RF][S::NF],
                                               F meanwhile)
{
    using T = typename S::T;
    constexpr int RF = S::RF, NF = S::NF, KSTEP = S::KSTEP, VEC = S::VEC, ES = S::ES;
    // the row (of A, or of a k-contiguous B) and chunk of 16 bytes that load t of
    // a batch takes within a fragment of 16 rows
    const int q_row = 4 * ((lane >> 2) & 3), q_chunk = 4 * (lane >> 4) + (lane & 3);
    auto last = [](int r, int n) { return r < n ? r : n - 1; };
    uint32_t off_a[RF][4], off_b[S::KC ? NF : 1][4];
#pragma unroll
    for (int i = 0; i < RF; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
            off_a[i][t] = (uint32_t)(((int64_t)last(i * 16 + q_row + t, rows) * lda + VEC * q_chunk) * ES);
    if constexpr (S::KC) {
#pragma unroll
        for (int j = 0; j < NF; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                off_b[j][t] = (uint32_t)(((int64_t)last(j * 16 + q_row + t, cols) * ldb +
                                          VEC * q_chunk) * ES);
    } else {
        const int c = NF * (lane % 16);
        off_b[0][0] = (uint32_t)(((int64_t)4 * VEC * (lane / 16) * ldb +
                                  (c < cols ? c : cols - NF)) * ES);
    }
    // VEC rows of an n-contiguous B, from the one at `row`
    auto load_rows = [&](uint32_t (&x)[S::KC ? 1 : NF * 4], const T* row, uint32_t off)
                         __attribute__((always_inline)) {
        if constexpr (!S::KC) {
            constexpr int W = NF * ES / 4, PW = W > 4 ? 4 : W;  // words per row of k, per load
            using V = typename RawLoad<4 * PW>::T;
#pragma unroll
            for (int r = 0; r < VEC; ++r) {
                const char* b = reinterpret_cast<const char*>(row + (int64_t)r * ldb);
#pragma unroll
                for (int h = 0; h < W / PW; ++h) {
                    const V v = *reinterpret_cast<const V*>(b + off + h * 16);
#pragma unroll
                    for (int q = 0; q < PW; ++q) x[W * r + PW * h + q] = v[q];
                }
            }
        }
    };
    auto load = [&](StreamBatch<S>& x, int batch) __attribute__((always_inline)) {
        const int k = batch * 4 * KSTEP;
        const char* a = reinterpret_cast<const char*>(A + k);
        const char* b = reinterpret_cast<const char*>(B + k);
#pragma unroll
        for (int i = 0; i < RF; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                x.a[i][t] = *reinterpret_cast<const u32x4_elem<T>*>(a + off_a[i][t]);
        if constexpr (S::KC) {
#pragma unroll
            for (int j = 0; j < NF; ++j)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    x.b[j][t] = *reinterpret_cast<const u32x4_elem<T>*>(b + off_b[j][t]);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                load_rows(x.r[t], B + (int64_t)(k + VEC * t) * ldb, off_b[0][0]);
        }
    };
    auto multiply = [&](StreamBatch<S>& x) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < RF; ++i) quad_turn(x.a[i], lane);
        if constexpr (S::KC)
#pragma unroll
            for (int j = 0; j < NF; ++j) quad_turn(x.b[j], lane);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                u32x4 b;
                if constexpr (S::KC) b = x.b[j][t];
                else b = rows_fragment<S>(x.r[t], j);
#pragma unroll
                for (int i = 0; i < RF; ++i) mfma16<T>(x.a[i][t], b, acc[i][j]);
            }
    };
    // whole batches of K, split evenly over the waves
    const bool narrow = !S::KC && cols < S::BN && cols % NF != 0;
    const int steps = narrow ? 0 : K / KSTEP, batches = steps / 4;
    const int b_lo = (int)((int64_t)batches * wave / S::WAVES);
    const int b_hi = (int)((int64_t)batches * (wave + 1) / S::WAVES);
    // Loads stand in no branch inside the loop: the compiler would have to wait
    // for all of them wherever such a branch ends.
    StreamBatch<S> x0;
    if (b_lo < b_hi) load(x0, b_lo);
    meanwhile();
    if (b_lo < b_hi) {
        int b = b_lo;
        if constexpr (S::TWO) {
            StreamBatch<S> x1;
            for (; b + 2 < b_hi; b += 2) {
                load(x1, b + 1);
                multiply(x0);
                load(x0, b + 2);
                multiply(x1);
            }
            if (b + 1 < b_hi) {
                load(x1, b + 1);
                multiply(x0);
                multiply(x1);
            } else {
                multiply(x0);
            }
        } else {
            for (; b + 1 < b_hi; ++b) {
                multiply(x0);
                __builtin_amdgcn_sched_barrier(0);
                load(x0, b + 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            multiply(x0);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // the steps that fill no batch, K's ragged end, and every step of a narrow
    // matrix: one fragment step at a time, in the MFMA's lane order
    const int all = (K + KSTEP - 1) / KSTEP;
    for (int t = 4 * batches + (S::WAVES - 1 - wave); t < all; t += S::WAVES) {
        const int k = t * KSTEP + VEC * (lane / 16);
        const bool whole = t < steps;
        u32x4 fa[RF];
        uint32_t br[S::KC ? 1 : NF * 4];
        if constexpr (!S::KC)
            if (whole)
                load_rows(br, B + (int64_t)t * KSTEP * ldb,
                          off_b[0][0] - (uint32_t)((int64_t)3 * VEC * (lane / 16) * ldb * ES));
#pragma unroll
        for (int i = 0; i < RF; ++i) {
            const T* row = A + (int64_t)last(i * 16 + lane % 16, rows) * lda;
            fa[i] = whole ? *reinterpret_cast<const u32x4_elem<T>*>(row + k)
                          : clamped_chunk<T>(row, 1, k, K);
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const int c = last(S::column(j, lane % 16), cols);
            u32x4 fb;
            if constexpr (S::KC) {
                const T* row = B + (int64_t)c * ldb;
                fb = whole ? *reinterpret_cast<const u32x4_elem<T>*>(row + k)
                           : clamped_chunk<T>(row, 1, k, K);
            } else {
                fb = whole ? rows_fragment<S>(br, j) : clamped_chunk<T>(B + c, ldb, k, K);
            }
#pragma unroll
            for (int i = 0; i < RF; ++i) mfma16<T>(fa[i], fb, acc[i][j]);
        }
    }
}

template <class S, typename OutT, int RAG>
__global__ __launch_bounds__(S::THREADS) void stream_kernel(RaggedArgs p)
{
    using T = typename S::T;
    constexpr int RF = S::RF, NF = S::NF, ES = S::ES;
    __shared__ f32x4 part[S::WAVES][S::SLOTS][64];
    constexpr bool LORA = RAG == RAG_LORA || RAG == RAG_LORA_ONE;
    __shared__ int adapter[LORA ? S::BM : 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn, start = 0, size = p.M, g = 0;
    if constexpr (RAG == RAG_ROWS || RAG == RAG_SHRINK) {
        RowTile t;
        if (!find_row_tile<S::BM>(p, blockIdx.x, p.tiles_n, t)) return;
        g = t.group;
        if constexpr (RAG == RAG_SHRINK) {
            if (p.ids) g = __builtin_amdgcn_readfirstlane(p.ids[g]);
            if (g < 0 || g >= p.adapters) return;
        }
        start = t.start;
        size = t.size;
        p.tiles_m = t.tiles_m;
        tile_of(p, t.in_group, tm, tn);
        if (p.scales) p.alpha *= p.scales[g];
    } else {
        tile_coords(p, tm, tn);
    }
    const int r0 = tm * S::BM, n0 = tn * S::BN;  // r0 within the group
    // with an n-contiguous B the last tile of a row moves back to end at
    // column N
    const int nb = S::KC || n0 + S::BN <= p.N ? n0 : (p.N >= S::BN ? p.N - S::BN : 0);
    const T* A = static_cast<const T*>(p.A) + (int64_t)(start + r0) * p.lda;
    const T* B = static_cast<const T*>(p.B) + (int64_t)g * p.stride_b +
                 (S::KC ? (int64_t)nb * p.ldb : nb);
    if constexpr (RAG == RAG_SHRINK) {
        const int k_lo = blockIdx.y * p.k_slice;
        A += k_lo;
        B += S::KC ? (int64_t)k_lo : (int64_t)k_lo * p.ldb;
        p.K = p.K - k_lo < p.k_slice ? p.K - k_lo : p.k_slice;
        p.D += (int64_t)blockIdx.y * p.rows * p.rank_pad;
    }
    const int rows = size - r0;  // of the group, from the tile's first

    f32x4 acc[RF][NF] = {};
    stream_product<S>(A, p.lda, rows, B, p.ldb, p.N - nb, p.K, wave, lane, acc, [&] {
        if constexpr (LORA) map_adapters<S::BM, S::THREADS>(p, r0, tid, adapter);
    });

    // RAG_LORA_ONE: T here instead of in a launch of its own, an adapter and 16
    // ranks at a time
    __shared__ __attribute__((aligned(16))) float t_row[RAG == RAG_LORA_ONE ? S::BM : 1][LORA_ONE_RANK];
    if constexpr (RAG == RAG_LORA_ONE) {
        using D = StreamConfig<T, true, 1, 1>;
        static_assert(RF == 1, "a fragment of rows");
        const int mine = lane % 16 < rows ? adapter[lane % 16] : -1;
        for (uint64_t left = __ballot(mine >= 0); left != 0;) {
            const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
            left &= ~__ballot(mine == a);
            const T* down = static_cast<const T*>(p.down) + (int64_t)a * p.stride_down;
            for (int c0 = 0; c0 < p.rank; c0 += 16) {
                f32x4 t[1][1] = {};
                stream_product<D>(A, p.lda, rows, down + (int64_t)c0 * p.ld_down, p.ld_down,
                                  p.rank - c0, p.K, wave, lane, t, [] {});
                part[wave][0][lane] = t[0][0];
                __syncthreads();
                if (wave == 0 && mine == a) {
                    f32x4 v = part[0][0][lane];
#pragma unroll
                    for (int w = 1; w < S::WAVES; ++w) v += part[w][0][lane];
                    v *= p.scales ? p.scales[a] : 1.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        t_row[lane % 16][c0 + 4 * (lane / 16) + e] =
                            c0 + 4 * (lane / 16) + e < p.rank ? v[e] : 0.0f;
                }
                __syncthreads();
            }
        }
    }

    // the low-rank part of this thread's outputs
    f32x4 low[LORA ? S::PASSES * S::IPT : 1];
    if constexpr (LORA) {
#pragma unroll
        for (int q = 0; q < S::PASSES * S::IPT; ++q) {
            const int item = tid + (q % S::IPT) * S::THREADS, slot = item / 64, l = item & 63;
            const int row = ((q / S::IPT) * S::PF + slot / NF) * 16 + l % 16;
            const int col = nb + S::slot_column(slot % NF, l);
            low[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (item < S::ITEMS && row < rows && col < p.N && adapter[row] >= 0)
                low[q] = lora_row<T>(p, col, adapter[row], nb + S::BN <= p.N,
                                     [&](int r, f32x4 (&t)[2]) __attribute__((always_inline)) {
                                         if constexpr (RAG == RAG_LORA) {
                                             load_t(p, r0 + row, r, t);
                                         } else {
                                             t[0] = *reinterpret_cast<const f32x4*>(&t_row[row][r]);
                                             t[1] = *reinterpret_cast<const f32x4*>(&t_row[row][r + 4]);
                                         }
                                     });
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
            if (row >= rows || col >= (RAG == RAG_SHRINK ? p.rank_pad : p.N)) continue;
            f32x4 v = part[0][slot][l];
#pragma unroll
            for (int w = 1; w < S::WAVES; ++w) v += part[w][slot][l];
            if constexpr (LORA) v += low[pass * S::IPT + h];
            v *= p.alpha;
            const int64_t at = start + r0 + row;
            OutT* d = reinterpret_cast<OutT*>(p.D) + at * p.ldd + col;
            const OutT* c = reinterpret_cast<const OutT*>(p.C) + at * p.ldc + col;
            if constexpr (RAG == RAG_SHRINK) {  // columns past the rank are zero
#pragma unroll
                for (int s4 = 0; s4 < 4; ++s4) v[s4] = col + s4 < p.N ? v[s4] : 0.0f;
                *reinterpret_cast<f32x4*>(d) = v;
                if constexpr (ES == 2)
                    if (p.t_terms) store_terms(p, at, col, v);
                continue;
            }
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
