// Products of few rows with matrices that are read once: tiles of 16 to 64
// rows, for experts or requests with a handful of rows each.  Such a call is
// bound by the bytes of B, so the kernel is built around keeping them in
// flight rather than around reuse:
//
//  * one workgroup of eight waves per tile of 16*RF rows and 16*NF columns,
//    the waves splitting K into eight runs, so even a call of a few tiles has
//    every wave of a compute unit loading;
//  * operands go from memory straight into registers, four fragment steps of
//    K at a time and, where the registers hold them, two such batches in flight;
//    nothing is staged, so no barrier is met until the waves' sums are added;
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
// rows, one or two blocks of 16 ranks and a K that is not too long costs less
// than a launch and T's way through memory (one token, 2048x2048, rank 8: 12.6 ->
// 10.31 us).
//
// RAG_GATE (act.hpp) takes NF / 2 fragments of a gate's columns and as many of
// their partners'.
#pragma once

#include "act.hpp"
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
    static_assert(RF % PF == 0 && NF <= 4, "exchange");
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

// VEC rows of k, `bytes` apart, of NF adjacent columns per lane (lane % 16 the
// columns' place, lane / 16 the rows'), `off` the lane's place in them.
template <typename T, int NF>
__device__ __forceinline__ void load_rows(uint32_t* x, const T* row, int64_t ld, uint32_t off)
{
    constexpr int VEC = 16 / sizeof(T), W = NF * sizeof(T) / 4;  // words per row of k
    using V = typename RawLoad<4 * W>::T;
#pragma unroll
    for (int r = 0; r < VEC; ++r) {
        const V v = *reinterpret_cast<const V*>(reinterpret_cast<const char*>(row + (int64_t)r * ld) + off);
#pragma unroll
        for (int q = 0; q < W; ++q) x[W * r + q] = v[q];
    }
}

// Fragment j of them (columns j, j + NF, ...) as the MFMA operand.
template <typename T, int NF>
__device__ __forceinline__ u32x4 rows_fragment(const uint32_t* x, int j)
{
    u32x4 r;
    if constexpr (sizeof(T) == 4) {      // row k: words NF*k .. of the columns
#pragma unroll
        for (int q = 0; q < 4; ++q) r[q] = x[NF * q + j];
    } else {                             // row k: words NF/2*k .., two columns each
        constexpr int W = NF / 2;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            r[q] = __builtin_amdgcn_perm(x[W * (2 * q + 1) + j / 2], x[W * (2 * q) + j / 2],
                                         j % 2 ? 0x07060302u : 0x05040100u);
    }
    return r;
}

// This wave's part of a tile's product, added to acc: `rows` rows of A (at least
// one) and `cols` columns of B, from the tile's first, by all of K.  meanwhile()
// runs once, while the first loads are under way.  GATE: the tile's columns are
// twice `cols`, the second half of its fragments `split` columns further.
template <class S, bool GATE = false, class F>
__device__ __forceinline__ void stream_product(const typename S::T* A, int64_t lda, int rows,
                                               const typename S::T* B, int64_t ldb, int cols, int K,
                                               int wave, int lane, f32x4 (&acc)[S::RF][S::NF],
                                               F meanwhile, int64_t split = 0)
{
    using T = typename S::T;
    constexpr int RF = S::RF, NF = S::NF, KSTEP = S::KSTEP, VEC = S::VEC, ES = S::ES;
    // fragments of one half, and of what an n-contiguous B's rows are read in
    constexpr int HALVES = GATE ? 2 : 1, NH = NF / HALVES;
    static_assert(!GATE || NF % 2 == 0, "halves");
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
                off_b[j][t] = (uint32_t)(((last(j % NH * 16 + q_row + t, cols) + j / NH * split) * ldb +
                                          VEC * q_chunk) * ES);
    } else {
        const int c = NH * (lane % 16);
        off_b[0][0] = (uint32_t)(((int64_t)4 * VEC * (lane / 16) * ldb +
                                  (c < cols ? c : cols - NH)) * ES);
    }
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
#pragma unroll
                for (int half = 0; half < HALVES; ++half)
                    load_rows<T, NH>(x.r[t] + half * NH * 4,
                                     B + (int64_t)(k + VEC * t) * ldb + half * split, ldb, off_b[0][0]);
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
                else b = rows_fragment<T, NH>(x.r[t] + j / NH * NH * 4, j % NH);
#pragma unroll
                for (int i = 0; i < RF; ++i) mfma16<T>(x.a[i][t], b, acc[i][j]);
            }
    };
    // whole batches of K, split evenly over the waves
    const bool narrow = !S::KC && cols < S::BN / HALVES && cols % NH != 0;
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
#pragma unroll
                for (int half = 0; half < HALVES; ++half)
                    load_rows<T, NH>(br + half * NH * 4, B + (int64_t)t * KSTEP * ldb + half * split, ldb,
                                     off_b[0][0] - (uint32_t)((int64_t)3 * VEC * (lane / 16) * ldb * ES));
#pragma unroll
        for (int i = 0; i < RF; ++i) {
            const T* row = A + (int64_t)last(i * 16 + lane % 16, rows) * lda;
            fa[i] = whole ? *reinterpret_cast<const u32x4_elem<T>*>(row + k)
                          : clamped_chunk<T>(row, 1, k, K);
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const int c = last(GATE ? StreamConfig<T, S::KC, RF, NH>::column(j % NH, lane % 16)
                                    : S::column(j, lane % 16), cols);
            const int64_t far = j / NH * split;  // to the half of fragment j
            u32x4 fb;
            if constexpr (S::KC) {
                const T* row = B + (c + far) * ldb;
                fb = whole ? *reinterpret_cast<const u32x4_elem<T>*>(row + k)
                           : clamped_chunk<T>(row, 1, k, K);
            } else {
                fb = whole ? rows_fragment<T, NH>(br + j / NH * NH * 4, j % NH)
                           : clamped_chunk<T>(B + c + far, ldb, k, K);
            }
#pragma unroll
            for (int i = 0; i < RF; ++i) mfma16<T>(fa[i], fb, acc[i][j]);
        }
    }
}

// Four adjacent columns of D from `col`, plus beta times C's; those outside
// [n0, N) are not stored.
template <typename OutT>
__device__ __forceinline__ void store_piece(OutT* d, const OutT* c, f32x4 v, float beta, int col, int n0,
                                            int N)
{
    using Piece = typename RawLoad<4 * sizeof(OutT)>::T;
    if (col >= n0 && col + 4 <= N) {
        OutT e[4];
        if (beta != 0.0f) {
            const Piece w = *reinterpret_cast<const Piece*>(c);
            __builtin_memcpy(e, &w, sizeof(e));
#pragma unroll
            for (int s = 0; s < 4; ++s) v[s] += beta * to_f32(e[s]);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) e[s] = from_f32<OutT>(v[s]);
        Piece w;
        __builtin_memcpy(&w, e, sizeof(e));
        *reinterpret_cast<Piece*>(d) = w;
    } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (col + s < n0 || col + s >= N) continue;
            float o = v[s];
            if (beta != 0.0f) o += beta * to_f32(c[s]);
            d[s] = from_f32<OutT>(o);
        }
    }
}

// Four columns of a row of T from `col`, and of its terms; columns from the rank
// to rank_pad are zero (the direct-to-LDS kernels read them).  A tile that moved
// back to end at the rank (`moved`) has its first column n0 anywhere in a piece
// and reaches none of the padding: it stores element by element, and the piece
// that ends at the rank goes on to rank_pad.
template <typename T>
__device__ __forceinline__ void store_t(const RaggedArgs& p, int64_t row, int col, f32x4 v, int n0,
                                        bool moved)
{
    float* d = reinterpret_cast<float*>(p.D) + row * p.ldd;
    if (!moved) {
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s] = col + s < p.N ? v[s] : 0.0f;
        *reinterpret_cast<f32x4*>(d + col) = v;
        if constexpr (sizeof(T) == 2)
            if (p.t_terms) store_terms(p, row, col, v);
        return;
    }
    auto store = [&](int k, float t) __attribute__((always_inline)) {
        d[k] = t;
        if constexpr (sizeof(T) == 2)
            if (p.t_terms) store_term(p, row, k, t);
    };
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (col + s >= n0) store(col + s, v[s]);
    if (col + 4 == p.N)
        for (int k = p.N; k < p.rank_pad; ++k) store(k, 0.0f);
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
            if constexpr (RAG == RAG_SHRINK) {
                store_t<T>(p, at, col, v, n0, nb != n0);
                continue;
            }
            store_piece(d, c, v, p.beta, col, n0, p.N);
        }
    });
}

// RAG_ACT and RAG_GATE: the same product, whose sums go through act_outputs.
template <class S, typename OutT, bool GATE>
__global__ __launch_bounds__(S::THREADS) void stream_act_kernel(ActArgs p)
{
    using T = typename S::T;
    constexpr int RF = S::RF, HALVES = GATE ? 2 : 1, NH = S::NF / HALVES, BNO = 16 * NH;
    using H = StreamConfig<T, S::KC, RF, NH>;  // one half's columns
    constexpr int ITEMS = S::PF * NH * 64, IPT = (ITEMS + S::THREADS - 1) / S::THREADS;
    __shared__ f32x4 part[S::WAVES][S::SLOTS][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    if (!narrow_act<S::BM, T, OutT>(p, tm, tn)) return;
    const int r0 = tm * S::BM, n0 = tn * BNO;
    // with an n-contiguous B the last tile of a row moves back to end at column N
    const int nb = S::KC || n0 + BNO <= p.N ? n0 : (p.N >= BNO ? p.N - BNO : 0);
    const T* A = static_cast<const T*>(p.A) + (int64_t)r0 * p.lda;
    const T* B = static_cast<const T*>(p.B) + (S::KC ? (int64_t)nb * p.ldb : nb);
    const int rows = p.M - r0;

    f32x4 acc[RF][S::NF] = {};
    stream_product<S, GATE>(A, p.lda, rows, B, p.ldb, p.N - nb, p.K, wave, lane, acc, [] {},
                            GATE ? p.N : 0);

    static_for<S::PASSES>([&](auto pass_c) __attribute__((always_inline)) {
        constexpr int pass = decltype(pass_c)::value;
        if constexpr (pass > 0) __syncthreads();
        static_for<S::SLOTS>([&](auto q_c) __attribute__((always_inline)) {
            constexpr int slot = decltype(q_c)::value, i = pass * S::PF + slot / S::NF;
            constexpr int half = slot % S::NF / NH, q = slot % NH;
            f32x4 v;
            if constexpr (S::KC) v = acc[i][half * NH + q];
            else
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][half * NH + (4 * q + e) % NH][(4 * q + e) / NH];
            part[wave][slot][lane] = v;
        });
        __syncthreads();
#pragma unroll
        for (int h = 0; h < IPT; ++h) {
            const int item = tid + h * S::THREADS, l = item & 63;
            if (item >= ITEMS) break;
            const int f = item / 64 / NH, q = item / 64 % NH, slot = f * S::NF + q;
            const int row = (pass * S::PF + f) * 16 + l % 16, col = nb + H::slot_column(q, l);
            if (row >= rows || col >= p.N) continue;
            f32x4 g = part[0][slot][l], u{};
#pragma unroll
            for (int w = 1; w < S::WAVES; ++w) g += part[w][slot][l];
            if constexpr (GATE) {
                u = part[0][slot + NH][l];
#pragma unroll
                for (int w = 1; w < S::WAVES; ++w) u += part[w][slot + NH][l];
            }
            // (a tile that moved back computes its neighbour's columns again:
            // those are not stored twice, since D may be R)
            const int n = p.N - col, skip = n0 - col;
            act_outputs<GATE, OutT>(p, r0 + row, col, n, g, u, act_bias<OutT>(p, col, n),
                                    GATE ? act_bias<OutT>(p, p.N + col, n) : f32x4{}, skip);
        }
    });
}

// The K-ragged product (RAG_K) in the same manner, for outputs of few tiles
// over many rows (adapters' gradients: 64 x 4096 from thousands of rows): tiles
// of 16 F x 16 F, the eight waves splitting the group's rows, which are K, so
// 36 tiles use the card as 288 would.  Both operands are stored by rows of K.
// Four adapters' gradients of 64x4096 from 8192 rows: 26 -> 22.5 us; three of
// 192x200 in fp32 from 11000 rows: 127 -> 35 us.
template <typename T, int F, typename OutT>
__global__ __launch_bounds__(512) void stream_k_kernel(RaggedArgs p)
{
    using S = StreamConfig<T, false, F, F>;
    constexpr int KSTEP = S::KSTEP, VEC = S::VEC, ES = S::ES;
    __shared__ f32x4 part[S::WAVES][S::SLOTS][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int g, t, tm, tn;
    if (!find_k_tile(p, blockIdx.x, g, t)) return;
    tile_of(p, t, tm, tn);
    int start, K;
    group_span(p, g, start, K);
    start = __builtin_amdgcn_readfirstlane(start);
    K = __builtin_amdgcn_readfirstlane(K);
    p.alpha = group_alpha(p, g, K);
    // the last tile of a row or column moves back to end at the matrix's end
    auto moved = [](int x0, int extent) {
        return x0 + S::BM <= extent ? x0 : (extent >= S::BM ? extent - S::BM : 0);
    };
    const int m0 = tm * S::BM, n0 = tn * S::BN, mb = moved(m0, p.M), nb = moved(n0, p.N);
    const int rows = p.M - mb, cols = p.N - nb;
    const T* A = static_cast<const T*>(p.A) + (int64_t)start * p.lda + mb;
    const T* B = static_cast<const T*>(p.B) + (int64_t)start * p.ldb + nb;

    f32x4 acc[F][F] = {};
    const int c = F * (lane % 16);
    const uint32_t ca = (uint32_t)((c < rows ? c : rows - F) * ES);
    const uint32_t cb = (uint32_t)((c < cols ? c : cols - F) * ES);
    const uint32_t ka = (uint32_t)((int64_t)VEC * (lane / 16) * p.lda * ES);
    const uint32_t kb = (uint32_t)((int64_t)VEC * (lane / 16) * p.ldb * ES);
    struct Batch {
        uint32_t a[4][F * 4], b[4][F * 4];
    };
    // lane group lane / 16 takes the VEC rows from VEC (4 (lane / 16) + s) in step s
    auto load = [&](Batch& x, int batch) __attribute__((always_inline)) {
        const int k = batch * 4 * KSTEP;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            load_rows<T, F>(x.a[s], A + (int64_t)(k + VEC * s) * p.lda, p.lda, 4 * ka + ca);
            load_rows<T, F>(x.b[s], B + (int64_t)(k + VEC * s) * p.ldb, p.ldb, 4 * kb + cb);
        }
    };
    auto multiply_step = [&](const uint32_t (&a)[F * 4], const uint32_t (&b)[F * 4])
                             __attribute__((always_inline)) {
        u32x4 fa[F];
#pragma unroll
        for (int i = 0; i < F; ++i) fa[i] = rows_fragment<T, F>(a, i);
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const u32x4 fb = rows_fragment<T, F>(b, j);
#pragma unroll
            for (int i = 0; i < F; ++i) mfma16<T>(fa[i], fb, acc[i][j]);
        }
    };
    auto multiply = [&](const Batch& x) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 4; ++s) multiply_step(x.a[s], x.b[s]);
    };
    const bool narrow = rows < F || cols < F || (rows < S::BM && rows % F != 0) ||
                        (cols < S::BN && cols % F != 0);
    const int steps = narrow ? 0 : K / KSTEP, batches = steps / 4;
    const int b_lo = (int)((int64_t)batches * wave / S::WAVES);
    const int b_hi = (int)((int64_t)batches * (wave + 1) / S::WAVES);
    if (b_lo < b_hi) {
        Batch x0;
        load(x0, b_lo);
        int b = b_lo;
        if constexpr (F <= 2) {
            Batch x1;
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
    // the steps that fill no batch, K's ragged end and narrow matrices
    const int all = (K + KSTEP - 1) / KSTEP;
    for (int s = 4 * batches + (S::WAVES - 1 - wave); s < all; s += S::WAVES) {
        if (s < steps) {
            uint32_t xa[F * 4], xb[F * 4];
            load_rows<T, F>(xa, A + (int64_t)s * KSTEP * p.lda, p.lda, ka + ca);
            load_rows<T, F>(xb, B + (int64_t)s * KSTEP * p.ldb, p.ldb, kb + cb);
            multiply_step(xa, xb);
            continue;
        }
        const int k = s * KSTEP + VEC * (lane / 16);
        u32x4 fa[F];
#pragma unroll
        for (int i = 0; i < F; ++i)
            fa[i] = clamped_chunk<T>(A + (c + i < rows ? c + i : rows - 1), p.lda, k, K);
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const u32x4 fb = clamped_chunk<T>(B + (c + j < cols ? c + j : cols - 1), p.ldb, k, K);
#pragma unroll
            for (int i = 0; i < F; ++i) mfma16<T>(fa[i], fb, acc[i][j]);
        }
    }

    static_for<S::PASSES>([&](auto pass_c) __attribute__((always_inline)) {
        constexpr int pass = decltype(pass_c)::value;
        if constexpr (pass > 0) __syncthreads();
        static_for<S::SLOTS>([&](auto q_c) __attribute__((always_inline)) {
            constexpr int slot = decltype(q_c)::value, i = pass * S::PF + slot / F, q = slot % F;
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[i][(4 * q + e) % F][(4 * q + e) / F];
            part[wave][slot][lane] = v;
        });
        __syncthreads();
#pragma unroll
        for (int h = 0; h < S::IPT; ++h) {
            const int item = tid + h * S::THREADS, slot = item / 64, l = item & 63;
            if (item >= S::ITEMS) break;
            const int row = mb + F * (l % 16) + pass * S::PF + slot / F;
            const int col = nb + S::slot_column(slot % F, l);
            if (row < m0 || row >= p.M || col >= p.N) continue;
            f32x4 v = part[0][slot][l];
#pragma unroll
            for (int w = 1; w < S::WAVES; ++w) v += part[w][slot][l];
            v *= p.alpha;
            store_piece(reinterpret_cast<OutT*>(p.D) + g * p.stride_d + (int64_t)row * p.ldd + col,
                        reinterpret_cast<const OutT*>(p.C) + g * p.stride_c + (int64_t)row * p.ldc + col,
                        v, p.beta, col, n0, p.N);
        }
    });
}

}  // namespace dg
