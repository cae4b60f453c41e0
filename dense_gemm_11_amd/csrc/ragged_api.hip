// C ABI of the products over ragged groups of rows: argument validation, tile
// choice and launches.  Declared in include/dense_gemm.h.
#include <algorithm>
#include <climits>
#include <cstdio>

#include "handle.hpp"
#include "ragged_variants.hpp"
#include "lora.hpp"

namespace dg {
namespace {

constexpr int MAX_GROUPS = 1 << 16;

// The kernels form row, column and step numbers in 32 bits up to a tile or a
// batch of steps past the end (a last tile of 192 rows would pass 2^31 from M =
// 2^31 - 128), and twice the padded rank.
constexpr int64_t MAX_EXTENT = INT_MAX - 512;

// The layout, type and size checks that the three calls share.
gemm_status_t check_common(gemm_handle_t h, gemm_op_t transB, int64_t M, int64_t N, int64_t K,
                           gemm_dtype_t dtype)
{
    if (!h) return GEMM_ERR_INVALID_VALUE;
    if (transB != GEMM_OP_N && transB != GEMM_OP_T) return GEMM_ERR_INVALID_VALUE;
    if (dtype != GEMM_DTYPE_F32 && dtype != GEMM_DTYPE_BF16_F32 && dtype != GEMM_DTYPE_BF16_BF16)
        return GEMM_ERR_INVALID_VALUE;
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    return GEMM_OK;
}

// Byte offsets inside a panel of `rows` rows of `ld` elements and `cols` more
// stay below 2^32.
bool panel_fits(int64_t rows, int64_t ld, int64_t cols, int64_t es)
{
    return (rows * ld + cols) * es < ((int64_t)1 << 32) - 64;
}

// A launch has fewer than 2^32 threads along its first axis.
bool grid_fits(int64_t grid, int threads) { return grid * threads < (int64_t)1 << 32; }

// C against D: the same matrix with the same strides, or disjoint.
bool c_d_ok(const void* C, int64_t span_c, const void* D, int64_t span_d, bool same_strides)
{
    return C == D ? same_strides : !ranges_overlap(C, span_c, D, span_d);
}

// A call's tiles, tallest first: the direct-to-LDS ones, then the streaming
// ones.
struct TileList {
    const RaggedTile* dma;
    const RaggedTile* stream;
    int n_dma, n;
    const RaggedTile& operator[](int i) const { return i < n_dma ? dma[i] : stream[i - n_dma]; }
};
typedef const RaggedTile* (*TileTable)(int* count);
TileList tile_list(TileTable dma, TileTable stream)
{
    TileList l{};
    int n_stream = 0;
    l.dma = dma(&l.n_dma);
    l.stream = stream(&n_stream);
    l.n = l.n_dma + n_stream;
    return l;
}

// Number of tile i among those of its height.
int nth_of_height(const TileList& t, int i)
{
    int n = 0;
    for (int j = 0; j < i; ++j) n += t[j].bm == t[i].bm;
    return n;
}

// The forced tile (gemm_set_group_tile_nth), else the one of least expected
// time among those whose grid fits; tiles(t) is the number of output tiles of t a
// call has, or expects, grid(t) its workgroups, and `bytes` what it reads and
// writes at the least.
template <class F, class G>
const RaggedTile& pick_tile(gemm_handle_t h, const TileList& t, bool b_kc, int64_t K, double bytes,
                            F tiles, G grid)
{
    int best = t.n - 1;
    if (h->forced_rows > 0) {
        int height = t[best].bm;
        for (int i = 0; i < t.n; ++i)
            if (t[i].bm <= h->forced_rows && t[i].bm > height) height = t[i].bm;
        for (int i = 0; i < t.n; ++i)
            if (t[i].bm == height) {
                best = i;
                if (nth_of_height(t, i) == h->forced_nth) break;
            }
        return t[best];
    }
    double best_us = 0.0;
    for (int i = 0; i < t.n; ++i) {
        if (!grid_fits(grid(t[i]), t[i].threads)) continue;
        const double us = expected_us(t[i], b_kc, (double)tiles(t[i]), (double)K, bytes, device_cus());
        if (best_us == 0.0 || us < best_us) {
            best = i;
            best_us = us;
        }
    }
    return t[best];
}

// Rows of tiles of height bm in `busy` groups of avg rows on average: the last
// tile of a group is half full.
double row_tiles(double busy, double avg, int bm)
{
    return busy * std::max(1.0, avg / bm + 0.5);
}

// Notes and logs the launch of tile t.
void note_call(gemm_handle_t h, const char* what, const RaggedArgs& a, const TileList& tiles,
               const RaggedTile& t, int bn, int64_t grid, int launches = 1)
{
    int i = 0;
    while (&tiles[i] != &t) ++i;
    const int bm = t.bm;
    h->last_group = gemm_group_launch_t{bm, bn, nth_of_height(tiles, i), launches, 0, 0, 0};
    if (h->log)
        std::fprintf(stderr, "gemm: %s %dx%d rows=%d groups=%d M=%d N=%d K=%d grid=%lld\n", what, bm,
                     bn, a.rows, a.groups, a.M, a.N, a.K, (long long)grid);
}

}  // namespace
}  // namespace dg

extern "C" {

gemm_status_t gemm_set_group_tile_nth(gemm_handle_t h, int rows, int nth)
{
    if (!h || rows < 0 || nth < 0) return GEMM_ERR_INVALID_VALUE;
    h->forced_rows = rows;
    h->forced_nth = nth;
    return GEMM_OK;
}

gemm_status_t gemm_set_group_tile(gemm_handle_t h, int rows)
{
    return gemm_set_group_tile_nth(h, rows, 0);
}

int gemm_last_group_tile(gemm_handle_t h) { return h ? h->last_group.rows : -1; }

gemm_status_t gemm_last_group_launch(gemm_handle_t h, gemm_group_launch_t* out)
{
    if (!h || !out) return GEMM_ERR_INVALID_VALUE;
    *out = h->last_group;
    return GEMM_OK;
}

gemm_status_t gemm_run_grouped(gemm_handle_t h, gemm_op_t transB, int64_t M, int64_t N, int64_t K,
                               float alpha, const void* A, int64_t lda, const void* B, int64_t ldb,
                               int64_t strideB, float beta, const void* C, int64_t ldc, void* D,
                               int64_t ldd, gemm_dtype_t dtype, const gemm_groups_t* groups,
                               hipStream_t stream)
{
    using namespace dg;
    const gemm_status_t st = check_common(h, transB, M, N, K, dtype);
    if (st != GEMM_OK) return st;
    if (!groups || groups->groups < 0 || strideB < 0) return GEMM_ERR_INVALID_VALUE;
    const int64_t one = 1;
    const int64_t es = dtype == GEMM_DTYPE_F32 ? 4 : 2, eo = dtype == GEMM_DTYPE_BF16_BF16 ? 2 : 4;
    const bool b_kc = transB == GEMM_OP_T;
    if (lda < std::max(one, K) || ldb < std::max(one, b_kc ? K : N) || ldd < std::max(one, N) ||
        (beta != 0.0f && ldc < std::max(one, N)))
        return GEMM_ERR_INVALID_VALUE;
    h->last_group = {};
    if (M == 0 || N == 0 || groups->groups == 0) return GEMM_OK;
    const bool reads_ab = K > 0 && alpha != 0.0f;
    if (!groups->offsets || !D || (beta != 0.0f && !C) || (reads_ab && (!A || !B)))
        return GEMM_ERR_INVALID_VALUE;
    if (M > MAX_EXTENT || N > MAX_EXTENT || K > MAX_EXTENT || lda > INT_MAX || ldb > INT_MAX ||
        ldd > INT_MAX || (beta != 0.0f && ldc > INT_MAX) || groups->groups > MAX_GROUPS)
        return GEMM_ERR_NOT_SUPPORTED;
    if (beta != 0.0f &&
        !c_d_ok(C, ((M - 1) * ldc + N) * eo, D, ((M - 1) * ldd + N) * eo, ldc == ldd))
        return GEMM_ERR_INVALID_VALUE;
    if (reads_ab && (!aligned_to(A, es) || !aligned_to(B, es))) return GEMM_ERR_NOT_SUPPORTED;

    RaggedArgs a{};
    a.A = A;
    a.B = B;
    a.C = beta != 0.0f ? static_cast<const float*>(C) : nullptr;
    a.D = static_cast<float*>(D);
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = beta != 0.0f ? ldc : 0;
    a.ldd = ldd;
    a.M = (int)M;
    a.N = (int)N;
    a.K = reads_ab ? (int)K : 0;  // no K-steps: D = beta * C
    a.alpha = reads_ab ? alpha : 0.0f;
    a.beta = beta;
    a.c_vec = beta != 0.0f && aligned_to(C, eo);
    a.d_vec = aligned_to(D, eo);
    a.d_lines = aligned_to(D, 128) && ldd * eo % 128 == 0;
    a.offsets = groups->offsets;
    a.scales = reads_ab ? groups->scales : nullptr;
    a.groups = groups->groups;
    a.rows = (int)M;
    a.stride_b = strideB;
    // a group holds M / groups rows on average, and the host knows no more
    const int64_t busy = std::min<int64_t>(groups->groups, M);
    const double bytes = (double)es * K * ((double)busy * N + M) + (double)eo * M * N;
    const TileList tiles = dtype == GEMM_DTYPE_F32 ? tile_list(ragged_rows_f32, stream_rows_f32)
                                                   : tile_list(ragged_rows_bf16, stream_rows_bf16);
    // the most tile-rows any split into groups needs
    auto grid_of = [&](const RaggedTile& x) {
        return (M + busy * (x.bm - 1)) / x.bm * ceil_div(N, x.bn[b_kc]);
    };
    const RaggedTile& t = pick_tile(h, tiles, b_kc, K, bytes, [&](const RaggedTile& x) {
        return ceil_div(N, x.bn[b_kc]) *
               (busy > 1 ? row_tiles((double)busy, (double)M / busy, x.bm) : (double)ceil_div(M, x.bm));
    }, grid_of);
    const int bn = t.bn[b_kc];
    const int64_t kk = K + t.bk;
    if (!panel_fits(t.bm - 1, lda, kk, es) ||
        !(b_kc ? panel_fits(bn - 1, ldb, kk, es) : panel_fits(kk, ldb, bn, es)))
        return GEMM_ERR_NOT_SUPPORTED;
    a.tiles_n = (int)ceil_div(N, bn);
    a.group_m = 4;
    const int64_t grid = grid_of(t);
    if (!grid_fits(grid, t.threads)) return GEMM_ERR_NOT_SUPPORTED;
    if (h->fail_launch) return GEMM_ERR_HIP;
    if (t.fn[b_kc][dtype == GEMM_DTYPE_BF16_BF16](a, (int)grid, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    note_call(h, "grouped", a, tiles, t, bn, grid);
    return GEMM_OK;
}

gemm_status_t gemm_run_grouped_wgrad(gemm_handle_t h, int64_t M, int64_t N, int64_t rows, float alpha,
                                     const void* A, int64_t lda, const void* B, int64_t ldb,
                                     float beta, const void* C, int64_t ldc, int64_t strideC, void* D,
                                     int64_t ldd, int64_t strideD, gemm_dtype_t dtype,
                                     const gemm_groups_t* groups, hipStream_t stream)
{
    using namespace dg;
    const gemm_status_t st = check_common(h, GEMM_OP_N, M, N, rows, dtype);
    if (st != GEMM_OK) return st;
    if (!groups || groups->groups < 0) return GEMM_ERR_INVALID_VALUE;
    const int64_t one = 1, G = groups->groups;
    const int64_t es = dtype == GEMM_DTYPE_F32 ? 4 : 2, eo = dtype == GEMM_DTYPE_BF16_BF16 ? 2 : 4;
    if (lda < std::max(one, M) || ldb < std::max(one, N) || ldd < std::max(one, N) ||
        (beta != 0.0f && ldc < std::max(one, N)))
        return GEMM_ERR_INVALID_VALUE;
    h->last_group = {};
    if (M == 0 || N == 0 || G == 0) return GEMM_OK;
    const bool reads_ab = rows > 0 && alpha != 0.0f;
    if (!groups->offsets || !D || (beta != 0.0f && !C) || (reads_ab && (!A || !B)))
        return GEMM_ERR_INVALID_VALUE;
    if (M > MAX_EXTENT || N > MAX_EXTENT || rows > MAX_EXTENT || lda > INT_MAX || ldb > INT_MAX ||
        ldd > INT_MAX || (beta != 0.0f && ldc > INT_MAX) || G > MAX_GROUPS)
        return GEMM_ERR_NOT_SUPPORTED;
    // the groups' outputs apart from each other: one after another, or
    // beside each other within the rows
    const int64_t span_d = (M - 1) * ldd + N;
    if (G > 1 && strideD < span_d && !(strideD >= N && ldd >= (G - 1) * strideD + N))
        return GEMM_ERR_INVALID_VALUE;
    if (beta != 0.0f) {
        if (G > 1 && strideC < 0) return GEMM_ERR_INVALID_VALUE;
        const int64_t gap_c = G > 1 ? (G - 1) * strideC : 0, gap_d = G > 1 ? (G - 1) * strideD : 0;
        if (!c_d_ok(C, (gap_c + (M - 1) * ldc + N) * eo, D, (gap_d + span_d) * eo,
                    ldc == ldd && (G == 1 || strideC == strideD)))
            return GEMM_ERR_INVALID_VALUE;
    }
    if (reads_ab && (!aligned_to(A, es) || !aligned_to(B, es))) return GEMM_ERR_NOT_SUPPORTED;

    RaggedArgs a{};
    a.A = A;
    a.B = B;
    a.C = beta != 0.0f ? static_cast<const float*>(C) : nullptr;
    a.D = static_cast<float*>(D);
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = beta != 0.0f ? ldc : 0;
    a.ldd = ldd;
    a.M = (int)M;
    a.N = (int)N;
    a.alpha = alpha;
    a.beta = beta;
    a.c_vec = beta != 0.0f && aligned_to(C, eo);
    a.d_vec = aligned_to(D, eo);
    a.d_lines = aligned_to(D, 128) && ldd * eo % 128 == 0 && strideD * eo % 128 == 0;
    a.offsets = groups->offsets;
    a.scales = groups->scales;
    a.groups = (int)G;
    a.rows = reads_ab ? (int)rows : 0;  // no rows: D_g = beta * C_g
    a.stride_c = strideC;
    a.stride_d = strideD;
    const TileList tiles =
        dtype == GEMM_DTYPE_F32 ? tile_list(ragged_k_f32, stream_k_f32)
                                : tile_list(ragged_k_bf16, stream_k_bf16);
    auto tiles_of = [&](const RaggedTile& x) { return G * ceil_div(M, x.bm) * ceil_div(N, x.bn[0]); };
    // (every way of dealing them: a slice may round up to a tile more per XCD)
    auto most = [&](const RaggedTile& x) { return tiles_of(x) + DEAL_XCDS * G; };
    const RaggedTile& t = pick_tile(h, tiles, false, rows / G, 0.0, tiles_of, most);
    const int bn = t.bn[0];
    // offsets of one K-step, or of one batch of them (the kernels base each anew)
    const int64_t ks = t.stream ? 4 * t.bk : t.bk;
    if (!panel_fits(ks, 2 * lda, t.bm, es) || !panel_fits(ks, 2 * ldb, bn, es))
        return GEMM_ERR_NOT_SUPPORTED;
    a.tiles_m = (int)ceil_div(M, t.bm);
    a.tiles_n = (int)ceil_div(N, bn);
    a.group_m = std::min(a.tiles_m, 4);
    const int64_t per = (int64_t)a.tiles_m * a.tiles_n;
    a.deal = !a.d_lines && rows < 128 * G ? DEAL_RANGES
             : per < 2 * DEAL_XCDS        ? DEAL_TILES
                                          : DEAL_SLICES;
    const int64_t grid = deal_grid(a.deal, per, G);
    if (!grid_fits(grid, t.threads)) return GEMM_ERR_NOT_SUPPORTED;
    if (h->fail_launch) return GEMM_ERR_HIP;
    if (t.fn[0][dtype == GEMM_DTYPE_BF16_BF16](a, (int)grid, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    note_call(h, "grouped wgrad", a, tiles, t, bn, grid);
    return GEMM_OK;
}

size_t gemm_lora_workspace_bytes(int64_t M, int rank)
{
    using namespace dg;
    if (M <= 0 || rank <= 0) return 0;
    // rows of T's partial sums: at most 4 slices, and at most ceil(8192 / M)
    // of them; or T and its bf16 terms, three of half the size (gemm_run_lora);
    // does not decrease with M
    const int64_t pad = ceil_div(rank, LORA_PAD) * LORA_PAD;
    return (size_t)(std::max<int64_t>((5 * M + 1) / 2, std::min<int64_t>(4 * M, 8192 + M)) * pad) *
           sizeof(float);
}

gemm_status_t gemm_run_lora(gemm_handle_t h, gemm_op_t transB, int64_t M, int64_t N, int64_t K,
                            float alpha, const void* A, int64_t lda, const void* B, int64_t ldb,
                            float beta, const void* C, int64_t ldc, void* D, int64_t ldd,
                            gemm_dtype_t dtype, const gemm_lora_t* lora, void* ws, size_t ws_bytes,
                            hipStream_t stream)
{
    using namespace dg;
    const gemm_status_t st = check_common(h, transB, M, N, K, dtype);
    if (st != GEMM_OK) return st;
    if (!lora || lora->segments < 0 || lora->adapters < 0 || lora->rank < 0 ||
        lora->stride_down < 0 || lora->stride_up < 0 ||
        (lora->trans_down != GEMM_OP_N && lora->trans_down != GEMM_OP_T) ||
        (lora->trans_up != GEMM_OP_N && lora->trans_up != GEMM_OP_T))
        return GEMM_ERR_INVALID_VALUE;
    const int64_t one = 1, R = lora->rank;
    const int64_t es = dtype == GEMM_DTYPE_F32 ? 4 : 2, eo = dtype == GEMM_DTYPE_BF16_BF16 ? 2 : 4;
    const bool b_kc = transB == GEMM_OP_T;
    const bool down_kc = lora->trans_down == GEMM_OP_T, up_kc = lora->trans_up == GEMM_OP_T;
    h->last_group = {};
    // without an adapter, or with nothing to multiply, the call is gemm_run on a
    // handle of its own: h's forced variant and stream-K workspace, which other
    // streams may be using, have no part in it
    if (M == 0 || N == 0 || K == 0 || alpha == 0.0f || R == 0 || lora->segments == 0 ||
        lora->adapters == 0) {
        gemm_handle_s dense = *h;
        dense.forced_variant = dense.stream_k_mode = -1;
        dense.ws = nullptr;
        dense.ws_bytes = 0;
        return gemm_run(&dense, GEMM_OP_N, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, D,
                        ldd, dtype, stream);
    }
    if (lda < K || ldb < (b_kc ? K : N) || ldd < N || (beta != 0.0f && ldc < N) ||
        lora->ld_down < (down_kc ? K : R) || lora->ld_up < (up_kc ? R : N))
        return GEMM_ERR_INVALID_VALUE;
    if (!A || !B || !D || (beta != 0.0f && !C) || !lora->offsets || !lora->down || !lora->up)
        return GEMM_ERR_INVALID_VALUE;
    if (M > MAX_EXTENT || N > MAX_EXTENT || K > MAX_EXTENT || lda > INT_MAX || ldb > INT_MAX ||
        ldd > INT_MAX || (beta != 0.0f && ldc > INT_MAX) || lora->segments > MAX_GROUPS ||
        R > MAX_EXTENT / 2 || lora->ld_down > INT_MAX || lora->ld_up > INT_MAX)
        return GEMM_ERR_NOT_SUPPORTED;
    if (beta != 0.0f &&
        !c_d_ok(C, ((M - 1) * ldc + N) * eo, D, ((M - 1) * ldd + N) * eo, ldc == ldd))
        return GEMM_ERR_INVALID_VALUE;
    if (!ws || !aligned_to(ws, 256) || ws_bytes < gemm_lora_workspace_bytes(M, lora->rank))
        return GEMM_ERR_INVALID_VALUE;
    if (!aligned_to(A, es) || !aligned_to(B, es) || !aligned_to(lora->down, es) ||
        !aligned_to(lora->up, es))
        return GEMM_ERR_NOT_SUPPORTED;

    RaggedArgs a{};
    a.A = A;
    a.B = B;
    a.C = beta != 0.0f ? static_cast<const float*>(C) : nullptr;
    a.D = static_cast<float*>(D);
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = beta != 0.0f ? ldc : 0;
    a.ldd = ldd;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.alpha = alpha;
    a.beta = beta;
    a.c_vec = beta != 0.0f && aligned_to(C, eo);
    a.d_vec = aligned_to(D, eo);
    a.d_lines = aligned_to(D, 128) && ldd * eo % 128 == 0;
    a.offsets = lora->offsets;
    a.scales = lora->scales;
    a.groups = lora->segments;
    a.rows = (int)M;
    a.ids = lora->ids;
    a.adapters = lora->adapters;
    a.rank = lora->rank;
    a.rank_pad = (int)(ceil_div(R, LORA_PAD) * LORA_PAD);
    a.t = static_cast<const float*>(ws);
    a.up = lora->up;
    a.ld_up = lora->ld_up;
    a.stride_up = lora->stride_up;
    a.up_kc = up_kc;
    const double bytes = (double)es * K * (N + M) + (double)eo * M * N;
    const TileList tiles = dtype == GEMM_DTYPE_F32 ? tile_list(ragged_lora_f32, stream_lora_f32)
                                                   : tile_list(ragged_lora_bf16, stream_lora_bf16);
    auto grid_of = [&](const RaggedTile& x) { return ceil_div(M, x.bm) * ceil_div(N, x.bn[b_kc]); };
    const RaggedTile& t = pick_tile(h, tiles, b_kc, K, bytes, grid_of, grid_of);
    const int bn = t.bn[b_kc];
    const int64_t kk = K + t.bk;
    if (!panel_fits(t.bm - 1, lda, kk, es) ||
        !(b_kc ? panel_fits(bn - 1, ldb, kk, es) : panel_fits(kk, ldb, bn, es)))
        return GEMM_ERR_NOT_SUPPORTED;
    a.tiles_m = (int)ceil_div(M, t.bm);
    a.tiles_n = (int)ceil_div(N, bn);
    a.group_m = std::min(a.tiles_m, 4);
    const int64_t grid = grid_of(t);
    if (!grid_fits(grid, t.threads)) return GEMM_ERR_NOT_SUPPORTED;
    // One tile of rows and little to do for T: both products in one launch, whose
    // workgroups each go through all of down, a block of 16 ranks of an adapter
    // at a time, after W's.  Against two launches (1 to 16 rows, both layouts of
    // B): two blocks take 11.2 us for 14.5 at K, N = 1024, 11.8 for 16.3 at 2048,
    // 17.8 for 18.9 at 4096 and 35.5 for 35.5 at K = 4096, N = 14336, but 24.6 for
    // 20.1 at K = 8192, N = 2048 and 58.7 for 51.9 at N = 14336; one block takes
    // 17.8 for 19.6 and 51.4 for 50.9 there.
    const int64_t segs = std::min<int64_t>(lora->segments, M), t_blocks = segs * ceil_div(R, 16);
    if (t.stream && t.bm == 16 && M <= 16 && down_kc && R <= LORA_ONE_RANK && t_blocks <= 2 &&
        t_blocks * K <= 8192 && panel_fits(15, lora->ld_down, kk, es)) {
        int n_one = 0;
        const RaggedTile* one_launch =
            (dtype == GEMM_DTYPE_F32 ? stream_lora_one_f32 : stream_lora_one_bf16)(&n_one);
        const RaggedTile& ot = one_launch[t.bn[b_kc] < 64 ? 1 : 0];
        a.down = lora->down;
        a.ld_down = lora->ld_down;
        a.stride_down = lora->stride_down;
        if (h->fail_launch) return GEMM_ERR_HIP;
        if (ot.fn[b_kc][dtype == GEMM_DTYPE_BF16_BF16](a, (int)grid, stream) != hipSuccess)
            return GEMM_ERR_HIP;
        note_call(h, "lora in one launch", a, tiles, t, bn, grid);
        return GEMM_OK;
    }
    // the first product: blocks of as many rows as a segment has on average,
    // as narrow as the rank allows, and slices of K until there is a
    // workgroup per compute unit or a slice is two batches per wave
    RaggedArgs f = a;
    f.B = lora->down;
    f.ldb = lora->ld_down;
    f.stride_b = lora->stride_down;
    f.N = (int)R;
    f.C = nullptr;
    f.D = static_cast<float*>(ws);
    f.ldd = a.rank_pad;
    f.alpha = 1.0f;
    f.beta = 0.0f;
    f.group_m = 4;
    const int64_t avg = ceil_div(M, segs);
    int n_first = 0;
    const RaggedTile* first = (dtype == GEMM_DTYPE_F32 ? stream_shrink_f32 : stream_shrink_bf16)(&n_first);
    int fi = 0;
    while (fi + 1 < n_first &&
           ((fi + 2 < n_first && first[fi].bn[down_kc] < R) ||
            (first[fi].bm > 16 && (avg <= first[fi].bm / 2 || 2 * M < device_cus() * first[fi].bm))))
        ++fi;
    const RaggedTile& ft = first[fi];
    f.tiles_n = (int)ceil_div(R, ft.bn[down_kc]);
    const int64_t blocks = (M + segs * (ft.bm - 1)) / ft.bm * f.tiles_n;
    int64_t splits = std::min<int64_t>({4, ceil_div(device_cus(), blocks), ceil_div(8192, M),
                                        K / (8 * 4 * ft.bk)});
    // the direct-to-LDS tiles want T whole, for their K-steps
    splits = t.stream ? std::max<int64_t>(1, splits) : 1;
    a.terms = f.terms = dtype == GEMM_DTYPE_BF16_BF16 ? 2 : 3;
    if (!t.stream && dtype != GEMM_DTYPE_F32)
        a.t_terms = f.t_terms = reinterpret_cast<uint16_t*>(static_cast<float*>(ws) + M * a.rank_pad);
    f.k_slice = (int)(ceil_div(ceil_div(K, splits), ft.bk) * ft.bk);
    f.splits = a.splits = (int)ceil_div(K, f.k_slice);
    if (!grid_fits(blocks, ft.threads) ||
        !(down_kc ? panel_fits(ft.bn[1] - 1, f.ldb, kk, es) : panel_fits(kk, f.ldb, ft.bn[0], es)))
        return GEMM_ERR_NOT_SUPPORTED;
    if (h->fail_launch) return GEMM_ERR_HIP;
    if (ft.fn[down_kc][0](f, (int)blocks, stream) != hipSuccess ||
        t.fn[b_kc][dtype == GEMM_DTYPE_BF16_BF16](a, (int)grid, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    note_call(h, "lora", a, tiles, t, bn, grid, 2);
    h->last_group.first_rows = ft.bm;
    h->last_group.first_columns = ft.bn[down_kc];
    h->last_group.first_slices = f.splits;
    return GEMM_OK;
}

}  // extern "C"
