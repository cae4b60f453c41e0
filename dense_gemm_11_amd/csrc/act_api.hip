// C ABI of the products with bias, activation, gate and residual and of their
// gradient: argument validation, tile choice and launches.  Declared in
// include/dense_gemm.h.
#include <algorithm>
#include <climits>
#include <cstdio>

#include "act_grad.hpp"
#include "act_variants.hpp"
#include "tile_choice.hpp"

namespace dg {
namespace {

bool known(gemm_dtype_t t)
{
    return t == GEMM_DTYPE_F32 || t == GEMM_DTYPE_BF16_F32 || t == GEMM_DTYPE_BF16_BF16;
}
bool known(gemm_activation_t a)
{
    return a == GEMM_ACT_NONE || a == GEMM_ACT_RELU || a == GEMM_ACT_GELU || a == GEMM_ACT_SILU ||
           a == GEMM_ACT_GELU_TANH;
}
static_assert((int)GEMM_ACT_SILU == EPI_ACT_SILU && (int)GEMM_ACT_GELU_TANH == EPI_ACT_GELU_TANH &&
                  (int)GEMM_ACT_GELU == EPI_ACT_GELU && (int)GEMM_ACT_RELU == EPI_ACT_RELU,
              "the kernels' numbers");

// Bytes of a matrix of rows x cols.
int64_t span(int64_t rows, int64_t ld, int64_t cols, int64_t es) { return ((rows - 1) * ld + cols) * es; }

// The same matrix in the same places, or disjoint ones.
bool in_place_or_apart(const void* x, int64_t span_x, const void* y, int64_t span_y, bool same)
{
    return x == y ? same : !ranges_overlap(x, span_x, y, span_y);
}

typedef void (*GradFn)(ActGradArgs);
GradFn grad_fn(gemm_dtype_t t, bool gated)
{
    if (t == GEMM_DTYPE_F32) return gated ? act_grad_kernel<float, float, true> : act_grad_kernel<float, float, false>;
    if (t == GEMM_DTYPE_BF16_F32)
        return gated ? act_grad_kernel<bf16_t, float, true> : act_grad_kernel<bf16_t, float, false>;
    return gated ? act_grad_kernel<bf16_t, bf16_t, true> : act_grad_kernel<bf16_t, bf16_t, false>;
}

// Rows of tiles that any split of M rows into groups needs at the most.
int64_t grad_tiles(int64_t M, int64_t groups)
{
    return (M + std::min(M, groups) * (ACT_GRAD_ROWS - 1)) / ACT_GRAD_ROWS;
}

}  // namespace
}  // namespace dg

extern "C" {

gemm_status_t gemm_run_grouped_act(gemm_handle_t h, gemm_op_t transB, int64_t M, int64_t N, int64_t K,
                                   float alpha, const void* A, int64_t lda, const void* B, int64_t ldb,
                                   int64_t strideB, void* D, int64_t ldd, gemm_dtype_t dtype,
                                   const gemm_groups_t* groups, const gemm_act_t* act,
                                   hipStream_t stream)
{
    using namespace dg;
    if (!h || (transB != GEMM_OP_N && transB != GEMM_OP_T) || !known(dtype) || M < 0 || N < 0 || K < 0)
        return GEMM_ERR_INVALID_VALUE;
    if (!act || !known(act->activation) || strideB < 0 || (groups && groups->groups < 0) ||
        act->stride_bias < 0)
        return GEMM_ERR_INVALID_VALUE;
    const int64_t one = 1, G = groups ? groups->groups : 1, halves = act->gated ? 2 : 1;
    const int64_t es = dtype == GEMM_DTYPE_F32 ? 4 : 2, eo = dtype == GEMM_DTYPE_BF16_BF16 ? 2 : 4;
    const bool b_kc = transB == GEMM_OP_T;
    if (N > MAX_EXTENT / 2) return GEMM_ERR_NOT_SUPPORTED;
    const int64_t width = halves * N;
    if (lda < std::max(one, K) || ldb < std::max(one, b_kc ? K : width) || ldd < std::max(one, N) ||
        (act->Z && act->ldz < std::max(one, width)) || (act->R && act->ldr < std::max(one, N)))
        return GEMM_ERR_INVALID_VALUE;
    h->last_group = {};
    if (M == 0 || N == 0 || G == 0) return GEMM_OK;
    const bool reads_ab = K > 0 && alpha != 0.0f;
    if ((groups && !groups->offsets) || !D || (reads_ab && (!A || !B))) return GEMM_ERR_INVALID_VALUE;
    if (M > MAX_EXTENT || K > MAX_EXTENT || lda > INT_MAX || ldb > INT_MAX || ldd > INT_MAX ||
        (act->Z && act->ldz > INT_MAX) || (act->R && act->ldr > INT_MAX) || G > MAX_GROUPS)
        return GEMM_ERR_NOT_SUPPORTED;
    // D may be R; Z lies apart from both, and the bias from what is written
    const int64_t span_d = span(M, ldd, N, eo), span_z = act->Z ? span(M, act->ldz, width, eo) : 0;
    const int64_t span_r = act->R ? span(M, act->ldr, N, eo) : 0;
    const int64_t span_b = act->bias ? ((G - 1) * act->stride_bias + width) * eo : 0;
    if ((act->R && !in_place_or_apart(act->R, span_r, D, span_d, act->ldr == ldd)) ||
        (act->Z && (ranges_overlap(act->Z, span_z, D, span_d) ||
                    (act->R && ranges_overlap(act->Z, span_z, act->R, span_r)) ||
                    (act->bias && ranges_overlap(act->Z, span_z, act->bias, span_b)))) ||
        (act->bias && ranges_overlap(act->bias, span_b, D, span_d)))
        return GEMM_ERR_INVALID_VALUE;
    if ((reads_ab && (!aligned_to(A, es) || !aligned_to(B, es))) || !aligned_to(D, eo) ||
        !aligned_to(act->Z, eo) || !aligned_to(act->R, eo) || !aligned_to(act->bias, eo) ||
        (groups && (!aligned_to(groups->offsets, 4) || !aligned_to(groups->scales, 4))))
        return GEMM_ERR_NOT_SUPPORTED;

    ActArgs a{};
    a.A = A;
    a.B = B;
    a.D = static_cast<float*>(D);
    a.lda = lda;
    a.ldb = ldb;
    a.ldd = ldd;
    a.M = (int)M;
    a.N = (int)N;
    a.K = reads_ab ? (int)K : 0;  // no K-steps: Z = bias
    a.alpha = reads_ab ? alpha : 0.0f;
    a.act = (int)act->activation;
    a.offsets = groups ? groups->offsets : nullptr;
    a.scales = reads_ab && groups ? groups->scales : nullptr;
    a.groups = (int)G;
    a.rows = (int)M;
    a.stride_b = strideB;
    a.z_bias = act->bias;
    a.stride_bias = act->stride_bias;
    a.Z = act->Z;
    a.ldz = act->ldz;
    a.R = act->R;
    a.ldr = act->ldr;
    // a group holds M / G rows on average, and the host knows no more
    const int64_t busy = std::min(G, M);
    const double bytes = (double)es * K * ((double)busy * width + M) +
                         (double)eo * M * (N * (act->R ? 2 : 1) + (act->Z ? width : 0));
    const auto tiles =
        dtype == GEMM_DTYPE_F32
            ? (act->gated ? tile_list(gate_tiles_f32, stream_gate_f32) : tile_list(act_tiles_f32, stream_act_f32))
            : (act->gated ? tile_list(gate_tiles_bf16, stream_gate_bf16)
                          : tile_list(act_tiles_bf16, stream_act_bf16));
    auto outputs = [&](const ActTile& x) { return x.bn[b_kc] / halves; };  // a tile's columns of D
    auto grid_of = [&](const ActTile& x) {
        return (M + (groups ? busy : 1) * (x.bm - 1)) / x.bm * ceil_div(N, outputs(x));
    };
    const ActTile& t = pick_tile(h, tiles, b_kc, K, bytes, [&](const ActTile& x) {
        return ceil_div(N, outputs(x)) *
               (busy > 1 ? row_tiles((double)busy, (double)M / busy, x.bm) : (double)ceil_div(M, x.bm));
    }, grid_of);
    const int64_t bn = outputs(t), far = (halves - 1) * N, kk = K + t.bk;
    if (!panel_fits(t.bm - 1, lda, kk, es) ||
        !(b_kc ? panel_fits(far + bn - 1, ldb, kk, es) : panel_fits(kk, ldb, far + bn, es)))
        return GEMM_ERR_NOT_SUPPORTED;
    a.tiles_n = (int)ceil_div(N, bn);
    // tiles go down 12 rows of them before the next column, so that most groups read
    // each column of B at once (8 groups of 2048 rows, 4096 x 14336 gated bf16, by 4
    // and 12 rows: 3.31 and 3.24 ms, n-contiguous 3.27 and 3.18); one matrix, whose A
    // is read by more columns the fewer rows there are, 4 (2.99 ms, by 12 3.03)
    a.group_m = groups ? 12 : 4;
    const int64_t grid = grid_of(t);
    if (!grid_fits(grid, t.threads)) return GEMM_ERR_NOT_SUPPORTED;
    if (h->fail_launch) return GEMM_ERR_HIP;
    if (t.fn[b_kc][dtype == GEMM_DTYPE_BF16_BF16](a, (int)grid, stream) != hipSuccess) return GEMM_ERR_HIP;
    int i = 0;
    while (&tiles[i] != &t) ++i;
    h->last_group = gemm_group_launch_t{t.bm, (int)bn, nth_of_height(tiles, i), 1, 0, 0, 0};
    if (h->log)
        std::fprintf(stderr, "gemm: grouped act %dx%d gated=%d rows=%d groups=%d N=%d K=%d grid=%lld\n", t.bm,
                     (int)bn, act->gated != 0, a.rows, a.groups, a.N, a.K, (long long)grid);
    return GEMM_OK;
}

size_t gemm_act_grad_workspace_bytes(int64_t M, int64_t width, int groups)
{
    using namespace dg;
    if (M <= 0 || width <= 0 || groups <= 0) return 0;
    return (size_t)(grad_tiles(M, groups) * width + groups) * 4;
}

gemm_status_t gemm_run_grouped_act_grad(gemm_handle_t h, int64_t M, int64_t N,
                                        gemm_activation_t activation, int gated, const void* Z,
                                        int64_t ldz, const void* dD, int64_t lddd, void* dZ,
                                        int64_t lddz, void* H, int64_t ldh, float* dbias,
                                        gemm_dtype_t dtype, const gemm_groups_t* groups, void* ws,
                                        size_t ws_bytes, hipStream_t stream)
{
    using namespace dg;
    if (!h || !known(dtype) || !known(activation) || M < 0 || N < 0 || (groups && groups->groups < 0))
        return GEMM_ERR_INVALID_VALUE;
    const int64_t one = 1, G = groups ? groups->groups : 1, halves = gated ? 2 : 1;
    const int64_t es = dtype == GEMM_DTYPE_F32 ? 4 : 2, eo = dtype == GEMM_DTYPE_BF16_BF16 ? 2 : 4;
    if (N > MAX_EXTENT / 2) return GEMM_ERR_NOT_SUPPORTED;
    const int64_t width = halves * N;
    if (ldz < std::max(one, width) || lddd < std::max(one, N) || lddz < std::max(one, width) ||
        (H && ldh < std::max(one, N)))
        return GEMM_ERR_INVALID_VALUE;
    if (N == 0 || G == 0 || (M == 0 && !dbias)) return GEMM_OK;
    if ((groups && !groups->offsets) || (M > 0 && (!Z || !dD || !dZ))) return GEMM_ERR_INVALID_VALUE;
    if (M > MAX_EXTENT || ldz > INT_MAX || lddd > INT_MAX || lddz > INT_MAX || (H && ldh > INT_MAX) ||
        G > MAX_GROUPS)
        return GEMM_ERR_NOT_SUPPORTED;
    const size_t needed = dbias && M > 0 ? gemm_act_grad_workspace_bytes(M, width, (int)G) : 0;
    if (needed && (!ws || !aligned_to(ws, 256) || ws_bytes < needed)) return GEMM_ERR_INVALID_VALUE;
    // dZ may be Z and H may be dD, of one type; else what is written lies apart
    const int64_t sz = M > 0 ? span(M, ldz, width, eo) : 0, sd = M > 0 ? span(M, lddd, N, eo) : 0;
    const int64_t so = M > 0 ? span(M, lddz, width, es) : 0, sh = M > 0 && H ? span(M, ldh, N, es) : 0;
    const MemoryRange off{groups ? groups->offsets : nullptr, (G + 1) * 4};
    if (M > 0 && (!in_place_or_apart(Z, sz, dZ, so, ldz == lddz && es == eo) ||
                  (H && !in_place_or_apart(dD, sd, H, sh, lddd == ldh && es == eo)) ||
                  written_overlap({{dZ, so}, {H, sh}, {dD, sd}, off}, 1) ||
                  written_overlap({{H, sh}, {Z, sz}, off}, 1)))
        return GEMM_ERR_INVALID_VALUE;
    if (written_overlap({{dbias, G * width * 4}, {needed ? ws : nullptr, (int64_t)needed}, {dZ, so}, {H, sh},
                         {Z, sz}, {dD, sd}, off}, 2))
        return GEMM_ERR_INVALID_VALUE;
    if (!aligned_to(Z, eo) || !aligned_to(dD, eo) || !aligned_to(dZ, es) || !aligned_to(H, es) ||
        !aligned_to(dbias, 4) || (groups && !aligned_to(groups->offsets, 4)))
        return GEMM_ERR_NOT_SUPPORTED;

    ActGradArgs a{};
    a.Z = Z;
    a.dD = dD;
    a.dZ = dZ;
    a.H = H;
    a.ldz = ldz;
    a.ld_dd = lddd;
    a.ld_dz = lddz;
    a.ldh = ldh;
    a.M = a.rows = (int)M;
    a.N = (int)N;
    a.width = (int)width;
    a.act = (int)activation;
    a.offsets = groups ? groups->offsets : nullptr;
    a.groups = (int)G;
    a.dbias = dbias;
    const int64_t tile_rows = groups ? grad_tiles(M, G) : ceil_div(M, ACT_GRAD_ROWS);
    if (dbias && M > 0) {
        a.sums = static_cast<float*>(ws);
        a.tile_rows = (int)grad_tiles(M, G);
        a.firsts = reinterpret_cast<int32_t*>(a.sums + grad_tiles(M, G) * width);
    }
    a.tiles_n = (int)ceil_div(N, 64 * (16 / es));
    const int64_t grid = tile_rows * a.tiles_n;
    if (!grid_fits(grid, 256) || ceil_div(width, 64) * 256 >= (int64_t)1 << 32) return GEMM_ERR_NOT_SUPPORTED;
    if (h->fail_launch) return GEMM_ERR_HIP;
    void* args[] = {&a};
    if (M > 0 && hipLaunchKernel(reinterpret_cast<const void*>(grad_fn(dtype, gated)), dim3((unsigned)grid),
                                 dim3(256), args, 0, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    if (dbias && hipLaunchKernel(reinterpret_cast<const void*>(act_bias_kernel<4>),
                                 dim3((unsigned)ceil_div(width, 64), (unsigned)std::min<int64_t>(G, 65535)),
                                 dim3(256), args, 0, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    if (h->log)
        std::fprintf(stderr, "gemm: grouped act grad gated=%d rows=%d groups=%d N=%d\n", gated != 0, a.rows,
                     a.groups, a.N);
    return GEMM_OK;
}

}  // extern "C"
