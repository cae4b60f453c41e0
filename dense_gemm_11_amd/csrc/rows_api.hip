// C ABI of the calls that move rows by a routing's plan: argument validation and
// launches.  Declared in include/dense_gemm.h.
#include <climits>
#include <cstdio>

#include "handle.hpp"
#include "rows.hpp"

namespace dg {
namespace {

// Element sizes of operands and outputs (0: no such type).
int64_t in_bytes(gemm_dtype_t t)
{
    return t == GEMM_DTYPE_F32 ? 4 : t == GEMM_DTYPE_BF16_F32 || t == GEMM_DTYPE_BF16_BF16 ? 2 : 0;
}
int64_t out_bytes(gemm_dtype_t t) { return t == GEMM_DTYPE_BF16_BF16 ? 2 : 4; }

// What the calls refuse alike: tokens x top assignments and `rows` rows of cols
// columns, with the numbers that the kernels hold in 32 bits.
gemm_status_t check_rows(gemm_handle_t h, int64_t tokens, int64_t cols, int top, int64_t rows,
                         gemm_dtype_t dtype)
{
    if (!h || tokens < 0 || cols < 0 || rows < 0 || top < 1 || in_bytes(dtype) == 0)
        return GEMM_ERR_INVALID_VALUE;
    return GEMM_OK;
}
// (a launch has a workgroup of 256 threads to a row or token at the most, below
// 2^32 threads, and along its second axis one to 1024 columns, below 2^16)
bool rows_fit(int64_t tokens, int64_t cols, int top, int64_t rows)
{
    return tokens < (1 << 24) && rows < (1 << 24) && tokens * top <= INT_MAX && cols <= 65535 * 1024;
}

bool matrix_ok(const void* p, int64_t es) { return aligned_to(p, es); }

int64_t span(int64_t rows, int64_t ld, int64_t cols, int64_t es)
{
    return rows > 0 ? ((rows - 1) * ld + cols) * es : 0;
}

typedef void (*MoveFn)(RowsArgs, int);

// One launch over `rows` rows of cols columns: as many lanes to a row as it has
// vectors, 16 to 256, and the workgroups along y for what is left.
hipError_t launch_move(MoveFn fn, const RowsArgs& a, int64_t rows, int vec, hipStream_t stream)
{
    RowsArgs copy = a;
    int lanes_log = 4;
    while (lanes_log < 8 && ((int64_t)vec << lanes_log) < a.cols) ++lanes_log;
    void* args[] = {&copy, &lanes_log};
    return hipLaunchKernel(reinterpret_cast<const void*>(fn),
                           dim3((unsigned)ceil_div(rows, 256 >> lanes_log),
                                (unsigned)ceil_div(a.cols, (int64_t)vec << lanes_log)),
                           dim3(256), args, 0, stream);
}

// Rows of a token to take at a time, 1 to 4: those with the fewest too many (one too
// many rather than each alone), of these the most.
int pick_batch(int top)
{
    int best = 1;
    for (int b = 2; b <= 4; ++b)
        if (ceil_div(top, b) * b <= ceil_div(top, best) * best + (best == 1 && top > 4 ? 1 : 0)) best = b;
    return best;
}

MoveFn gather_fn(gemm_dtype_t t)
{
    return t == GEMM_DTYPE_F32        ? gather_rows_kernel<float, float>
           : t == GEMM_DTYPE_BF16_F32 ? gather_rows_kernel<bf16_t, float>
                                      : gather_rows_kernel<bf16_t, bf16_t>;
}
template <typename T, typename O>
MoveFn combine_fn(int batch)
{
    return batch == 1   ? combine_rows_kernel<T, O, 1>
           : batch == 2 ? combine_rows_kernel<T, O, 2>
           : batch == 3 ? combine_rows_kernel<T, O, 3>
                        : combine_rows_kernel<T, O, 4>;
}
typedef void (*GradFn)(RowsArgs);
template <typename T, typename O>
GradFn combine_grad_fn(int batch)
{
    return batch == 1   ? combine_rows_grad_kernel<T, O, 1>
           : batch == 2 ? combine_rows_grad_kernel<T, O, 2>
           : batch == 3 ? combine_rows_grad_kernel<T, O, 3>
                        : combine_rows_grad_kernel<T, O, 4>;
}

}  // namespace
}  // namespace dg

extern "C" {

gemm_status_t gemm_gather_rows(gemm_handle_t h, int64_t tokens, int64_t cols, int top, const void* X,
                               int64_t ldx, int64_t rows, const int32_t* order, const float* weights,
                               void* D, int64_t ldd, gemm_dtype_t dtype, hipStream_t stream)
{
    using namespace dg;
    const gemm_status_t st = check_rows(h, tokens, cols, top, rows, dtype);
    if (st != GEMM_OK) return st;
    const int64_t es = in_bytes(dtype), eo = out_bytes(dtype);
    if (ldx < cols || ldd < cols) return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0 || cols == 0 || rows == 0) return GEMM_OK;
    if (!X || !order || !D) return GEMM_ERR_INVALID_VALUE;
    if (!rows_fit(tokens, cols, top, rows) || ldx > INT_MAX || ldd > INT_MAX) return GEMM_ERR_NOT_SUPPORTED;
    if (written_overlap({{D, span(rows, ldd, cols, eo)}, {X, span(tokens, ldx, cols, es)}, {order, rows * 4},
                         {weights, tokens * top * 4}}, 1))
        return GEMM_ERR_INVALID_VALUE;
    if (!matrix_ok(X, es) || !matrix_ok(D, eo) || !aligned_to(order, 4) || !aligned_to(weights, 4))
        return GEMM_ERR_NOT_SUPPORTED;
    RowsArgs a{};
    a.X = X;
    a.index = order;
    a.weights = weights;
    a.D = D;
    a.ldx = ldx;
    a.ldd = ldd;
    a.tokens = (int)tokens;
    a.cols = (int)cols;
    a.top = top;
    a.rows = (int)rows;
    if (h->fail_launch) return GEMM_ERR_HIP;
    if (launch_move(gather_fn(dtype), a, rows, (int)(16 / es), stream) != hipSuccess)
        return GEMM_ERR_HIP;
    if (h->log)
        std::fprintf(stderr, "gemm: gather rows=%d tokens=%d cols=%d\n", a.rows, a.tokens, a.cols);
    return GEMM_OK;
}

gemm_status_t gemm_combine_rows(gemm_handle_t h, int64_t tokens, int64_t cols, int top, const void* Y,
                                int64_t ldy, int64_t rows, const int32_t* position,
                                const float* weights, float beta, const void* C, int64_t ldc, void* D,
                                int64_t ldd, gemm_dtype_t dtype, hipStream_t stream)
{
    using namespace dg;
    const gemm_status_t st = check_rows(h, tokens, cols, top, rows, dtype);
    if (st != GEMM_OK) return st;
    const int64_t es = in_bytes(dtype), eo = out_bytes(dtype);
    if (ldy < cols || ldd < cols || (beta != 0.0f && ldc < cols)) return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0 || cols == 0) return GEMM_OK;
    if ((rows > 0 && !Y) || !position || !D || (beta != 0.0f && !C)) return GEMM_ERR_INVALID_VALUE;
    if (!rows_fit(tokens, cols, top, rows) || ldy > INT_MAX || ldd > INT_MAX ||
        (beta != 0.0f && ldc > INT_MAX))
        return GEMM_ERR_NOT_SUPPORTED;
    const int64_t span_d = span(tokens, ldd, cols, eo);
    if (written_overlap({{D, span_d}, {Y, span(rows, ldy, cols, es)}, {position, tokens * top * 4},
                         {weights, tokens * top * 4}}, 1) ||
        (beta != 0.0f && (C == D ? ldc != ldd : ranges_overlap(C, span(tokens, ldc, cols, eo), D, span_d))))
        return GEMM_ERR_INVALID_VALUE;
    if (!matrix_ok(Y, es) || !matrix_ok(D, eo) || (beta != 0.0f && !matrix_ok(C, eo)) ||
        !aligned_to(position, 4) || !aligned_to(weights, 4))
        return GEMM_ERR_NOT_SUPPORTED;
    RowsArgs a{};
    a.X = Y;
    a.index = position;
    a.weights = weights;
    a.C = beta != 0.0f ? C : nullptr;
    a.D = D;
    a.ldx = ldy;
    a.ldc = ldc;
    a.ldd = ldd;
    a.tokens = (int)tokens;
    a.cols = (int)cols;
    a.top = top;
    a.rows = (int)rows;
    a.beta = beta;
    if (h->fail_launch) return GEMM_ERR_HIP;
    const int batch = pick_batch(top);
    const MoveFn fn = dtype == GEMM_DTYPE_F32        ? combine_fn<float, float>(batch)
                      : dtype == GEMM_DTYPE_BF16_F32 ? combine_fn<bf16_t, float>(batch)
                                                     : combine_fn<bf16_t, bf16_t>(batch);
    if (launch_move(fn, a, tokens, (int)(16 / es), stream) != hipSuccess)
        return GEMM_ERR_HIP;
    if (h->log)
        std::fprintf(stderr, "gemm: combine rows=%d tokens=%d cols=%d\n", a.rows, a.tokens, a.cols);
    return GEMM_OK;
}

gemm_status_t gemm_combine_rows_grad(gemm_handle_t h, int64_t tokens, int64_t cols, int top,
                                     const void* Y, int64_t ldy, int64_t rows, const int32_t* position,
                                     const float* weights, const void* dD, int64_t lddd, void* dY,
                                     int64_t lddy, float* dweights, gemm_dtype_t dtype,
                                     hipStream_t stream)
{
    using namespace dg;
    const gemm_status_t st = check_rows(h, tokens, cols, top, rows, dtype);
    if (st != GEMM_OK) return st;
    const int64_t es = in_bytes(dtype), eo = out_bytes(dtype);
    if (ldy < cols || lddd < cols || lddy < cols) return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0) return GEMM_OK;
    if (!position || !weights || !dweights || (cols > 0 && (!dD || (rows > 0 && (!Y || !dY)))))
        return GEMM_ERR_INVALID_VALUE;
    if (!rows_fit(tokens, cols, top, rows) || ldy > INT_MAX || lddd > INT_MAX || lddy > INT_MAX)
        return GEMM_ERR_NOT_SUPPORTED;
    const int64_t span_dy = span(rows, lddy, cols, es);
    if (rows > 0 && cols > 0 &&
        ((Y == dY ? ldy != lddy : ranges_overlap(Y, span(rows, ldy, cols, es), dY, span_dy)) ||
         ranges_overlap(dD, span(tokens, lddd, cols, eo), dY, span_dy)))
        return GEMM_ERR_INVALID_VALUE;
    const int64_t assigned = tokens * top * 4;
    if (written_overlap({{dweights, assigned}, {cols > 0 ? dY : nullptr, span_dy}, {position, assigned},
                         {weights, assigned}, {cols > 0 ? Y : nullptr, span(rows, ldy, cols, es)},
                         {cols > 0 ? dD : nullptr, span(tokens, lddd, cols, eo)}}, 1) ||
        written_overlap({{cols > 0 ? dY : nullptr, span_dy}, {position, assigned}, {weights, assigned}}, 1))
        return GEMM_ERR_INVALID_VALUE;
    if (!matrix_ok(Y, es) || !matrix_ok(dY, es) || !matrix_ok(dD, eo) || !aligned_to(position, 4) ||
        !aligned_to(weights, 4) || !aligned_to(dweights, 4))
        return GEMM_ERR_NOT_SUPPORTED;
    RowsArgs a{};
    a.X = Y;
    a.index = position;
    a.weights = weights;
    a.D = dY;
    a.dD = dD;
    a.dweights = dweights;
    a.ldx = ldy;
    a.ldd = lddy;
    a.ld_dd = lddd;
    a.tokens = (int)tokens;
    a.cols = (int)cols;
    a.top = top;
    a.rows = (int)rows;
    if (h->fail_launch) return GEMM_ERR_HIP;
    const int batch = pick_batch(top);
    const GradFn fn = dtype == GEMM_DTYPE_F32        ? combine_grad_fn<float, float>(batch)
                      : dtype == GEMM_DTYPE_BF16_F32 ? combine_grad_fn<bf16_t, float>(batch)
                                                     : combine_grad_fn<bf16_t, bf16_t>(batch);
    void* args[] = {&a};
    if (hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)tokens),
                        dim3(256), args, 0, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    if (h->log)
        std::fprintf(stderr, "gemm: combine grad rows=%d tokens=%d cols=%d\n", a.rows, a.tokens, a.cols);
    return GEMM_OK;
}

}  // extern "C"
