// Moving tokens' rows by the plan of their experts (route.hpp): token t's j-th
// choice is assignment a = t top + j, which has row position[a] among the rows
// sorted by expert, and row r has assignment order[r].
//
//   gather:   D[r] = w[order[r]] X[order[r] / top]          (w: 1 without weights)
//   combine:  D[t] = sum_j w[t,j] Y[position[t,j]] + beta C[t]
//   its gradient: dY[position[t,j]] = w[t,j] dD[t],  dw[t,j] = <Y[position[t,j]], dD[t]>
//
// All three are bound by the rows' bytes.  Combining by position, a token's sum
// formed where it is written and always in the order of j, needs no atomics and
// no zeroed output, and repeats exactly.
#pragma once

#include "common.hpp"

namespace dg {

struct RowsArgs {
    const void* X;          // gather: X; else Y
    const int32_t* index;   // gather: order; else position
    const float* weights;   // or null
    const void* C;          // combine: or null
    void* D;                // gather, combine: D; gradient: dY
    const void* dD;         // gradient
    float* dweights;
    int64_t ldx, ldc, ldd, ld_dd;
    int tokens, cols, top, rows;
    float beta;
};

// VEC elements from x as fp32, or (not FULL) n of them and zeros.  Every row but
// gather's is read once, and every one written once: those loads and stores are
// non-temporal (16384 rows of 4096 bf16 gathered 50.5 -> 39.6 us, their combination
// 60.2 -> 55.5; non-temporal loads of rows that are read twice cost 19 % there).
template <bool FULL, bool ONCE = true, int VEC, typename T>
__device__ __forceinline__ void load_row_vec(float (&v)[VEC], const T* x, int n)
{
    auto load = [](const auto* q) __attribute__((always_inline)) {
        if constexpr (ONCE) return __builtin_nontemporal_load(q);
        else return *q;
    };
    if constexpr (FULL) {
        constexpr int W = 16 / sizeof(T) < VEC ? 16 / sizeof(T) : VEC;  // elements per load
#pragma unroll
        for (int s = 0; s < VEC; s += W) {
            T e[W];
            if constexpr (W * sizeof(T) == 16) {
                const u32x4 r = load(reinterpret_cast<const u32x4_elem<T>*>(x + s));
                __builtin_memcpy(e, &r, 16);
            } else {
                const u16x4 r = load(reinterpret_cast<const u16x4_a2*>(x + s));
                __builtin_memcpy(e, &r, 8);
            }
#pragma unroll
            for (int i = 0; i < W; ++i) v[s + i] = to_f32(e[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = i < n ? to_f32(x[i]) : 0.0f;
    }
}

// VEC values to d, or (not FULL) n of them.
template <bool FULL, int VEC, typename T>
__device__ __forceinline__ void store_row_vec(T* d, const float (&v)[VEC], int n)
{
    if constexpr (FULL) {
        constexpr int W = 16 / sizeof(T) < VEC ? 16 / sizeof(T) : VEC;  // elements per store
#pragma unroll
        for (int s = 0; s < VEC; s += W) {
            T e[W];
#pragma unroll
            for (int i = 0; i < W; ++i) e[i] = from_f32<T>(v[s + i]);
            if constexpr (W * sizeof(T) == 16) {
                u32x4 r;
                __builtin_memcpy(&r, e, 16);
                __builtin_nontemporal_store(r, reinterpret_cast<u32x4_elem<T>*>(d + s));
            } else {
                u16x4 r;
                __builtin_memcpy(&r, e, 8);
                __builtin_nontemporal_store(r, reinterpret_cast<u16x4_a2*>(d + s));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < n) d[i] = from_f32<T>(v[i]);
    }
}

// A lane's row and first column: 1 << lanes_log lanes to a row, the workgroups of
// blockIdx.y each a part of its columns.
struct RowPlace {
    int64_t row;
    int col;
};
template <int VEC>
__device__ __forceinline__ RowPlace row_place(int lanes_log)
{
    const int lanes = 1 << lanes_log;
    return {(int64_t)blockIdx.x * (256 >> lanes_log) + (threadIdx.x >> lanes_log),
            (int)(blockIdx.y * lanes + (threadIdx.x & (lanes - 1))) * VEC};
}

// 16384 rows of 4096 bf16 from 8192: 39.6 us, 5.1 TB/s; few rows a launch.
template <typename T, typename OutT>
__global__ __launch_bounds__(256) void gather_rows_kernel(RowsArgs p, int lanes_log)
{
    constexpr int VEC = 16 / sizeof(T);
    const RowPlace at = row_place<VEC>(lanes_log);
    if (at.row >= p.rows || at.col >= p.cols) return;
    const int a = p.index[at.row];
    if (a < 0 || a >= p.tokens * p.top) return;
    const float w = p.weights ? p.weights[a] : 1.0f;
    const T* x = static_cast<const T*>(p.X) + (int64_t)(a / p.top) * p.ldx + at.col;
    OutT* d = static_cast<OutT*>(p.D) + at.row * p.ldd + at.col;
    const int n = p.cols - at.col;
    auto move = [&](auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        float v[VEC];
        load_row_vec<FULL, false>(v, x, n);
        if (p.weights) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] *= w;
        }
        store_row_vec<FULL>(d, v, n);
    };
    if (n >= VEC) move(std::true_type{});
    else move(std::false_type{});
}

// JB of a token's rows at a time, all of them asked for before the first is used.
// JB divides `top` as well as it can (pick_batch): a row too many is read as one
// that is there already, and is not free (two rows of 4096 bf16 a token: 55 us in
// batches of 4, 48 in batches of 2).
template <typename T, typename OutT, int JB>
__global__ __launch_bounds__(256) void combine_rows_kernel(RowsArgs p, int lanes_log)
{
    constexpr int VEC = 16 / sizeof(T);
    const RowPlace at = row_place<VEC>(lanes_log);
    if (at.row >= p.tokens || at.col >= p.cols) return;
    const int n = p.cols - at.col;
    const T* Y = static_cast<const T*>(p.X) + at.col;
    const int64_t a0 = at.row * p.top;
    const int top = p.rows > 0 ? p.top : 0;
    auto sum_up = [&](auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        float sum[VEC] = {};
        for (int j0 = 0; j0 < top; j0 += JB) {
            float y[JB][VEC], w[JB];
            bool in[JB];
            // (a row that is not there is read as row 0 and dropped: loads in
            // branches would be waited for one by one)
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                const int64_t a = a0 + (j0 + j < top ? j0 + j : 0);
                const int r = p.index[a];
                in[j] = j0 + j < top && r >= 0 && r < p.rows;
                w[j] = p.weights ? p.weights[a] : 1.0f;
                load_row_vec<FULL>(y[j], Y + (in[j] ? r : 0) * p.ldx, n);
            }
#pragma unroll
            for (int j = 0; j < JB; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum[i] += in[j] ? w[j] * y[j][i] : 0.0f;
        }
        if (p.C) {
            float c[VEC];
            load_row_vec<FULL>(c, static_cast<const OutT*>(p.C) + at.row * p.ldc + at.col, n);
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[i] += p.beta * c[i];
        }
        store_row_vec<FULL>(static_cast<OutT*>(p.D) + at.row * p.ldd + at.col, sum, n);
    };
    if (n >= VEC) sum_up(std::true_type{});
    else sum_up(std::false_type{});
}

// A workgroup per token, JB of its rows at a time.  dD, read again for each JB of
// them, is loaded in the ordinary way: 4096 tokens of 4096 bf16, 8 rows each 119 ->
// 110 us (5.2 TB/s), 5 rows 79 -> 70, and of 2 no slower (8192 tokens 65 -> 64).
template <typename T, typename OutT, int JB>
__global__ __launch_bounds__(256) void combine_rows_grad_kernel(RowsArgs p)
{
    constexpr int VEC = 16 / sizeof(T);
    __shared__ float part[4][JB];
    const int64_t a0 = (int64_t)blockIdx.x * p.top;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const OutT* dD = static_cast<const OutT*>(p.dD) + blockIdx.x * p.ld_dd;
    for (int j0 = 0; j0 < p.top; j0 += JB) {
        int64_t row[JB];
        float w[JB], dot[JB] = {};
        bool in[JB];
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const int64_t a = a0 + (j0 + j < p.top ? j0 + j : 0);
            const int r = p.index[a];
            in[j] = j0 + j < p.top && r >= 0 && r < p.rows;
            row[j] = in[j] ? r : 0;
            w[j] = p.weights[a];
        }
        auto piece = [&](auto full, int col, int n) __attribute__((always_inline)) {
            constexpr bool FULL = decltype(full)::value;
            float d[VEC], y[JB][VEC];
            load_row_vec<FULL, false>(d, dD + col, n);
            if (p.rows > 0) {
#pragma unroll
                for (int j = 0; j < JB; ++j)
                    load_row_vec<FULL>(y[j], static_cast<const T*>(p.X) + row[j] * p.ldx + col, n);
            }
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                if (!in[j]) continue;
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    dot[j] += y[j][i] * d[i];
                    o[i] = w[j] * d[i];
                }
                store_row_vec<FULL>(static_cast<T*>(p.D) + row[j] * p.ldd + col, o, n);
            }
        };
        for (int col = tid * VEC; col < p.cols; col += 256 * VEC) {
            if (p.cols - col >= VEC) piece(std::true_type{}, col, VEC);
            else piece(std::false_type{}, col, p.cols - col);
        }
#pragma unroll
        for (int j = 0; j < JB; ++j) {
#pragma unroll
            for (int s = 1; s < 64; s *= 2) dot[j] += __shfl_xor(dot[j], s);
            if (lane == 0) part[wave][j] = dot[j];
        }
        __syncthreads();
        if (tid < JB && j0 + tid < p.top)
            p.dweights[a0 + j0 + tid] = part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid];
        __syncthreads();
    }
}

}  // namespace dg
