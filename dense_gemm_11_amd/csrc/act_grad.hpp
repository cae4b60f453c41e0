// Gradient of bias, activation and gate (act.hpp) from the kept Z:
//     dZ = dD act'(Z)                                            , H = act(Z)
//     gated, Z = [G U]: dZ = [dD U act'(G), dD act(G)]           , H = act(G) U
// and the bias's, the sums of dZ's columns over each group's rows, taken before
// dZ is rounded.
//
// One pass, bound by the bytes: a workgroup takes 16 rows of one group by 64
// vectors of columns, its waves every fourth row, all asked for at once.  A lane
// sums its columns down its rows in registers, the waves' sums meet in LDS, and
// each tile's go to a row of the workspace that a second, small launch adds up in
// order: no atomics, so the sums repeat exactly.  16 rows, since the fewer the more
// workgroups there are to share the card out evenly (8192 rows, 2 x 5632 columns of
// 16 groups, gated bf16 with H and dbias, 64, 32, 16 and 8 rows: 118, 112, 107 and
// 116 us, 5.2 TB/s with 16, where the sums' way through memory begins to tell).
#pragma once

#include "act.hpp"
#include "rows.hpp"

namespace dg {

constexpr int ACT_GRAD_ROWS = 16;

struct ActGradArgs : RaggedArgs {
    const void* Z;
    const void* dD;
    void* dZ;
    void* H;           // or null
    float* sums;       // tile rows x width, or null
    int32_t* firsts;   // each group's first row of tiles (groups with rows)
    float* dbias;
    int64_t ldz, ld_dd, ld_dz, ldh;
    int width;
    int tile_rows;     // of sums
};

template <typename T, typename OutT, bool GATE>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs p)
{
    constexpr int VEC = 16 / sizeof(T), COLS = 64 * VEC, WAVES = 4, U = 4;
    constexpr bool PRECISE = sizeof(T) == 4;
    constexpr int HALVES = GATE ? 2 : 1;
    __shared__ float part[WAVES - 1][HALVES * VEC][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    RowTile t;
    if (!find_act_tile<ACT_GRAD_ROWS>(p, p.tiles_n, t)) return;
    const int tm = t.in_group / p.tiles_n, tn = t.in_group - tm * p.tiles_n;
    const int left = t.size - tm * ACT_GRAD_ROWS, rows = left < ACT_GRAD_ROWS ? left : ACT_GRAD_ROWS;
    const int64_t row0 = t.start + tm * ACT_GRAD_ROWS;
    const int col = tn * COLS + lane * VEC, n = p.N - col;
    float sum[HALVES][VEC] = {};
    auto work = [&](auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        for (int r0 = wave; r0 < rows; r0 += WAVES * U) {
            float z[U][HALVES][VEC], d[U][VEC];
            // (past the last row: that row again, and nothing of it is kept)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = row0 + (r0 + u * WAVES < rows ? r0 + u * WAVES : r0);
                const OutT* zr = static_cast<const OutT*>(p.Z) + row * p.ldz + col;
#pragma unroll
                for (int h = 0; h < HALVES; ++h) load_row_vec<FULL>(z[u][h], zr + (int64_t)h * p.N, n);
                load_row_vec<FULL>(d[u], static_cast<const OutT*>(p.dD) + row * p.ld_dd + col, n);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r0 + u * WAVES >= rows) break;
                const int64_t row = row0 + r0 + u * WAVES;
                float o[HALVES][VEC], hv[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float value, slope;
                    act_slope<PRECISE>(z[u][0][i], p.act, value, slope);
                    if constexpr (GATE) {
                        o[0][i] = d[u][i] * z[u][1][i] * slope;
                        o[1][i] = d[u][i] * value;
                        hv[i] = value * z[u][1][i];
                    } else {
                        o[0][i] = d[u][i] * slope;
                        hv[i] = value;
                    }
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) sum[h][i] += o[h][i];
                }
#pragma unroll
                for (int h = 0; h < HALVES; ++h)
                    store_row_vec<FULL>(static_cast<T*>(p.dZ) + row * p.ld_dz + col + (int64_t)h * p.N,
                                        o[h], n);
                if (p.H) store_row_vec<FULL>(static_cast<T*>(p.H) + row * p.ldh + col, hv, n);
            }
        }
    };
    if (n >= VEC) work(std::true_type{});
    else if (n > 0) work(std::false_type{});
    if (!p.sums) return;
    if (wave > 0)
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int i = 0; i < VEC; ++i) part[wave - 1][h * VEC + i][lane] = sum[h][i];
    __syncthreads();
    if (wave > 0) return;
    if (tm == 0 && tn == 0 && lane == 0) p.firsts[t.group] = t.first;
    // (offsets that do not ascend can make more tiles than the workspace has rows)
    if ((unsigned)(t.first + tm) >= (unsigned)p.tile_rows) return;
    float* out = p.sums + (int64_t)(t.first + tm) * p.width + col;
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float s = sum[h][i];
#pragma unroll
            for (int w = 0; w < WAVES - 1; ++w) s += part[w][h * VEC + i][lane];
            if (i < n) out[(int64_t)h * p.N + i] = s;
        }
}

// dbias of one group (blockIdx.y) and 64 columns: its tiles' sums, every fourth
// by one wave (520 rows of sums of 11264 columns, 16 groups: 5 us, a launch and
// 23 MB from the caches).  With one group and few columns a few waves add up all of
// it: 16384 rows of 2 x 128 columns 22 us on top of the pass's 9.5, of 2 x 1024
// 24 on top of 29, and 2^20 rows of 2 x 128 1.35 ms on top of 0.37.
template <int WAVES = 4>
__global__ __launch_bounds__(64 * WAVES) void act_bias_kernel(ActGradArgs p)
{
    __shared__ float part[WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
    for (int g = blockIdx.y; g < p.groups; g += gridDim.y) {
        int start = 0, size = p.M;
        if (p.offsets) group_span(p, g, start, size);
        int tiles = (int)(((unsigned)size + ACT_GRAD_ROWS - 1) / ACT_GRAD_ROWS);
        int first = tiles > 0 ? p.firsts[g] : 0;
        // (nor has then every group a first tile)
        if (first < 0 || first > p.tile_rows - tiles) first = tiles = 0;
        float s = 0.0f;
        if (col < p.width) {
            const float* in = p.sums + (int64_t)first * p.width + col;
#pragma unroll 4
            for (int t = wave; t < tiles; t += WAVES) s += in[(int64_t)t * p.width];
        }
        part[wave][lane] = s;
        __syncthreads();
        if (wave == 0 && col < p.width) {
#pragma unroll
            for (int w = 1; w < WAVES; ++w) s += part[w][lane];
            p.dbias[(int64_t)g * p.width + col] = s;
        }
        __syncthreads();
    }
}

}  // namespace dg
