// Products over ragged runs of rows.  Group g of `groups` holds the rows
// offsets[g] .. offsets[g+1]-1, an int32 array on the device, so the host
// knows neither the group sizes nor how many output tiles a call has: it
// launches the most tiles any split of the rows could need and each workgroup
// finds its own tile (find_row_tile) or ends.
//
// Offsets are clamped to [0, rows] and to a non-negative length wherever they
// are read, so no value of theirs leads outside the operands.
#pragma once

#include "common.hpp"

namespace dg {

// What a launch computes beside the plain GEMM:
//  RAG_ROWS: D[rows of g] = alpha s_g A[rows of g] op(B_g) + beta C[rows of g];
//  RAG_K   : D_g = alpha s_g op(A)[:, rows of g] op(B)[rows of g, :] + beta C_g
//            (the rows are the product's K);
//  RAG_LORA: D = alpha (A op(B) + T op(up_a)) + beta C, T the rows' products
//            with their segment's adapter, already scaled (lora.hpp);
//  RAG_SHRINK: those products, T[rows of s] = s_a A[rows of s] op(down_a)
//            (stream.hpp);
//  RAG_LORA_ONE: RAG_LORA and RAG_SHRINK in one launch, for one tile of rows.
enum : int { RAG_NONE = 0, RAG_ROWS = 1, RAG_K = 2, RAG_LORA = 3, RAG_SHRINK = 4, RAG_LORA_ONE = 5 };

struct RaggedArgs : GemmArgs {
    const int32_t* offsets;  // groups + 1
    const float* scales;     // one per group (RAG_LORA: per adapter), or null
    int groups;
    int deal;                // RAG_K: DEAL_*
    int rows;                // the rows that offsets divide
    int d_lines;             // D's rows (and groups) start on 128-byte lines
    int64_t stride_b;        // elements between the groups' B (RAG_ROWS)
    int64_t stride_c, stride_d;  // ... C and D (RAG_K)
    // RAG_LORA: adapter of each segment (< 0 or >= adapters: none; null: the
    // segment's own index), T as `splits` partial sums of rows x rank_pad
    // fp32, op(up_a): rank x N
    const int32_t* ids;
    int adapters, rank, rank_pad, splits;
    const float* t;
    const void* up;
    int64_t ld_up, stride_up;
    const void* down;        // RAG_LORA_ONE: rank x K
    int64_t ld_down, stride_down;
    int up_kc;               // up stored N x rank (rank contiguous)
    int k_slice;             // RAG_SHRINK: K of each of the `splits` slices
    uint16_t* t_terms;       // bf16 operands: T as `terms` terms (lora.hpp), or null
    int terms;
};

// First row and length of group g.
__device__ __forceinline__ void group_span(const RaggedArgs& p, int g, int& start, int& size)
{
    const int lo = p.offsets[g], hi = p.offsets[g + 1];
    start = lo < 0 ? 0 : (lo > p.rows ? p.rows : lo);
    const int end = hi > p.rows ? p.rows : hi;
    size = end > start ? end - start : 0;
}

// Inclusive prefix sum over the 64 lanes (row shifts, then the two
// broadcasts that carry a row's and a half-wave's sum on).
__device__ __forceinline__ int wave_scan(int x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);  // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);  // row_shr:2
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);  // row_shr:4
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);  // row_shr:8
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast:15
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // row_bcast:31
    return x;
}

// A workgroup's output tile of the row-ragged product: tile (tm, tn) of group
// `group`, which holds rows start .. start+size-1 in tiles_m tiles of BM.
struct RowTile {
    int group, start, size, tiles_m, in_group;
};

// Number of the tile that workgroup w takes: workgroups go round the 8 XCDs, and
// each XCD takes blocks of 32 consecutive numbers, a tile per compute unit, in
// turn (of the last, smaller round an eighth).  So an XCD's concurrent tiles
// share panels in its L2, and the XCDs' blocks share them in the cache behind:
// with a range of all tiles each, eight experts' matrices stream from memory at
// once.
__device__ __forceinline__ int block_cyclic(int w, int tiles)
{
    constexpr int XCDS = 8, BLOCK = 32, ROUND = XCDS * BLOCK;
    const int base = tiles / ROUND * ROUND;
    const int block = w < base ? BLOCK : (tiles - base) / XCDS;
    const int first = w < base ? w / ROUND * ROUND : base;
    const int r = w - first;
    return r < XCDS * block ? first + r % XCDS * block + r / XCDS : w;
}

// The tile of workgroup `w`, or false when there are fewer tiles.  Tiles are
// numbered group after group, tiles_m * tiles_n of them each.  Every lane of
// the wave takes part; the result is the same in each.
template <int BM>
__device__ __forceinline__ bool find_row_tile(const RaggedArgs& p, int w, int tiles_n, RowTile& t)
{
    const int lane = threadIdx.x & 63;
    auto chunk = [&](int g0, int& start, int& size, int& cnt) __attribute__((always_inline)) {
        start = size = 0;
        if (g0 + lane < p.groups) group_span(p, g0 + lane, start, size);
        cnt = (int)(((unsigned)size + (BM - 1)) / BM);
        return wave_scan(cnt);
    };
    int start, size, cnt, incl = chunk(0, start, size, cnt);
    int total = __builtin_amdgcn_readlane(incl, 63);
    for (int g0 = 64; g0 < p.groups; g0 += 64) {
        int s, z, c;
        total += __builtin_amdgcn_readlane(chunk(g0, s, z, c), 63);
    }
    const int tiles = total * tiles_n;
    if (w >= tiles) return false;
    w = block_cyclic(w, tiles);
    const int q = w / tiles_n;  // tile-row number over all groups
    int base = 0;
    for (int g0 = 0;;) {
        const int ex = base + incl - cnt;
        const uint64_t hit = __ballot(q >= ex && q < ex + cnt);
        if (hit != 0) {
            const int src = __builtin_ctzll(hit);
            t.group = g0 + src;
            t.start = __builtin_amdgcn_readlane(start, src);
            t.size = __builtin_amdgcn_readlane(size, src);
            t.tiles_m = __builtin_amdgcn_readlane(cnt, src);
            t.in_group = w - __builtin_amdgcn_readlane(ex, src) * tiles_n;
            return true;
        }
        base += __builtin_amdgcn_readlane(incl, 63);
        g0 += 64;
        if (g0 >= p.groups) return false;
        incl = chunk(g0, start, size, cnt);
    }
}

// How the tiles of a RAG_K launch are dealt to the XCDs (workgroups w % 8).  A
// tile takes as long as its group has rows, so XCDs that took whole groups
// would end when the longest ones do: each takes a slice of every group's tiles
// instead, one group after another (16 groups of 290 to 1200 rows, 2048x5632:
// 0.345 -> 0.287 ms).  Groups of few tiles are dealt out tile by tile.  Where
// groups have few rows and D's rows share lines, the call is the writing of D,
// and a range of whole groups each is faster (59 groups of one or two rows,
// 1216x4680 bf16: 0.334 ms against 0.385).
enum : int { DEAL_TILES = 0, DEAL_SLICES = 1, DEAL_RANGES = 2 };
constexpr int DEAL_XCDS = 8;

// Workgroups of such a launch of `groups` groups of `per` tiles each.
inline int64_t deal_grid(int deal, int64_t per, int64_t groups)
{
    return deal == DEAL_SLICES ? DEAL_XCDS * ((per + DEAL_XCDS - 1) / DEAL_XCDS) * groups
                               : per * groups;
}

// Tile t of group g for workgroup w, or false when it has none.
__device__ __forceinline__ bool find_k_tile(const RaggedArgs& p, int w, int& g, int& t)
{
    const int per = p.tiles_m * p.tiles_n;
    if (p.deal == DEAL_SLICES) {
        const int x = w % DEAL_XCDS, i = w / DEAL_XCDS;
        const int lo = (int)((int64_t)per * x / DEAL_XCDS);
        const int n = (int)((int64_t)per * (x + 1) / DEAL_XCDS) - lo;
        g = i / n;
        t = lo + i - g * n;
        return g < p.groups;
    }
    if (p.deal == DEAL_RANGES) {
        const int full = per * p.groups / DEAL_XCDS * DEAL_XCDS;
        if (w < full) w = (w % DEAL_XCDS) * (full / DEAL_XCDS) + w / DEAL_XCDS;
    }
    g = w / per;
    t = w - g * per;
    return true;
}

// alpha times group g's factor.  An empty group of a RAG_K launch has no product
// and takes none: its factor may well be infinite (one over its rows).
__device__ __forceinline__ float group_alpha(const RaggedArgs& p, int g, int rows)
{
    return rows == 0 ? 0.0f : p.scales ? p.alpha * p.scales[g] : p.alpha;
}

// Narrow p to the workgroup's group: operands, output, M (or K) and alpha
// become those of the group, and (tm, tn) its output tile.  False when the
// workgroup has none.
template <int RAG, int BM, typename T, typename OutT>
__device__ __forceinline__ bool narrow_to_group(RaggedArgs& p, int& tm, int& tn)
{
    const T* A = static_cast<const T*>(p.A);
    const T* B = static_cast<const T*>(p.B);
    const OutT* C = reinterpret_cast<const OutT*>(p.C);
    OutT* D = reinterpret_cast<OutT*>(p.D);
    int g;
    if constexpr (RAG == RAG_ROWS) {
        RowTile t;
        if (!find_row_tile<BM>(p, blockIdx.x, p.tiles_n, t)) return false;
        g = t.group;
        p.M = t.size;
        p.tiles_m = t.tiles_m;
        tile_of(p, t.in_group, tm, tn);
        p.A = A + (int64_t)t.start * p.lda;
        p.B = B + (int64_t)g * p.stride_b;
        if (C) p.C = reinterpret_cast<const float*>(C + (int64_t)t.start * p.ldc);
        p.D = reinterpret_cast<float*>(D + (int64_t)t.start * p.ldd);
    } else {
        int t;
        if (!find_k_tile(p, blockIdx.x, g, t)) return false;
        tile_of(p, t, tm, tn);
        int start, size;
        group_span(p, g, start, size);
        start = __builtin_amdgcn_readfirstlane(start);
        p.K = __builtin_amdgcn_readfirstlane(size);
        p.A = A + (int64_t)start * p.lda;
        p.B = B + (int64_t)start * p.ldb;
        if (C) p.C = reinterpret_cast<const float*>(C + (int64_t)g * p.stride_c);
        p.D = reinterpret_cast<float*>(D + (int64_t)g * p.stride_d);
    }
    p.alpha = group_alpha(p, g, RAG == RAG_K ? p.K : p.M);
    return true;
}

}  // namespace dg
