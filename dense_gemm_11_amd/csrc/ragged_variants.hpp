// Launch tables of the ragged products (ragged.hpp): one tile configuration
// each, instantiated for the operand layouts and output types it serves.
#pragma once

#include "ragged.hpp"

namespace dg {

typedef hipError_t (*RaggedFn)(const RaggedArgs&, int grid, hipStream_t);

// Microseconds of a launch whose tiles find a compute unit each, and of each
// tile where they share the units: a fixed part and a part per 1000 of K.
struct TileCost {
    float alone, alone_k, each, each_k;
};

template <class Fn>
struct TileOf {
    int bm, bn[2], bk, threads;  // bn of either layout of B
    Fn fn[2][2];        // [B k-contiguous][bf16 output] (RAG_K: [0] only)
    bool stream;        // a streaming tile
    TileCost cost;
    TileCost cost_kc;   // with a k-contiguous B, where it is another (alone > 0)

    const TileCost& cost_of(bool b_kc) const { return b_kc && cost_kc.alone > 0.0f ? cost_kc : cost; }
};
using RaggedTile = TileOf<RaggedFn>;

// Expected time of `tiles` tiles of t.  The costs are least-squares fits of
// this form to timings of every tile on random calls of each kind (80 to 170
// of bf16 operands, 30 to 60 of fp32: 1 to 16384 rows, 1 to 128 groups, K 128
// to 8192, N 8 to 14336).  On 680 other calls of those ranges the tile of least
// expected time was within 2 % of the fastest in 70 %, within 10 % in 83 %, and
// up to 1.85 times it.  No tile is expected to beat the time of the call's
// `bytes` at 5.2 TB/s, which tiles narrower than 64 columns miss by 15 % (64
// experts of 4096x1792, 384 rows: 0.196 ms against 0.167 where B is n-contiguous,
// 0.178 against 0.163 where it is not); among tiles held to it the one with the
// least to do is taken.  A tenth of a round over whole ones is not counted, which
// suits the row-ragged calls, whose tiles are a guess, and now and then costs the
// others, whose tiles are known (276 tiles of 192x256 on 256 units, counted as
// one round: 0.298 ms where 184 of 256x256 take 0.193).
template <class Tile>
double expected_us(const Tile& t, bool b_kc, double tiles, double K, double bytes, int cus)
{
    const double n = tiles > cus ? tiles / cus : 1.0, k = K / 1000.0;
    const TileCost& cost = t.cost_of(b_kc);
    const double alone = cost.alone + k * cost.alone_k;
    // tiles that have a unit to themselves come in whole rounds, the others
    // leave a part of one
    const double rounds = t.stream || t.bm * t.bn[0] >= 192 * 256 ? (double)(int64_t)(n + 0.9)
                          : n > 1.0                               ? n + 0.4
                                                                  : 1.0;
    const double full = rounds * (cost.each + k * cost.each_k);
    const double us = alone > full ? alone : full;
    const double floor_us = bytes / 5.2e6 * (t.bn[b_kc] < 64 ? 1.15 : 1.0);
    return (us > floor_us ? us : floor_us) + 0.01 * us;
}

// Streaming tiles (stream.hpp), tallest first, the narrowest last; *count of
// them.
const RaggedTile* stream_rows_bf16(int* count);
const RaggedTile* stream_rows_f32(int* count);
const RaggedTile* stream_k_bf16(int* count);
const RaggedTile* stream_k_f32(int* count);
const RaggedTile* stream_lora_bf16(int* count);
const RaggedTile* stream_lora_f32(int* count);
// RAG_LORA_ONE: 16 rows, the wide tile first
const RaggedTile* stream_lora_one_bf16(int* count);
const RaggedTile* stream_lora_one_f32(int* count);

// Direct-to-LDS tiles, tallest first; *count of them.
const RaggedTile* ragged_rows_bf16(int* count);
const RaggedTile* ragged_rows_f32(int* count);
const RaggedTile* ragged_k_bf16(int* count);
const RaggedTile* ragged_k_f32(int* count);
const RaggedTile* ragged_lora_bf16(int* count);
const RaggedTile* ragged_lora_f32(int* count);

// Streaming tiles of T = s_a X op(down_a) (stream.hpp), by the narrowest that
// holds the rank and by descending height; *count of them.
const RaggedTile* stream_shrink_bf16(int* count);
const RaggedTile* stream_shrink_f32(int* count);

// SPLIT: a.splits workgroups along the second axis (RAG_SHRINK).
template <auto KERNEL, int THREADS, bool SPLIT = false>
hipError_t launch_ragged(const RaggedArgs& a, int grid, hipStream_t s)
{
    RaggedArgs copy = a;
    void* args[] = {&copy};
    return hipLaunchKernel(reinterpret_cast<const void*>(KERNEL), dim3(grid, SPLIT ? a.splits : 1),
                           dim3(THREADS), args, 0, s);
}

}  // namespace dg

// RaggedTile entry of configuration CFG for launch kind RAG, with its cost, A
// stored by rows: both layouts of B, both output types (fp32 operands: fp32 only).
#define DG_RAGGED_BF16(CFG, RAG, ...)                                                        \
    {CFG::BM, {CFG::BN, CFG::BN}, CFG::BK, CFG::THREADS,                                     \
     {{dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, false, false, RAG>, CFG::THREADS>, \
       dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, false, true, RAG>, CFG::THREADS>}, \
      {dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, true, false, RAG>, CFG::THREADS>,  \
       dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, true, true, RAG>, CFG::THREADS>}}, false, __VA_ARGS__}
#define DG_RAGGED_F32(CFG, RAG, ...)                                                         \
    {CFG::BM, {CFG::BN, CFG::BN}, CFG::BK, CFG::THREADS,                                     \
     {{dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, false, false, RAG>, CFG::THREADS>, \
       nullptr},                                                                             \
      {dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, true, false, RAG>, CFG::THREADS>,  \
       nullptr}}, false, __VA_ARGS__}
// ... and for RAG_K (both operands stored by rows).
#define DG_RAGGED_K_BF16(CFG, ...)                                                                 \
    {CFG::BM, {CFG::BN, CFG::BN}, CFG::BK, CFG::THREADS,                                           \
     {{dg::launch_ragged<dg::dma_ragged_kernel<CFG, false, false, false, RAG_K>, CFG::THREADS>,    \
       dg::launch_ragged<dg::dma_ragged_kernel<CFG, false, false, true, RAG_K>, CFG::THREADS>},    \
      {nullptr, nullptr}}, false, __VA_ARGS__}
#define DG_RAGGED_K_F32(CFG, ...)                                                                  \
    {CFG::BM, {CFG::BN, CFG::BN}, CFG::BK, CFG::THREADS,                                           \
     {{dg::launch_ragged<dg::dma_ragged_kernel<CFG, false, false, false, RAG_K>, CFG::THREADS>,    \
       nullptr},                                                                                   \
      {nullptr, nullptr}}, false, __VA_ARGS__}
