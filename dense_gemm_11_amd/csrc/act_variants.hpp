// Launch tables of the products with bias, activation, gate and residual
// (act.hpp): one tile configuration each, for both layouts of B and both output
// types.  bn counts B's columns: gated, twice the outputs'.
//
// The costs of the gated tiles and of those of fp32 operands are fits of their
// own for either layout of B (100 random calls of each kind: 1 to 16384 rows, 1 to
// 128 groups, K 128 to 8192, N 128 to 14336), the others are gemm_run_grouped's.
// On 50 other calls of each kind the tile chosen took 1.02 to 1.06 times the
// fastest one's time on average, and up to 1.7 times; with gemm_run_grouped's costs
// throughout 1.26 on average where a gated bf16 B is n-contiguous (a row piece is
// half as long there, and streaming tiles half as fast) and 1.13 where a gated fp32
// one is not.
#pragma once

#include "act.hpp"
#include "ragged_variants.hpp"

namespace dg {

typedef hipError_t (*ActFn)(const ActArgs&, int grid, hipStream_t);
using ActTile = TileOf<ActFn>;

template <auto KERNEL, int THREADS>
hipError_t launch_act(const ActArgs& a, int grid, hipStream_t s)
{
    ActArgs copy = a;
    void* args[] = {&copy};
    return hipLaunchKernel(reinterpret_cast<const void*>(KERNEL), dim3(grid), dim3(THREADS), args, 0, s);
}

// Direct-to-LDS tiles, tallest first; *count of them.
const ActTile* act_tiles_bf16(int* count);
const ActTile* act_tiles_f32(int* count);
const ActTile* gate_tiles_bf16(int* count);
const ActTile* gate_tiles_f32(int* count);

// Streaming tiles (stream.hpp), tallest first, the narrowest last; *count of them.
const ActTile* stream_act_bf16(int* count);
const ActTile* stream_act_f32(int* count);
const ActTile* stream_gate_bf16(int* count);
const ActTile* stream_gate_f32(int* count);

}  // namespace dg

#define DG_ACT_BF16(CFG, RAG, ...)                                                      \
    {CFG::BM, {CFG::BN, CFG::BN}, CFG::BK, CFG::THREADS,                                \
     {{dg::launch_act<dg::dma_act_kernel<CFG, false, false, RAG>, CFG::THREADS>,        \
       dg::launch_act<dg::dma_act_kernel<CFG, false, true, RAG>, CFG::THREADS>},        \
      {dg::launch_act<dg::dma_act_kernel<CFG, true, false, RAG>, CFG::THREADS>,         \
       dg::launch_act<dg::dma_act_kernel<CFG, true, true, RAG>, CFG::THREADS>}}, false, __VA_ARGS__}
#define DG_ACT_F32(CFG, RAG, ...)                                                       \
    {CFG::BM, {CFG::BN, CFG::BN}, CFG::BK, CFG::THREADS,                                \
     {{dg::launch_act<dg::dma_act_kernel<CFG, false, false, RAG>, CFG::THREADS>, nullptr}, \
      {dg::launch_act<dg::dma_act_kernel<CFG, true, false, RAG>, CFG::THREADS>, nullptr}}, false, __VA_ARGS__}
