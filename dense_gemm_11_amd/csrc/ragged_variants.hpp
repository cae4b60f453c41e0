// Launch tables of the ragged products (ragged.hpp): one tile configuration
// each, instantiated for the operand layouts and output types it serves.
#pragma once

#include "ragged.hpp"

namespace dg {

typedef hipError_t (*RaggedFn)(const RaggedArgs&, int grid, hipStream_t);

struct RaggedTile {
    int bm, bn[2], bk;  // bn of either layout of B
    RaggedFn fn[2][2];  // [B k-contiguous][bf16 output] (RAG_K: [0] only)
};

// Streaming tiles (stream.hpp), tallest first, the narrowest last; *count of
// them.
const RaggedTile* stream_rows_bf16(int* count);
const RaggedTile* stream_rows_f32(int* count);
const RaggedTile* stream_lora_bf16(int* count);
const RaggedTile* stream_lora_f32(int* count);

// Direct-to-LDS tiles, tallest first; *count of them.
const RaggedTile* ragged_rows_bf16(int* count);
const RaggedTile* ragged_rows_f32(int* count);
const RaggedTile* ragged_k_bf16(int* count);
const RaggedTile* ragged_k_f32(int* count);
const RaggedTile* ragged_lora_bf16(int* count);
const RaggedTile* ragged_lora_f32(int* count);

// T = s X op(down) (lora.hpp).  `tall`: blocks of 32 rows in place of 16.
struct ShrinkCall {
    const void* down;
    int64_t ld_down, stride_down;
    bool down_kc;
    int k_slice, splits;
    bool tall;
    float* t;
};
hipError_t launch_shrink(const RaggedArgs& a, const ShrinkCall& c, bool bf16, hipStream_t s);

template <auto KERNEL, int THREADS>
hipError_t launch_ragged(const RaggedArgs& a, int grid, hipStream_t s)
{
    RaggedArgs copy = a;
    void* args[] = {&copy};
    return hipLaunchKernel(reinterpret_cast<const void*>(KERNEL), dim3(grid), dim3(THREADS), args,
                           0, s);
}

}  // namespace dg

// RaggedTile entry of configuration CFG for launch kind RAG with A stored by
// rows: both layouts of B, both output types (fp32 operands: fp32 only).
#define DG_RAGGED_BF16(CFG, RAG)                                                             \
    {CFG::BM, {CFG::BN, CFG::BN}, CFG::BK,                                                   \
     {{dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, false, false, RAG>, CFG::THREADS>, \
       dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, false, true, RAG>, CFG::THREADS>}, \
      {dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, true, false, RAG>, CFG::THREADS>,  \
       dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, true, true, RAG>, CFG::THREADS>}}}
#define DG_RAGGED_F32(CFG, RAG)                                                              \
    {CFG::BM, {CFG::BN, CFG::BN}, CFG::BK,                                                   \
     {{dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, false, false, RAG>, CFG::THREADS>, \
       nullptr},                                                                             \
      {dg::launch_ragged<dg::dma_ragged_kernel<CFG, true, true, false, RAG>, CFG::THREADS>,  \
       nullptr}}}
// ... and for RAG_K (both operands stored by rows).
#define DG_RAGGED_K_BF16(CFG)                                                                      \
    {CFG::BM, {CFG::BN, CFG::BN}, CFG::BK,                                                         \
     {{dg::launch_ragged<dg::dma_ragged_kernel<CFG, false, false, false, RAG_K>, CFG::THREADS>,    \
       dg::launch_ragged<dg::dma_ragged_kernel<CFG, false, false, true, RAG_K>, CFG::THREADS>},    \
      {nullptr, nullptr}}}
#define DG_RAGGED_K_F32(CFG)                                                                       \
    {CFG::BM, {CFG::BN, CFG::BN}, CFG::BK,                                                         \
     {{dg::launch_ragged<dg::dma_ragged_kernel<CFG, false, false, false, RAG_K>, CFG::THREADS>,    \
       nullptr},                                                                                   \
      {nullptr, nullptr}}}
