// Shared products of bf16 operands with low-rank adapters added (gemm_run_lora).
#include "mfma_dma_gemm.hpp"
#include "selected_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_lora_bf16(int* count)
{
    static const RaggedTile tiles[] = {DG_RAGGED_BF16(SelBf16Big, RAG_LORA), DG_RAGGED_BF16(SelBf16Mid, RAG_LORA)};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
