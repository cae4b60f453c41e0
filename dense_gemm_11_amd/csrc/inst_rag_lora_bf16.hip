// Shared products of bf16 operands with low-rank adapters added (gemm_run_lora).
#include "mfma_dma_gemm.hpp"
#include "ragged_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_lora_bf16(int* count)
{
    static const RaggedTile tiles[] = {
        DG_RAGGED_BF16(SelBf16Big, RAG_LORA, {8.0f, 22.84f, 20.8f, 22.75f}),
        DG_RAGGED_BF16(Dma192x256s3L, RAG_LORA, {8.0f, 17.66f, 19.5f, 17.31f}),
        DG_RAGGED_BF16(RagBf16Mid, RAG_LORA, {15.4f, 7.11f, 8.7f, 9.87f}),
        DG_RAGGED_BF16(RagBf16Low, RAG_LORA, {14.0f, 6.08f, 6.6f, 6.41f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
