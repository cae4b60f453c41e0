// Shared products of bf16 operands with low-rank adapters added (gemm_run_lora).
#include "mfma_dma_gemm.hpp"
#include "ragged_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_lora_bf16(int* count)
{
    static const RaggedTile tiles[] = {
        DG_RAGGED_BF16(SelBf16Big, RAG_LORA, {27.8f, 21.5f, 20.6f, 26.9f}),
        DG_RAGGED_BF16(Dma192x256s3L, RAG_LORA, {25.2f, 15.5f, 17.4f, 21.3f}),
        DG_RAGGED_BF16(RagBf16Mid, RAG_LORA, {20.0f, 8.9f, 6.0f, 10.8f}),
        DG_RAGGED_BF16(RagBf16Low, RAG_LORA, {18.1f, 7.1f, 4.7f, 6.5f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
