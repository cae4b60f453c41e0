// Row-ragged products of bf16 operands (gemm_run_grouped).
#include "mfma_dma_gemm.hpp"
#include "ragged_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_rows_bf16(int* count)
{
    static const RaggedTile tiles[] = {
        DG_RAGGED_BF16(SelBf16Big, RAG_ROWS, {10.8f, 15.8f, 10.5f, 20.4f}),
        DG_RAGGED_BF16(Dma192x256s3L, RAG_ROWS, {10.1f, 15.1f, 9.9f, 16.6f}),
        DG_RAGGED_BF16(Dma128x256s3L, RAG_ROWS, {8.0f, 12.8f, 10.4f, 13.6f}),
        DG_RAGGED_BF16(SelBf16Mid, RAG_ROWS, {7.5f, 8.0f, 5.7f, 8.3f}),
        DG_RAGGED_BF16(RagBf16Low, RAG_ROWS, {7.5f, 4.4f, 4.2f, 6.6f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
