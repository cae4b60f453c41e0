// Row-ragged products of bf16 operands (gemm_run_grouped).
#include "mfma_dma_gemm.hpp"
#include "ragged_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_rows_bf16(int* count)
{
    static const RaggedTile tiles[] = {
        DG_RAGGED_BF16(SelBf16Big, RAG_ROWS, {8.0f, 3.23f, 8.2f, 20.15f}),
        DG_RAGGED_BF16(Dma192x256s3L, RAG_ROWS, {8.7f, 5.87f, 7.9f, 15.29f}),
        DG_RAGGED_BF16(Dma128x256s3L, RAG_ROWS, {8.0f, 4.93f, 8.0f, 11.80f}),
        DG_RAGGED_BF16(SelBf16Mid, RAG_ROWS, {6.2f, 5.74f, 4.3f, 7.15f}),
        DG_RAGGED_BF16(RagBf16Low, RAG_ROWS, {5.4f, 4.38f, 3.3f, 4.89f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
