// Row-ragged products of bf16 operands (gemm_run_grouped).
#include "mfma_dma_gemm.hpp"
#include "selected_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_rows_bf16(int* count)
{
    static const RaggedTile tiles[] = {DG_RAGGED_BF16(SelBf16Big, RAG_ROWS), DG_RAGGED_BF16(SelBf16Mid, RAG_ROWS)};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
