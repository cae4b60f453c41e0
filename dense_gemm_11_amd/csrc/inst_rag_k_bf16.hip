// K-ragged products of bf16 operands (gemm_run_grouped_wgrad).
#include "mfma_dma_gemm.hpp"
#include "selected_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_k_bf16(int* count)
{
    static const RaggedTile tiles[] = {DG_RAGGED_K_BF16(SelBf16Big), DG_RAGGED_K_BF16(SelBf16Mid)};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
