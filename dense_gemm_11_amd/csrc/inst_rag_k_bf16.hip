// K-ragged products of bf16 operands (gemm_run_grouped_wgrad).
#include "mfma_dma_gemm.hpp"
#include "ragged_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_k_bf16(int* count)
{
    static const RaggedTile tiles[] = {
        DG_RAGGED_K_BF16(SelBf16Big, {18.2f, 13.7f, 24.6f, 26.5f}),
        DG_RAGGED_K_BF16(Dma192x256s3L, {21.9f, 22.2f, 17.2f, 23.3f}),
        DG_RAGGED_K_BF16(Dma128x256s3L, {8.1f, 12.4f, 18.7f, 19.7f}),
        DG_RAGGED_K_BF16(SelBf16Mid, {15.9f, 11.3f, 5.8f, 12.5f}),
        DG_RAGGED_K_BF16(RagBf16Thin, {15.9f, 20.7f, 4.6f, 14.7f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
