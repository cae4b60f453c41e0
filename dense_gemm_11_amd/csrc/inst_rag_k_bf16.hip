// K-ragged products of bf16 operands (gemm_run_grouped_wgrad).
#include "mfma_dma_gemm.hpp"
#include "ragged_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_k_bf16(int* count)
{
    static const RaggedTile tiles[] = {
        DG_RAGGED_K_BF16(SelBf16Big, {8.0f, 3.40f, 22.1f, 26.08f}),
        DG_RAGGED_K_BF16(Dma192x256s3L, {8.0f, 2.68f, 18.0f, 20.54f}),
        DG_RAGGED_K_BF16(Dma128x256s3L, {19.7f, 16.58f, 11.2f, 14.69f}),
        DG_RAGGED_K_BF16(SelBf16Mid, {11.4f, 10.71f, 4.9f, 9.67f}),
        DG_RAGGED_K_BF16(RagBf16Thin, {10.8f, 22.55f, 3.8f, 9.47f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
