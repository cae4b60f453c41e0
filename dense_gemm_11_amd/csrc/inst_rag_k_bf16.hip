// K-ragged products of bf16 operands (gemm_run_grouped_wgrad).
#include "mfma_dma_gemm.hpp"
#include "ragged_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_k_bf16(int* count)
{
    static const RaggedTile tiles[] = {
        DG_RAGGED_K_BF16(SelBf16Big, {20.2f, 20.94f, 20.1f, 25.74f}),
        DG_RAGGED_K_BF16(Dma192x256s3L, {15.3f, 24.79f, 16.0f, 19.85f}),
        DG_RAGGED_K_BF16(Dma128x256s3L, {17.2f, 16.98f, 12.2f, 14.30f}),
        DG_RAGGED_K_BF16(SelBf16Mid, {11.5f, 11.67f, 5.8f, 8.96f}),
        DG_RAGGED_K_BF16(RagBf16Thin, {11.1f, 20.29f, 4.3f, 10.00f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
