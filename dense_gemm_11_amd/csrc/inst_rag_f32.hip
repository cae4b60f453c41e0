// Ragged products of fp32 operands: by rows (gemm_run_grouped), along K
// (gemm_run_grouped_wgrad) and with low-rank adapters (gemm_run_lora).
#include "mfma_dma_gemm.hpp"
#include "ragged_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_rows_f32(int* count)
{
    static const RaggedTile tiles[] = {
        DG_RAGGED_F32(SelF32Mid, RAG_ROWS, {8.1f, 58.65f, 4.4f, 57.93f}),
        DG_RAGGED_F32(RagF32Low, RAG_ROWS, {5.7f, 30.59f, 2.2f, 31.59f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

const RaggedTile* ragged_lora_f32(int* count)
{
    static const RaggedTile tiles[] = {
        DG_RAGGED_F32(SelF32Mid, RAG_LORA, {5.1f, 55.86f, 15.8f, 76.47f}),
        DG_RAGGED_F32(RagF32Low, RAG_LORA, {17.2f, 36.79f, 6.0f, 47.04f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

const RaggedTile* ragged_k_f32(int* count)
{
    static const RaggedTile tiles[] = {
        DG_RAGGED_K_F32(SelF32Mid, {11.9f, 71.58f, 5.9f, 70.77f}),
        DG_RAGGED_K_F32(RagF32Low, {7.3f, 49.28f, 3.0f, 35.35f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
