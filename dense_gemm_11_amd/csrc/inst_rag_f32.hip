// Ragged products of fp32 operands: by rows (gemm_run_grouped), along K
// (gemm_run_grouped_wgrad) and with low-rank adapters (gemm_run_lora).
#include "mfma_dma_gemm.hpp"
#include "selected_configs.hpp"
#include "ragged_variants.hpp"

namespace dg {

const RaggedTile* ragged_rows_f32(int* count)
{
    static const RaggedTile tiles[] = {DG_RAGGED_F32(SelF32Big, RAG_ROWS),
                                       DG_RAGGED_F32(SelF32Mid, RAG_ROWS)};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

const RaggedTile* ragged_lora_f32(int* count)
{
    static const RaggedTile tiles[] = {DG_RAGGED_F32(SelF32Big, RAG_LORA),
                                       DG_RAGGED_F32(SelF32Mid, RAG_LORA)};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

const RaggedTile* ragged_k_f32(int* count)
{
    static const RaggedTile tiles[] = {DG_RAGGED_K_F32(SelF32Big), DG_RAGGED_K_F32(SelF32Mid)};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
