// Products of fp32 operands with bias, activation and residual, and gated ones
// (gemm_run_grouped_act).
#include "mfma_dma_gemm.hpp"
#include "ragged_configs.hpp"
#include "act_variants.hpp"

namespace dg {

const ActTile* act_tiles_f32(int* count)
{
    static const ActTile tiles[] = {
        DG_ACT_F32(SelF32Mid, RAG_ACT, {9.4f, 55.28f, 4.8f, 57.45f}, {7.4f, 58.92f, 4.6f, 60.07f}),
        DG_ACT_F32(RagF32Low, RAG_ACT, {7.8f, 28.32f, 2.7f, 29.35f}, {6.0f, 30.69f, 3.5f, 30.33f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

const ActTile* gate_tiles_f32(int* count)
{
    static const ActTile tiles[] = {
        DG_ACT_F32(SelF32Mid, RAG_GATE, {5.9f, 58.30f, 2.4f, 60.27f}, {8.9f, 54.00f, 3.1f, 59.00f}),
        DG_ACT_F32(RagF32Low, RAG_GATE, {4.8f, 30.11f, 1.7f, 30.48f}, {6.4f, 28.91f, 2.7f, 30.61f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
