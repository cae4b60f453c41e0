// Products of fp32 operands with bias, activation and residual, and gated ones
// (gemm_run_grouped_act).
#include "mfma_dma_gemm.hpp"
#include "ragged_configs.hpp"
#include "act_variants.hpp"

namespace dg {

const ActTile* act_tiles_f32(int* count)
{
    static const ActTile tiles[] = {DG_ACT_F32(SelF32Mid, RAG_ACT, {8.1f, 58.65f, 4.4f, 57.93f}),
                                    DG_ACT_F32(RagF32Low, RAG_ACT, {5.7f, 30.59f, 2.2f, 31.59f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

const ActTile* gate_tiles_f32(int* count)
{
    static const ActTile tiles[] = {DG_ACT_F32(SelF32Mid, RAG_GATE, {8.1f, 58.65f, 4.4f, 57.93f}),
                                    DG_ACT_F32(RagF32Low, RAG_GATE, {5.7f, 30.59f, 2.2f, 31.59f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
