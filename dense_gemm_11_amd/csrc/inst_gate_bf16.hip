// Gated products of bf16 operands (gemm_run_grouped_act).
#include "mfma_dma_gemm.hpp"
#include "ragged_configs.hpp"
#include "act_variants.hpp"

namespace dg {

const ActTile* gate_tiles_bf16(int* count)
{
    static const ActTile tiles[] = {
        DG_ACT_BF16(SelBf16Big, RAG_GATE, {8.0f, 0.0f, 9.3f, 17.04f}, {8.0f, 1.08f, 7.9f, 21.35f}),
        DG_ACT_BF16(Dma192x256s3L, RAG_GATE, {8.6f, 9.99f, 8.3f, 13.97f}, {9.1f, 5.93f, 6.7f, 19.22f}),
        DG_ACT_BF16(Dma128x256s3L, RAG_GATE, {8.5f, 10.79f, 6.7f, 11.77f}, {8.3f, 5.85f, 6.8f, 13.60f}),
        DG_ACT_BF16(SelBf16Mid, RAG_GATE, {6.2f, 5.03f, 4.1f, 6.75f}, {6.3f, 4.10f, 3.3f, 8.65f}),
        DG_ACT_BF16(RagBf16Low, RAG_GATE, {5.6f, 4.03f, 3.2f, 5.02f}, {5.2f, 4.83f, 3.4f, 5.21f})};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
