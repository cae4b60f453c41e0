// K-ragged products of few tiles over many rows (gemm_run_grouped_wgrad):
// streaming tiles.
#include "stream_variants.hpp"

namespace dg {

const RaggedTile* stream_k_bf16(int* count)
{
    return stream_k_tiles<bf16_t>(count);
}

const RaggedTile* stream_k_f32(int* count)
{
    return stream_k_tiles<float>(count);
}

}  // namespace dg
