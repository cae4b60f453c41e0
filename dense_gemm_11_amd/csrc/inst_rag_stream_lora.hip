// Shared products of few rows with low-rank adapters (gemm_run_lora): streaming tiles.
#include "stream_variants.hpp"

namespace dg {

const RaggedTile* stream_lora_bf16(int* count)
{
    return stream_tiles<bf16_t, RAG_LORA>(count);
}

const RaggedTile* stream_lora_f32(int* count)
{
    return stream_tiles<float, RAG_LORA>(count);
}

}  // namespace dg
