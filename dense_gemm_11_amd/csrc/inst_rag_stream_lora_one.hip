// Products of up to 16 rows with low-rank adapters in one launch
// (gemm_run_lora): streaming tiles.
#include "stream_variants.hpp"

namespace dg {

const RaggedTile* stream_lora_one_bf16(int* count)
{
    return stream_tiles_lora_one<bf16_t>(count);
}

const RaggedTile* stream_lora_one_f32(int* count)
{
    return stream_tiles_lora_one<float>(count);
}

}  // namespace dg
