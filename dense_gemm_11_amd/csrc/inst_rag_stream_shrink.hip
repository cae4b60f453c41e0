// The first product of the low-rank adapters, T = s X op(down) (gemm_run_lora).
#include "stream_variants.hpp"

namespace dg {

const RaggedTile* stream_shrink_bf16(int* count)
{
    return stream_tiles_shrink<bf16_t>(count);
}

const RaggedTile* stream_shrink_f32(int* count)
{
    return stream_tiles_shrink<float>(count);
}

}  // namespace dg
