// Row-ragged products of few rows per group (gemm_run_grouped): streaming tiles.
#include "stream_variants.hpp"

namespace dg {

const RaggedTile* stream_rows_bf16(int* count)
{
    return stream_tiles<bf16_t, RAG_ROWS>(count);
}

const RaggedTile* stream_rows_f32(int* count)
{
    return stream_tiles<float, RAG_ROWS>(count);
}

}  // namespace dg
