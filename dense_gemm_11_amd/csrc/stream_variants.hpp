// Launch tables of the streaming tiles (stream.hpp), for the files that
// instantiate them for one kind of launch each.
#pragma once

#include "ragged_variants.hpp"
#include "stream.hpp"

namespace dg {

// Tiles of 16*RF rows; 16*NFK columns of a k-contiguous B, 16*NFN of the
// other, with UK and UN fragment steps per batch.
template <typename T, int RAG, int RF, int NFK, int UK, int NFN, int UN>
constexpr RaggedTile stream_tile()
{
    using SN = StreamConfig<T, false, RF, NFN, UN>;
    using SK = StreamConfig<T, true, RF, NFK, UK>;
    RaggedTile t{SN::BM,
                 {SN::BN, SK::BN},
                 SN::KSTEP,
                 {{launch_ragged<stream_kernel<SN, float, RAG>, SN::THREADS>, nullptr},
                  {launch_ragged<stream_kernel<SK, float, RAG>, SK::THREADS>, nullptr}}};
    if constexpr (sizeof(T) == 2) {
        t.fn[0][1] = launch_ragged<stream_kernel<SN, bf16_t, RAG>, SN::THREADS>;
        t.fn[1][1] = launch_ragged<stream_kernel<SK, bf16_t, RAG>, SK::THREADS>;
    }
    return t;
}

template <int RAG>
const RaggedTile* stream_tiles_bf16(int* count)
{
    static constexpr RaggedTile tiles[] = {
        stream_tile<bf16_t, RAG, 4, 4, 2, 4, 2>(), stream_tile<bf16_t, RAG, 2, 4, 2, 4, 2>(),
        stream_tile<bf16_t, RAG, 1, 4, 2, 4, 2>(), stream_tile<bf16_t, RAG, 1, 1, 4, 2, 4>()};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

template <int RAG>
const RaggedTile* stream_tiles_f32(int* count)
{
    static constexpr RaggedTile tiles[] = {
        stream_tile<float, RAG, 4, 4, 2, 4, 2>(), stream_tile<float, RAG, 2, 4, 2, 4, 2>(),
        stream_tile<float, RAG, 1, 4, 2, 4, 2>(), stream_tile<float, RAG, 1, 1, 4, 1, 4>()};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
