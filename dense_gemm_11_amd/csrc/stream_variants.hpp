// Launch tables of the streaming tiles (stream.hpp), for the files that
// instantiate them for one kind of launch each.
#pragma once

#include "ragged_variants.hpp"
#include "stream.hpp"

namespace dg {

// Tiles of 16*RF rows; 16*NFK columns of a k-contiguous B, 16*NFN of the other.
template <typename T, int RAG, int RF, int NFK, int NFN>
constexpr RaggedTile stream_tile(TileCost cost = {})
{
    using SN = StreamConfig<T, false, RF, NFN>;
    using SK = StreamConfig<T, true, RF, NFK>;
    constexpr bool SPLIT = RAG == RAG_SHRINK;
    RaggedTile t{SN::BM,
                 {SN::BN, SK::BN},
                 SN::KSTEP,
                 {{launch_ragged<stream_kernel<SN, float, RAG>, SN::THREADS, SPLIT>, nullptr},
                  {launch_ragged<stream_kernel<SK, float, RAG>, SK::THREADS, SPLIT>, nullptr}},
                 true,
                 cost};
    if constexpr (sizeof(T) == 2 && !SPLIT) {
        t.fn[0][1] = launch_ragged<stream_kernel<SN, bf16_t, RAG>, SN::THREADS>;
        t.fn[1][1] = launch_ragged<stream_kernel<SK, bf16_t, RAG>, SK::THREADS>;
    }
    return t;
}

// An n-contiguous row piece has at least 4 bytes: two columns of bf16.
template <typename T>
constexpr int STREAM_N1 = sizeof(T) == 2 ? 2 : 1;

template <typename T, int RAG>
const RaggedTile* stream_tiles(int* count)
{
    constexpr int N1 = STREAM_N1<T>;
    // costs of bf16 and fp32 operands, without and with adapters
    constexpr int X = (sizeof(T) == 4 ? 1 : 0) + (RAG == RAG_LORA ? 2 : 0);
    constexpr TileCost cost[5][4] = {
        {{5.5f, 1.4f, 3.3f, 2.9f}, {5.9f, 7.9f, 3.8f, 7.6f}, {11.9f, 3.0f, 5.8f, 3.6f}, {11.6f, 8.7f, 8.0f, 8.1f}},
        {{6.1f, 1.7f, 4.2f, 3.5f}, {11.1f, 0.0f, 4.7f, 12.0f}, {12.9f, 3.6f, 8.2f, 4.4f}, {13.6f, 13.6f, 11.0f, 13.1f}},
        {{4.4f, 2.0f, 2.8f, 2.1f}, {4.7f, 4.1f, 1.8f, 4.5f}, {10.5f, 2.4f, 5.8f, 2.1f}, {11.7f, 4.9f, 2.9f, 3.9f}},
        {{5.5f, 2.5f, 4.0f, 3.0f}, {5.6f, 6.5f, 3.5f, 7.5f}, {11.1f, 3.3f, 7.1f, 3.0f}, {11.9f, 8.9f, 6.5f, 7.7f}},
        {{5.4f, 1.2f, 2.0f, 1.6f}, {4.9f, 3.5f, 1.2f, 2.5f}, {11.4f, 1.5f, 2.3f, 1.5f}, {12.8f, 2.9f, 2.0f, 2.2f}}};
    static constexpr RaggedTile tiles[] = {
        stream_tile<T, RAG, 4, 1, N1>(cost[0][X]), stream_tile<T, RAG, 2, 4, 4>(cost[1][X]),
        stream_tile<T, RAG, 2, 1, N1>(cost[2][X]), stream_tile<T, RAG, 1, 4, 4>(cost[3][X]),
        stream_tile<T, RAG, 1, 1, N1>(cost[4][X])};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

template <typename T>
const RaggedTile* stream_tiles_shrink(int* count)
{
    constexpr int N1 = STREAM_N1<T>;
    static constexpr RaggedTile tiles[] = {
        stream_tile<T, RAG_SHRINK, 2, 1, N1>(), stream_tile<T, RAG_SHRINK, 1, 1, N1>(),
        stream_tile<T, RAG_SHRINK, 2, 2, 2>(),  stream_tile<T, RAG_SHRINK, 1, 2, 2>(),
        stream_tile<T, RAG_SHRINK, 2, 4, 4>(),  stream_tile<T, RAG_SHRINK, 1, 4, 4>()};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

}  // namespace dg
