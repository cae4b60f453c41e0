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
                 SN::THREADS,
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
    // costs of bf16 and fp32 operands without adapters, then with
    constexpr int X = (sizeof(T) == 4 ? 1 : 0) + (RAG == RAG_LORA ? 2 : 0);
    constexpr TileCost cost[5][4] = {
        {{4.9f, 2.01f, 3.7f, 2.06f}, {}, {10.4f, 2.80f, 5.8f, 3.31f}, {}},
        {{5.5f, 0.68f, 4.3f, 2.48f},
         {8.6f, 3.26f, 4.1f, 12.44f},
         {11.2f, 3.24f, 6.0f, 3.82f},
         {15.7f, 6.93f, 9.5f, 14.13f}},
        {{4.3f, 1.31f, 3.2f, 1.10f},
         {4.5f, 3.75f, 2.0f, 3.57f},
         {10.1f, 1.81f, 5.2f, 2.13f},
         {10.1f, 5.32f, 3.3f, 4.14f}},
        {{4.6f, 2.16f, 3.6f, 2.34f},
         {5.4f, 6.27f, 3.6f, 6.77f},
         {10.5f, 2.52f, 5.1f, 2.90f},
         {11.1f, 7.66f, 7.3f, 7.54f}},
        {{4.1f, 1.24f, 2.3f, 0.80f},
         {4.4f, 2.07f, 1.5f, 1.93f},
         {10.7f, 1.08f, 1.9f, 1.46f},
         {9.5f, 4.17f, 2.4f, 2.16f}}};
    // 64 rows of fp32 go to the direct-to-LDS tile of that height instead
    constexpr RaggedTile low[] = {
        stream_tile<T, RAG, 2, 4, 4>(cost[1][X]), stream_tile<T, RAG, 2, 1, N1>(cost[2][X]),
        stream_tile<T, RAG, 1, 4, 4>(cost[3][X]), stream_tile<T, RAG, 1, 1, N1>(cost[4][X])};
    if constexpr (sizeof(T) == 4) {
        static constexpr RaggedTile tiles[] = {low[0], low[1], low[2], low[3]};
        *count = 4;
        return tiles;
    } else {
        static constexpr RaggedTile tiles[] = {stream_tile<T, RAG, 4, 1, N1>(cost[0][X]), low[0], low[1],
                                               low[2], low[3]};
        *count = 5;
        return tiles;
    }
}

// ... of the K-ragged product.
template <typename T, int F>
constexpr RaggedTile stream_k_tile(TileCost cost)
{
    RaggedTile t{16 * F,
                 {16 * F, 16 * F},
                 StreamConfig<T, false, F, F>::KSTEP,
                 StreamConfig<T, false, F, F>::THREADS,
                 {{launch_ragged<stream_k_kernel<T, F, float>, 512>, nullptr}, {nullptr, nullptr}},
                 true,
                 cost};
    if constexpr (sizeof(T) == 2) t.fn[0][1] = launch_ragged<stream_k_kernel<T, F, bf16_t>, 512>;
    return t;
}

template <typename T>
const RaggedTile* stream_k_tiles(int* count)
{
    constexpr int X = sizeof(T) == 4;
    constexpr TileCost cost[2][2] = {{{8.3f, 5.95f, 5.5f, 4.51f}, {8.9f, 46.83f, 6.1f, 26.99f}},
                                     {{6.1f, 2.89f, 2.6f, 2.64f}, {5.3f, 9.50f, 1.7f, 8.59f}}};
    static constexpr RaggedTile tiles[] = {stream_k_tile<T, 4>(cost[0][X]),
                                           stream_k_tile<T, 2>(cost[1][X])};
    *count = (int)(sizeof(tiles) / sizeof(tiles[0]));
    return tiles;
}

template <typename T>
const RaggedTile* stream_tiles_lora_one(int* count)
{
    static constexpr RaggedTile tiles[] = {stream_tile<T, RAG_LORA_ONE, 1, 4, 4>(),
                                           stream_tile<T, RAG_LORA_ONE, 1, 1, STREAM_N1<T>>()};
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
