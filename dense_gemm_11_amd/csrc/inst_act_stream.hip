// Products of few rows per group with bias, activation, gate and residual
// (gemm_run_grouped_act): streaming tiles.
#include "act_variants.hpp"
#include "stream_variants.hpp"

namespace dg {
namespace {

// Tiles of 16*RF rows; 16*NFK columns of a k-contiguous B, 16*NFN of the other.
template <typename T, bool GATE, int RF, int NFK, int NFN>
constexpr ActTile act_tile(const TileCost (&cost)[2])
{
    using SN = StreamConfig<T, false, RF, NFN>;
    using SK = StreamConfig<T, true, RF, NFK>;
    ActTile t{SN::BM,
              {SN::BN, SK::BN},
              SN::KSTEP,
              SN::THREADS,
              {{launch_act<stream_act_kernel<SN, float, GATE>, SN::THREADS>, nullptr},
               {launch_act<stream_act_kernel<SK, float, GATE>, SK::THREADS>, nullptr}},
              true,
              cost[0],
              cost[1]};
    if constexpr (sizeof(T) == 2) {
        t.fn[0][1] = launch_act<stream_act_kernel<SN, bf16_t, GATE>, SN::THREADS>;
        t.fn[1][1] = launch_act<stream_act_kernel<SK, bf16_t, GATE>, SK::THREADS>;
    }
    return t;
}

// An n-contiguous row piece has at least 4 bytes, for each half of a gated tile
// (whose wide tile and narrow one are one with an n-contiguous bf16 B: pieces of 8
// bytes, 64 columns of either half, were the fastest tile of 7 of 200 calls only).
template <typename T, bool GATE>
const ActTile* act_tiles(int* count)
{
    constexpr int K1 = GATE ? 2 : 1, N1 = (GATE ? 2 : 1) * STREAM_N1<T>;
    // costs of either layout of B, of bf16 operands, gated ones, fp32, gated ones
    constexpr int X = (sizeof(T) == 4 ? 2 : 0) + (GATE ? 1 : 0);
    constexpr TileCost cost[5][4][2] = {
        {{{4.9f, 2.01f, 3.7f, 2.06f}, {}}, {{7.4f, 1.03f, 5.1f, 4.23f}, {5.3f, 1.31f, 3.8f, 2.46f}}, {}, {}},
        {{{5.5f, 0.68f, 4.3f, 2.48f}, {}},
         {{5.4f, 1.95f, 4.0f, 3.28f}, {5.7f, 1.11f, 4.4f, 2.32f}},
         {{8.4f, 1.31f, 4.6f, 10.96f}, {8.6f, 3.92f, 4.6f, 12.44f}},
         {{8.5f, 2.54f, 4.5f, 11.61f}, {7.5f, 7.54f, 5.1f, 12.18f}}},
        {{{4.3f, 1.31f, 3.2f, 1.10f}, {}},
         {{5.4f, 1.95f, 4.0f, 3.28f}, {4.8f, 0.83f, 3.3f, 1.64f}},
         {{4.4f, 3.47f, 1.8f, 3.20f}, {4.2f, 4.02f, 2.5f, 3.78f}},
         {{4.7f, 6.26f, 3.0f, 6.91f}, {4.5f, 6.61f, 3.6f, 7.11f}}},
        {{{4.6f, 2.16f, 3.6f, 2.34f}, {}},
         {{5.1f, 1.47f, 3.6f, 2.84f}, {5.3f, 0.79f, 3.6f, 2.46f}},
         {{4.6f, 6.27f, 3.1f, 6.53f}, {5.7f, 6.50f, 4.1f, 7.49f}},
         {{5.1f, 6.69f, 3.4f, 7.01f}, {5.6f, 6.82f, 4.1f, 7.78f}}},
        {{{4.1f, 1.24f, 2.3f, 0.80f}, {}},
         {{5.1f, 1.47f, 3.6f, 2.84f}, {4.4f, 0.80f, 2.5f, 1.28f}},
         {{4.2f, 1.85f, 1.4f, 2.39f}, {4.0f, 2.04f, 1.4f, 2.11f}},
         {{4.1f, 4.08f, 2.0f, 3.18f}, {4.2f, 3.91f, 2.4f, 4.65f}}}};
    constexpr ActTile low[] = {act_tile<T, GATE, 2, 4, 4>(cost[1][X]), act_tile<T, GATE, 2, K1, N1>(cost[2][X]),
                               act_tile<T, GATE, 1, 4, 4>(cost[3][X]), act_tile<T, GATE, 1, K1, N1>(cost[4][X])};
    if constexpr (sizeof(T) == 4) {
        static constexpr ActTile tiles[] = {low[0], low[1], low[2], low[3]};
        *count = 4;
        return tiles;
    } else {
        static constexpr ActTile tiles[] = {act_tile<T, GATE, 4, K1, N1>(cost[0][X]), low[0], low[1], low[2],
                                            low[3]};
        *count = 5;
        return tiles;
    }
}

}  // namespace

const ActTile* stream_act_bf16(int* count) { return act_tiles<bf16_t, false>(count); }
const ActTile* stream_act_f32(int* count) { return act_tiles<float, false>(count); }
const ActTile* stream_gate_bf16(int* count) { return act_tiles<bf16_t, true>(count); }
const ActTile* stream_gate_f32(int* count) { return act_tiles<float, true>(count); }

}  // namespace dg
