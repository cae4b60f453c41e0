// Products of few rows per group with bias, activation, gate and residual
// (gemm_run_grouped_act): streaming tiles.
#include "act_variants.hpp"
#include "stream_variants.hpp"

namespace dg {
namespace {

// Tiles of 16*RF rows; 16*NFK columns of a k-contiguous B, 16*NFN of the other.
template <typename T, bool GATE, int RF, int NFK, int NFN>
constexpr ActTile act_tile(TileCost cost)
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
              cost};
    if constexpr (sizeof(T) == 2) {
        t.fn[0][1] = launch_act<stream_act_kernel<SN, bf16_t, GATE>, SN::THREADS>;
        t.fn[1][1] = launch_act<stream_act_kernel<SK, bf16_t, GATE>, SK::THREADS>;
    }
    return t;
}

// An n-contiguous row piece has at least 4 bytes, for each half of a gated tile.
template <typename T, bool GATE>
const ActTile* act_tiles(int* count)
{
    constexpr int K1 = GATE ? 2 : 1, N1 = (GATE ? 2 : 1) * STREAM_N1<T>;
    constexpr int X = sizeof(T) == 4 ? 1 : 0;
    constexpr TileCost cost[5][2] = {{{4.9f, 2.01f, 3.7f, 2.06f}, {}},
                                     {{5.5f, 0.68f, 4.3f, 2.48f}, {8.6f, 3.26f, 4.1f, 12.44f}},
                                     {{4.3f, 1.31f, 3.2f, 1.10f}, {4.5f, 3.75f, 2.0f, 3.57f}},
                                     {{4.6f, 2.16f, 3.6f, 2.34f}, {5.4f, 6.27f, 3.6f, 6.77f}},
                                     {{4.1f, 1.24f, 2.3f, 0.80f}, {4.4f, 2.07f, 1.5f, 1.93f}}};
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
