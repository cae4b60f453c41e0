// Direct-to-LDS configurations of the ragged and adapted products beyond those
// of selected_configs.hpp and tile_configs.hpp:
//
//  * bf16, 128x128 tiles with adapters: the selected ring, held to the registers
//    of two workgroups per compute unit;
//  * bf16, 64x128 tiles: 4 waves, three 64-deep stages (72 KiB, two workgroups
//    per compute unit);
//  * bf16, 128x128 tiles of two stages, three workgroups per compute unit;
//  * fp32, 64x128 tiles: 4 waves, three 16-deep stages.
#pragma once

#include "selected_configs.hpp"
#include "tile_configs.hpp"

namespace dg {

using RagBf16Mid = DmaConfig<MFMA_BF16_32x32x16, 128, 128, 32, 2, 2, 4, true, PAIR_NONE, 2>;
using RagBf16Thin = DmaConfig<MFMA_BF16_32x32x16, 128, 128, 32, 2, 2, 2, true, PAIR_NONE, 3>;
using RagBf16Low = DmaConfig<MFMA_BF16_32x32x16, 64, 128, 64, 2, 2, 3, true>;
using RagF32Low = DmaConfig<MFMA_F32_32x32x2, 64, 128, 16, 2, 2, 3, true>;

}  // namespace dg
