// The first product of the low-rank adapters, T = s X op(down) (lora.hpp).
#include "lora.hpp"
#include "ragged_variants.hpp"

#include <algorithm>

namespace dg {

namespace {

template <typename T, int RF, int NF, bool KC>
hipError_t launch(const RaggedArgs& a, const ShrinkCall& c, hipStream_t s)
{
    constexpr int BM = 16 * RF;
    // the most blocks of BM rows any split of the rows into segments needs
    const int64_t segs = std::min(a.groups, a.rows);
    const int64_t blocks = ((int64_t)a.rows + segs * (BM - 1)) / BM;
    const int zs = (a.rank_pad + 16 * NF - 1) / (16 * NF);
    RaggedArgs p = a;
    const void* down = c.down;
    int64_t ld = c.ld_down, stride = c.stride_down;
    int slice = c.k_slice;
    float* t = c.t;
    void* args[] = {&p, &down, &ld, &stride, &slice, &t};
    return hipLaunchKernel(reinterpret_cast<const void*>(&lora_shrink_kernel<T, RF, NF, KC>),
                           dim3((unsigned)blocks, c.splits, zs), dim3(64 * SHRINK_WAVES), args, 0,
                           s);
}

template <typename T, int RF, bool KC>
hipError_t by_rank(const RaggedArgs& a, const ShrinkCall& c, hipStream_t s)
{
    if (a.rank <= 16) return launch<T, RF, 1, KC>(a, c, s);
    if (a.rank <= 32) return launch<T, RF, 2, KC>(a, c, s);
    return launch<T, RF, 4, KC>(a, c, s);
}

template <typename T>
hipError_t by_layout(const RaggedArgs& a, const ShrinkCall& c, hipStream_t s)
{
    if (c.tall) return c.down_kc ? by_rank<T, 2, true>(a, c, s) : by_rank<T, 2, false>(a, c, s);
    return c.down_kc ? by_rank<T, 1, true>(a, c, s) : by_rank<T, 1, false>(a, c, s);
}

}  // namespace

hipError_t launch_shrink(const RaggedArgs& a, const ShrinkCall& c, bool bf16, hipStream_t s)
{
    return bf16 ? by_layout<bf16_t>(a, c, s) : by_layout<float>(a, c, s);
}

}  // namespace dg
