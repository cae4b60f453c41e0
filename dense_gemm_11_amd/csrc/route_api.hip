// C ABI of the routing to experts: argument validation and launches.  Declared
// in include/dense_gemm.h.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdio>

#include "handle.hpp"
#include "route_plan.hpp"
#include "route_variants.hpp"

namespace dg {
namespace {

// Tokens, so that no launch has 2^32 threads (64 to a token) and 32 bits number
// tokens x ROUTE_MAX_TOP.
constexpr int64_t MAX_TOKENS = ((int64_t)1 << 26) - 64;
static_assert(MAX_TOKENS * ROUTE_MAX_TOP <= INT_MAX, "32-bit assignments");

// Tokens that share a count by expert, where one workgroup does not take them all:
// as few as make at most ROUTE_SUPER chunks, so the second launch needs no sums of
// sums, and 64 beyond (8192 tokens of 256 experts in groups with a bias by 32 and by
// 64: 13.4 us and 15.5; 2048 by 8 and by 16: 11.8 and 11.0).
int route_chunk(int64_t tokens)
{
    int chunk = 4;
    while (chunk < ROUTE_CHUNK && tokens > chunk * ROUTE_SUPER) chunk = std::max(2 * chunk, 16);
    return chunk;
}

bool ints_ok(const void* p) { return aligned_to(p, 4); }

// The gradient's kernel: one quad of experts to a lane, or four.
typedef void (*GradFn)(RouteGradArgs);
template <typename X>
GradFn grad_fn(bool lanes64, int experts, bool dense)
{
    if (lanes64) {
        if (experts <= 256) return dense ? route_grad_kernel<X, 64, 1, true> : route_grad_kernel<X, 64, 1, false>;
        return dense ? route_grad_kernel<X, 64, 4, true> : route_grad_kernel<X, 64, 4, false>;
    }
    if (experts <= 64) return dense ? route_grad_kernel<X, 16, 1, true> : route_grad_kernel<X, 16, 1, false>;
    return dense ? route_grad_kernel<X, 16, 4, true> : route_grad_kernel<X, 16, 4, false>;
}

gemm_status_t check_routing(const gemm_routing_t* r)
{
    if (!r || (r->scores != GEMM_SCORES_SOFTMAX && r->scores != GEMM_SCORES_SIGMOID))
        return GEMM_ERR_INVALID_VALUE;
    if (r->experts < 1 || r->top < 1 || r->top > r->experts || r->groups < 0 || !(std::isfinite(r->scale)))
        return GEMM_ERR_INVALID_VALUE;
    if (r->experts > ROUTE_MAX_EXPERTS || r->top > ROUTE_MAX_TOP) return GEMM_ERR_NOT_SUPPORTED;
    return GEMM_OK;
}

}  // namespace
}  // namespace dg

extern "C" {

size_t gemm_route_workspace_bytes(int64_t tokens, int experts)
{
    using namespace dg;
    if (tokens <= 0 || experts <= 0) return 0;
    // does not decrease with the tokens: up to ROUTE_SUPER chunks of any size
    const int64_t chunks = std::max<int64_t>(std::min<int64_t>(ceil_div(tokens, 4), ROUTE_SUPER),
                                             ceil_div(tokens, ROUTE_CHUNK));
    const int64_t counts = ceil_div(chunks * (ceil_div(experts, 4) * 4), 256) * 256;
    return (size_t)(counts + ceil_div(chunks, ROUTE_SUPER) * experts * 4);
}

gemm_status_t gemm_route(gemm_handle_t h, int64_t tokens, const void* logits, int64_t ld,
                         gemm_dtype_t dtype, const gemm_routing_t* routing, int32_t* ids, float* weights,
                         int32_t* offsets, int32_t* order, int32_t* position, void* ws,
                         size_t ws_bytes, hipStream_t stream)
{
    using namespace dg;
    if (!h || tokens < 0) return GEMM_ERR_INVALID_VALUE;
    if (dtype != GEMM_DTYPE_F32 && dtype != GEMM_DTYPE_BF16_F32 && dtype != GEMM_DTYPE_BF16_BF16)
        return GEMM_ERR_INVALID_VALUE;
    const gemm_status_t st = check_routing(routing);
    if (st != GEMM_OK) return st;
    const gemm_routing_t& r = *routing;
    const bool bf16 = dtype == GEMM_DTYPE_BF16_BF16;
    const int groups = std::max(r.groups, 1);
    if (ld < r.experts) return GEMM_ERR_INVALID_VALUE;
    if (groups > 1 && (r.experts % groups != 0 || r.top_groups < 1 || r.top_groups > groups ||
                       (r.group_top != 1 && r.group_top != 2) ||
                       (int64_t)r.top_groups * (r.experts / groups) < r.top))
        return GEMM_ERR_INVALID_VALUE;
    const bool plan = offsets || order || position;
    if (plan && (!offsets || (tokens > 0 && (!order || !position)))) return GEMM_ERR_INVALID_VALUE;
    if (tokens > 0 && (!logits || !ids || !weights)) return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0 && !plan) return GEMM_OK;
    if (groups > 64 || tokens > MAX_TOKENS || ld > INT_MAX) return GEMM_ERR_NOT_SUPPORTED;
    if (!aligned_to(logits, bf16 ? 2 : 4) || !ints_ok(ids) || !ints_ok(weights) || !ints_ok(offsets) ||
        !ints_ok(order) || !ints_ok(position) || !ints_ok(r.bias))
        return GEMM_ERR_NOT_SUPPORTED;

    const int64_t es = bf16 ? 2 : 4, chosen = tokens * r.top * 4;
    if (written_overlap({{ids, chosen}, {weights, chosen}, {offsets, ((int64_t)r.experts + 1) * 4}, {order, chosen},
                         {position, chosen}, {plan && tokens > 16 ? ws : nullptr, (int64_t)gemm_route_workspace_bytes(tokens, r.experts)},
                         {logits, ((tokens - 1) * ld + r.experts) * es}, {r.bias, (int64_t)r.experts * 4}}, 6))
        return GEMM_ERR_INVALID_VALUE;

    RouteArgs a{};
    a.logits = logits;
    a.bias = r.bias;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.order = plan ? (order ? order : offsets) : nullptr;  // (no tokens: nothing is written to it)
    a.position = position;
    a.ld = ld;
    a.tokens = (int)tokens;
    a.experts = r.experts;
    a.top = r.top;
    a.groups = groups;
    a.group_size = r.experts / groups;
    a.top_groups = r.top_groups;
    a.group_top = r.group_top;
    a.sigmoid = r.scores == GEMM_SCORES_SIGMOID;
    a.renormalize = r.renormalize != 0;
    a.scale = r.scale;
    // 16 lanes to a token where they have room (for a candidate more than are chosen,
    // too; 32 scores and biases to a lane spill): few lanes to a token take fewer
    // instructions, but a single token, or a token to each SIMD and no more, is
    // sooner done in 64 (one of 256 experts in groups with a bias 5.7 us, in 16 lanes
    // 6.8; 17 of 64 experts 6.2, in 16 3.9; 1024 of 256 experts 9.9, in 16 10.5, and
    // 2048 of them 10.5, in 16 9.6).
    int padded = 1;
    while (padded < groups) padded *= 2;
    auto per_lane = [&](int lanes) {  // log2 of the experts to a lane (in 64 lanes: 5 at most)
        int v = 0;
        while ((1 << v) * (lanes / padded) < a.group_size) ++v;
        return v;
    };
    const bool fits16 = padded <= 16 && r.top < 16 && per_lane(16) <= (r.bias ? 4 : 5);
    // One workgroup makes the plan with the choice (a launch less: 2.5 us for the
    // host) until its passes take longer than that: 96 tokens of 64 experts 6.5 us
    // against 7.1, 64 of 256 experts 8.0 against 7.7 and 96 of them 12.7 against 8.6, 32
    // of 256 in groups with a bias 6.8 against 8.4 and 64 of them 11.3 against 9.8.
    // (64 of 256 experts gain by it in eager calls alone: a replayed graph's host
    // time is none, and there they lose 0.3 us.)
    const bool one = tokens <= 16 ||  // (which is what needs no workspace)
                     (fits16 && tokens <= ROUTE_ONE && tokens << per_lane(16) <= (r.bias ? 512 : 1024));
    const bool lanes64 = !fits16 || tokens <= 4 || (!one && tokens <= 4 * ROUTE_SUPER);
    a.lanes_per_group = (lanes64 ? 64 : 16) / padded;
    const int v = per_lane(lanes64 ? 64 : 16);
    a.chunk = one ? ROUTE_ONE : route_chunk(tokens);
    a.chunks = (int)std::max<int64_t>(1, ceil_div(tokens, a.chunk));
    a.count_ld = (int)ceil_div(r.experts, 4) * 4;
    // (by the tokens alone, so that a call's needs do not turn on the choice above)
    if (plan && tokens > 16) {
        if (!ws || !aligned_to(ws, 256) || ws_bytes < gemm_route_workspace_bytes(tokens, r.experts))
            return GEMM_ERR_INVALID_VALUE;
        a.counts = static_cast<uint8_t*>(ws);
        a.supers = reinterpret_cast<int32_t*>(a.counts +
                                              ceil_div((int64_t)a.chunks * a.count_ld, 256) * 256);
    }
    if (h->fail_launch) return GEMM_ERR_HIP;
    // a workgroup's threads: its chunk at once, or in passes of 16 waves
    const int threads = (int)std::min<int64_t>(1024, std::max<int64_t>(1, std::min<int64_t>(tokens, a.chunk)) *
                                                         (lanes64 ? 64 : 16) + 63) / 64 * 64;
    const RouteFn fn = bf16 ? route_fn_bf16(lanes64, v, r.bias) : route_fn_f32(lanes64, v, r.bias);
    void* args[] = {&a};
    if (hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3(a.chunks), dim3(threads), args, 0, stream) !=
        hipSuccess)
        return GEMM_ERR_HIP;
    if (plan && a.chunks > 1) {
        const int supers = (int)ceil_div(a.chunks, ROUTE_SUPER);
        if (supers > 1 && hipLaunchKernel(reinterpret_cast<const void*>(route_super), dim3(supers),
                                          dim3(1024), args, 0, stream) != hipSuccess)
            return GEMM_ERR_HIP;
        if (hipLaunchKernel(reinterpret_cast<const void*>(route_place), dim3(a.chunks), dim3(1024), args, 0,
                            stream) != hipSuccess)
            return GEMM_ERR_HIP;
    }
    if (h->log)
        std::fprintf(stderr, "gemm: route tokens=%d experts=%d top=%d lanes=%d per lane=%d chunks=%d\n",
                     a.tokens, a.experts, a.top, lanes64 ? 64 : 16, 1 << v, a.chunks);
    return GEMM_OK;
}

gemm_status_t gemm_route_grad(gemm_handle_t h, int64_t tokens, const void* logits, int64_t ld,
                              gemm_dtype_t dtype, const gemm_routing_t* routing, const int32_t* ids,
                              const float* dweights, void* dlogits, int64_t ldd, hipStream_t stream)
{
    using namespace dg;
    if (!h || tokens < 0) return GEMM_ERR_INVALID_VALUE;
    if (dtype != GEMM_DTYPE_F32 && dtype != GEMM_DTYPE_BF16_F32 && dtype != GEMM_DTYPE_BF16_BF16)
        return GEMM_ERR_INVALID_VALUE;
    const gemm_status_t st = check_routing(routing);
    if (st != GEMM_OK) return st;
    const gemm_routing_t& r = *routing;
    const int64_t es = dtype == GEMM_DTYPE_BF16_BF16 ? 2 : 4;
    if (ld < r.experts || ldd < r.experts) return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0) return GEMM_OK;
    if (!logits || !ids || !dweights || !dlogits) return GEMM_ERR_INVALID_VALUE;
    if (tokens > MAX_TOKENS || ld > INT_MAX || ldd > INT_MAX) return GEMM_ERR_NOT_SUPPORTED;
    if (written_overlap({{dlogits, ((tokens - 1) * ldd + r.experts) * es},
                         {logits, ((tokens - 1) * ld + r.experts) * es}, {ids, tokens * r.top * 4},
                         {dweights, tokens * r.top * 4}}, 1))
        return GEMM_ERR_INVALID_VALUE;
    if (!aligned_to(logits, es) || !aligned_to(dlogits, es) || !ints_ok(ids) || !ints_ok(dweights))
        return GEMM_ERR_NOT_SUPPORTED;
    const int row = (int)ceil_div(r.experts, 4) * 4;
    RouteGradArgs a{logits, ids, dweights, dlogits, ld, ldd, (int)tokens, r.experts, r.top, row,
                    r.scores == GEMM_SCORES_SIGMOID, r.renormalize != 0, r.scale};
    const bool lanes64 = r.top > 16 || r.experts > 256 || tokens <= 4 * ROUTE_SUPER;
    const int per = lanes64 ? 4 : 16;
    const bool dense = !a.sigmoid && !a.renormalize;
    if (h->fail_launch) return GEMM_ERR_HIP;
    const GradFn fn = es == 2 ? grad_fn<bf16_t>(lanes64, r.experts, dense) : grad_fn<float>(lanes64, r.experts, dense);
    void* args[] = {&a};
    if (hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)ceil_div(tokens, per)), dim3(256),
                        args, (size_t)per * row * 4, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    if (h->log)
        std::fprintf(stderr, "gemm: route grad tokens=%d experts=%d top=%d\n", a.tokens, a.experts, a.top);
    return GEMM_OK;
}

}  // extern "C"
