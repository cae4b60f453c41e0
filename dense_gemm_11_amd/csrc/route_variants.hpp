// Launch tables of the routing kernels (route.hpp), for the files that
// instantiate them for one type of logits each.
#pragma once

#include "route.hpp"

namespace dg {

typedef void (*RouteFn)(RouteArgs);

// Kernels of L lanes to a token and 1 << v experts to a lane (v 0 to 5), by
// whether the choice is compared in 64 bits.
RouteFn route_fn_f32(bool lanes64, int v, bool wide);
RouteFn route_fn_bf16(bool lanes64, int v, bool wide);

template <typename X, int L, typename K>
RouteFn route_fn_of(int v)
{
    switch (v) {
    case 0: return route_kernel<X, L, 1, K>;
    case 1: return route_kernel<X, L, 2, K>;
    case 2: return route_kernel<X, L, 4, K>;
    case 3: return route_kernel<X, L, 8, K>;
    case 4: return route_kernel<X, L, 16, K>;
    default: return route_kernel<X, L, 32, K>;
    }
}

template <typename X>
RouteFn route_fn(bool lanes64, int v, bool wide)
{
    if (lanes64) return wide ? route_fn_of<X, 64, double>(v) : route_fn_of<X, 64, float>(v);
    return wide ? route_fn_of<X, 16, double>(v) : route_fn_of<X, 16, float>(v);
}

}  // namespace dg
