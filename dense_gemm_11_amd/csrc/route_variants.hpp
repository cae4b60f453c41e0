// Launch tables of the routing kernels (route.hpp), for the files that
// instantiate them for one type of logits each.
#pragma once

#include "route.hpp"

namespace dg {

typedef void (*RouteFn)(RouteArgs);

// Kernels of L lanes to a token and 1 << v experts to a lane (v 0 to 5), by
// whether there is a bias.
RouteFn route_fn_f32(bool lanes64, int v, bool bias);
RouteFn route_fn_bf16(bool lanes64, int v, bool bias);

template <typename X, int L, bool BIAS>
RouteFn route_fn_of(int v)
{
    switch (v) {
    case 0: return route_kernel<X, L, 1, BIAS>;
    case 1: return route_kernel<X, L, 2, BIAS>;
    case 2: return route_kernel<X, L, 4, BIAS>;
    case 3: return route_kernel<X, L, 8, BIAS>;
    case 4: return route_kernel<X, L, 16, BIAS>;
    default: return route_kernel<X, L, 32, BIAS>;
    }
}

template <typename X>
RouteFn route_fn(bool lanes64, int v, bool bias)
{
    if (lanes64) return bias ? route_fn_of<X, 64, true>(v) : route_fn_of<X, 64, false>(v);
    return bias ? route_fn_of<X, 16, true>(v) : route_fn_of<X, 16, false>(v);
}

}  // namespace dg
