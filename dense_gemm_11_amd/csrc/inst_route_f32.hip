// Routing from fp32 logits.
#include "route_variants.hpp"

namespace dg {

RouteFn route_fn_f32(bool lanes64, int v, bool bias) { return route_fn<float>(lanes64, v, bias); }

}  // namespace dg
