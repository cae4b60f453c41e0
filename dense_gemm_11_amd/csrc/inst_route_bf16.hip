// Routing from bf16 logits.
#include "route_variants.hpp"

namespace dg {

RouteFn route_fn_bf16(bool lanes64, int v, bool bias) { return route_fn<bf16_t>(lanes64, v, bias); }

}  // namespace dg
