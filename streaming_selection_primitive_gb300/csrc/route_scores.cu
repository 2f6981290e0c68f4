// Launch of the choice by scores and bias (route.cuh).
#include "route.cuh"

namespace profk {

cudaError_t launch_route_scores(const RouteArgs& a, cudaStream_t stream) { return launch_forward<true>(a, stream); }

}  // namespace profk
