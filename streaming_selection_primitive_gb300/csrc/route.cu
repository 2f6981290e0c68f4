// Launches of the choice by logits and bias, and of the gradient (route.cuh).
#include "route.cuh"

namespace profk {

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  return a.on_scores && a.bias ? launch_route_scores(a, stream) : launch_forward<false>(a, stream);
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t stream) {
  return by_type(a.type, [&](auto type) {
    return by_width(a.experts, [&](auto width) {
      return by_score(a.sigmoid, [&](auto sig) {
        using T = decltype(type);
        constexpr int R = decltype(width)::value;
        constexpr size_t smem = size_t(WARPS<R>) * (Ring<T, R>::BYTES + 32 * R * 4);
        return launch_with(k_route_backward<T, R, decltype(sig)::value>, route_grid(a.tokens, WARPS<R>, PER_SM<R>),
                           WARPS<R> * 32, smem, smem, stream, a);
      });
    });
  });
}

}  // namespace profk
