// Host-side launchers of the language-model selections (internal interface).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace profk {

// The library's stream-ordered memory pool of the current device (api.cu).
cudaError_t library_pool(cudaMemPool_t* out);
int sms();  // SMs of the current device

// Choice of one token per row (tokens.cu).
struct TokenArgs {
  const void* logits;  // rows of n values, row stride ld
  int type;            // a profk_type
  int64_t rows, n, ld;
  const float* noise;  // rows of n values, row stride noise_ld
  int64_t noise_ld;
  const uint32_t* mask;  // packed, row stride mask_ld words; null: everything is allowed
  int64_t mask_ld;
  const float* temperature;  // per row, or null: the `all_` value
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  float all_temperature;
  int32_t all_top_k;
  float all_top_p;
  float all_min_p;
  int64_t* out_tokens;
  float* out_logprobs;
};
cudaError_t launch_sample_tokens(const TokenArgs& a, cudaStream_t stream);

// Choice of k experts per token (route.cuh).
constexpr int ROUTE_MAX_EXPERTS = 1024;
constexpr int ROUTE_MAX_K = 32;
struct RouteArgs {
  const void* logits;  // tokens rows of `experts` values, row stride ld
  int type;            // a profk_type
  int64_t tokens;
  int experts;
  int64_t ld;
  int k;
  bool sigmoid, normalize, on_scores;  // on_scores: the bias is added to the scores, not to the logits
  const float* bias;    // experts, or null
  const uint8_t* mask;  // tokens, or null
  float* gates;         // tokens x k
  int64_t* chosen;      // tokens x k
  int64_t* counts;      // experts
  float* loss;          // one float, or null
};
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream);
cudaError_t launch_route_scores(const RouteArgs& a, cudaStream_t stream);  // on_scores, with a bias

struct RouteBackwardArgs {
  const void* logits;
  int type;
  int64_t tokens;
  int experts;
  int64_t ld;
  int k;
  bool sigmoid, normalize;
  const int64_t* chosen;
  const int64_t* counts;    // null when grad_loss is
  const float* grad_gates;  // tokens x k, or null
  const float* grad_loss;   // one float, or null
  void* grad_logits;        // tokens rows of `experts` values, row stride grad_ld
  int64_t grad_ld;
};
cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t stream);

}  // namespace profk
