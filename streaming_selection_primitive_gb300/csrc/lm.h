// Host-side launchers of the language-model selections (internal interface).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace profk {

// The library's stream-ordered memory pool of the current device (api.cu).
cudaError_t library_pool(cudaMemPool_t* out);
int sms();  // SMs of the current device
struct WaitCfg;
WaitCfg head_wait();  // test setting of head.cu's waits (PROFK_OPT_HEAD_WAIT_TEST)

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

// Log-probabilities of given tokens, their gradient, and the losses on them (logprobs.cu).
struct LogprobArgs {
  const void* logits;  // rows of n values, row stride ld
  int type;            // a profk_type
  int64_t rows, n, ld;
  const int64_t* tokens;     // negative: the row is left out
  const float* temperature;  // per row, or null: all_temperature
  float all_temperature;
  float* logprobs;
  float* entropies;        // or null
  float2* stats;           // or null: largest logit, sum of exp((l - largest) / T)
  float* lacks;            // or null: what each log-probability lacks as a float (0 of a row left out)
  const float* weights;    // or null; a row of weight 0 is left out
  const int64_t* offsets;  // or null; sequences + 1 of them: rows before the first and from the last on are left out
  int64_t sequences;
  void* grad_logits;  // with the policy loss, or null: rows of n values, row stride grad_ld
  int64_t grad_ld;
};
cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream);

struct LogprobBackwardArgs {
  const void* logits;
  int type;
  int64_t rows, n, ld;
  const int64_t* tokens;
  const float* temperature;
  float all_temperature;
  const float2* stats;
  const float* entropies;       // null when grad_entropies is
  const float* grad_logprobs;   // or null
  const float* grad_entropies;  // or null
  const float* scale;           // one float for both, or null
  void* grad_logits;
  int64_t grad_ld;
};
cudaError_t launch_token_logprobs_backward(const LogprobBackwardArgs& a, cudaStream_t stream);

struct PolicyHow {
  const float* old_logprobs;
  const float* advantages;
  const float* ref_logprobs;  // or null: no KL term
  const float* weights;       // or null: all_weight
  float all_weight, clip_low, clip_high, kl, entropy;
};
struct PolicyOut {
  float* loss;
  float* sums;  // three floats: weighted sums of KL terms, of clipped tokens, of entropies
  float* slopes;
  float* entropy_slopes;  // or null
};
cudaError_t launch_policy_loss(const LogprobArgs& a, const PolicyHow& how, const PolicyOut& out, cudaStream_t stream);

struct PreferenceHow {
  const float* ref_logprobs;  // or null
  float beta, smoothing, margin;
  bool average;
};
struct PreferenceOut {
  float* loss;
  float* margins;
  float* slopes;
};
cudaError_t launch_preference_loss(const LogprobArgs& a, const PreferenceHow& how, const PreferenceOut& out, cudaStream_t stream);

// The same log-probabilities from hidden states and the output matrix (head.cu).
struct HeadArgs {
  const void* hidden;  // rows of `width` values, row stride hidden_ld
  const void* weight;  // n rows of `width` values, row stride weight_ld
  int type;            // PROFK_BF16 or PROFK_F16
  int64_t rows, n, width, hidden_ld, weight_ld;
  const int64_t* tokens;
  const float* temperature;
  float all_temperature;
  float* logprobs;
  float* entropies;  // or null
};
cudaError_t launch_head_logprobs(const HeadArgs& a, cudaStream_t stream);

}  // namespace profk
