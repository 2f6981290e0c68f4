// C-ABI of the language-model selections: argument checks, then one launcher
// (tokens.cu, route.cu, route_scores.cu).  Nothing here waits for the device.
#include <cmath>

#include "../../include/profk.h"
#include "lm.h"

namespace profk {
namespace {

int64_t type_size(int type) { return type == PROFK_F32 ? 4 : 2; }

bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

bool type_ok(int type) { return type == PROFK_F32 || type == PROFK_BF16 || type == PROFK_F16; }

int status(cudaError_t e) { return e == cudaSuccess ? PROFK_OK : PROFK_ERR_CUDA; }

// A library call may throw (std::bad_alloc in the pool's bookkeeping); nothing
// crosses the ABI.
template <typename F>
int guarded(F&& f) {
  try {
    return status(f());
  } catch (...) {
    return PROFK_ERR_CUDA;
  }
}

bool sigmoid(const profk_routing* how) { return (how->score & ~PROFK_BIAS_ON_SCORES) == PROFK_SCORE_SIGMOID; }

// The limits that routing and its gradient share.
int check_route(const void* logits, int type, int64_t tokens, int64_t experts, int64_t ld, int64_t k,
                const profk_routing* how) {
  if (!how || !type_ok(type) || tokens < 0 || experts < 1 || ld < experts || k < 1 || k > experts)
    return PROFK_ERR_INVALID;
  const int score = how->score & ~PROFK_BIAS_ON_SCORES;
  if (score != PROFK_SCORE_SOFTMAX && score != PROFK_SCORE_SIGMOID) return PROFK_ERR_INVALID;
  if (tokens > 0 && !logits) return PROFK_ERR_INVALID;
  if (experts > ROUTE_MAX_EXPERTS || k > ROUTE_MAX_K || tokens >= (int64_t(1) << 32)) return PROFK_ERR_UNSUPPORTED;
  if (!aligned(logits, type_size(type))) return PROFK_ERR_UNSUPPORTED;
  return PROFK_OK;
}

}  // namespace
}  // namespace profk

using namespace profk;

extern "C" {

int profk_sample_tokens(const void* logits, int type, int64_t rows, int64_t n, int64_t ld, const float* noise,
                        int64_t noise_ld, const uint32_t* mask, int64_t mask_ld, const profk_sampling* how,
                        int64_t* out_tokens, float* out_logprobs, cudaStream_t stream) {
  if (!how || !type_ok(type) || rows < 0 || n < 1 || ld < n || (noise_ld != 0 && noise_ld < n)) return PROFK_ERR_INVALID;
  if (mask && mask_ld < (n + 31) / 32 && mask_ld != 0) return PROFK_ERR_INVALID;
  if (!how->temperature && !(how->all_temperature >= 0.f)) return PROFK_ERR_INVALID;
  if ((!how->top_p && std::isnan(how->all_top_p)) || (!how->min_p && std::isnan(how->all_min_p)))
    return PROFK_ERR_INVALID;
  if (n >= (int64_t(1) << 30) || rows >= (int64_t(1) << 28)) return PROFK_ERR_UNSUPPORTED;
  if (rows == 0) return PROFK_OK;
  if (!logits || !noise || !out_tokens || !out_logprobs) return PROFK_ERR_INVALID;
  if (!aligned(logits, type_size(type)) || !aligned(noise, 4) || !aligned(mask, 4) || !aligned(out_tokens, 8) ||
      !aligned(out_logprobs, 4) || !aligned(how->temperature, 4) || !aligned(how->top_k, 4) ||
      !aligned(how->top_p, 4) || !aligned(how->min_p, 4))
    return PROFK_ERR_UNSUPPORTED;
  const TokenArgs a{logits, type, rows, n, ld, noise, noise_ld, mask, mask_ld, how->temperature, how->top_k, how->top_p,
                    how->min_p, how->all_temperature, how->all_top_k, how->all_top_p, how->all_min_p, out_tokens,
                    out_logprobs};
  return guarded([&] { return launch_sample_tokens(a, stream); });
}

int profk_route(const void* logits, int type, int64_t tokens, int64_t experts, int64_t ld, int64_t k,
                const profk_routing* how, float* out_gates, int64_t* out_experts, int64_t* out_counts, float* out_loss,
                cudaStream_t stream) {
  const int bad = check_route(logits, type, tokens, experts, ld, k, how);
  if (bad != PROFK_OK) return bad;
  if (!out_counts || (tokens > 0 && (!out_gates || !out_experts))) return PROFK_ERR_INVALID;
  if (!aligned(out_gates, 4) || !aligned(out_experts, 8) || !aligned(out_counts, 8) || !aligned(out_loss, 4) ||
      !aligned(how->bias, 4))
    return PROFK_ERR_UNSUPPORTED;
  const RouteArgs a{logits, type, tokens, static_cast<int>(experts), ld, static_cast<int>(k),
                    sigmoid(how), how->normalize != 0, (how->score & PROFK_BIAS_ON_SCORES) != 0, how->bias, how->mask, out_gates,
                    out_experts, out_counts, out_loss};
  return guarded([&] { return launch_route(a, stream); });
}

int profk_route_backward(const void* logits, int type, int64_t tokens, int64_t experts, int64_t ld, int64_t k,
                         const profk_routing* how, const int64_t* chosen, const int64_t* counts,
                         const float* grad_gates, const float* grad_loss, void* grad_logits, int64_t grad_ld,
                         cudaStream_t stream) {
  const int bad = check_route(logits, type, tokens, experts, ld, k, how);
  if (bad != PROFK_OK) return bad;
  if (grad_ld < experts || (grad_loss && !counts)) return PROFK_ERR_INVALID;
  if (tokens == 0) return PROFK_OK;
  if (!chosen || !grad_logits) return PROFK_ERR_INVALID;
  if (!aligned(chosen, 8) || !aligned(counts, 8) || !aligned(grad_gates, 4) || !aligned(grad_loss, 4) ||
      !aligned(grad_logits, type_size(type)))
    return PROFK_ERR_UNSUPPORTED;
  const RouteBackwardArgs a{logits, type, tokens, static_cast<int>(experts), ld, static_cast<int>(k),
                            sigmoid(how), how->normalize != 0, chosen, counts, grad_gates,
                            grad_loss, grad_logits, grad_ld};
  return guarded([&] { return launch_route_backward(a, stream); });
}

}  // extern "C"
