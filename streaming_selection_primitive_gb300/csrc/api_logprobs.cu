// C-ABI of the log-probabilities and the losses on them: argument checks, then one
// launcher (logprobs.cu, head.cu).  Nothing here waits for the device.
#include <cmath>

#include "../../include/profk.h"
#include "lm.h"

namespace profk {
namespace {

bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <typename... P>
bool floats(const P*... p) {
  return (aligned(p, 4) && ...);
}

int64_t type_size(int type) { return type == PROFK_F32 ? 4 : 2; }

bool type_ok(int type) { return type == PROFK_F32 || type == PROFK_BF16 || type == PROFK_F16; }

// Nothing that a library call throws crosses the ABI.
template <typename F>
int guarded(F&& f) {
  try {
    return f() == cudaSuccess ? PROFK_OK : PROFK_ERR_CUDA;
  } catch (...) {
    return PROFK_ERR_CUDA;
  }
}

bool temperature_ok(const float* temperature, float all) {
  return temperature || (all > 0.f && std::isfinite(all) && std::isfinite(1.44269504f / all) && 1.44269504f / all > 0.f);
}

// What the calls on logits share.
int check_rows(const void* logits, int type, int64_t rows, int64_t n, int64_t ld, const int64_t* tokens,
               const float* temperature, float all_temperature) {
  if (!type_ok(type) || rows < 0 || n < 1 || ld < n || !temperature_ok(temperature, all_temperature)) return PROFK_ERR_INVALID;
  if (rows > 0 && (!logits || !tokens)) return PROFK_ERR_INVALID;
  if (n >= (int64_t(1) << 30) || rows >= (int64_t(1) << 28)) return PROFK_ERR_UNSUPPORTED;
  if (!aligned(logits, type_size(type)) || !aligned(tokens, 8) || !floats(temperature)) return PROFK_ERR_UNSUPPORTED;
  return PROFK_OK;
}

int check_gradient(const void* logits, int type, int64_t rows, int64_t n, int64_t ld, const void* grad, int64_t grad_ld) {
  if (grad_ld < n) return PROFK_ERR_INVALID;
  if (!aligned(grad, type_size(type))) return PROFK_ERR_UNSUPPORTED;
  // The gradient may stand in the logits' place, but not across them.
  const auto size = type_size(type);
  const auto first = reinterpret_cast<uintptr_t>(logits), other = reinterpret_cast<uintptr_t>(grad);
  const auto bytes = [&](int64_t stride) { return static_cast<uintptr_t>(((rows - 1) * stride + n) * size); };
  if (rows > 0 && first < other + bytes(grad_ld) && other < first + bytes(ld) && !(first == other && (ld == grad_ld || rows == 1)))
    return PROFK_ERR_INVALID;
  return PROFK_OK;
}

LogprobArgs row_args(const void* logits, int type, int64_t rows, int64_t n, int64_t ld, const int64_t* tokens,
                     const float* temperature, float all_temperature, float* logprobs, float* entropies, float* stats) {
  LogprobArgs a{};
  a.logits = logits;
  a.type = type;
  a.rows = rows;
  a.n = n;
  a.ld = ld;
  a.tokens = tokens;
  a.temperature = temperature;
  a.all_temperature = all_temperature;
  a.logprobs = logprobs;
  a.entropies = entropies;
  a.stats = reinterpret_cast<float2*>(stats);
  return a;
}

}  // namespace
}  // namespace profk

using namespace profk;

extern "C" {

int profk_token_logprobs(const void* logits, int type, int64_t rows, int64_t n, int64_t ld, const int64_t* tokens,
                         const float* temperature, float all_temperature, float* out_logprobs, float* out_entropies,
                         float* out_stats, cudaStream_t stream) {
  const int bad = check_rows(logits, type, rows, n, ld, tokens, temperature, all_temperature);
  if (bad != PROFK_OK) return bad;
  if (rows == 0) return PROFK_OK;
  if (!out_logprobs) return PROFK_ERR_INVALID;
  if (!floats(out_logprobs, out_entropies) || !aligned(out_stats, 8)) return PROFK_ERR_UNSUPPORTED;
  return guarded([&] {
    return launch_token_logprobs(
        row_args(logits, type, rows, n, ld, tokens, temperature, all_temperature, out_logprobs, out_entropies, out_stats), stream);
  });
}

int profk_token_logprobs_backward(const void* logits, int type, int64_t rows, int64_t n, int64_t ld,
                                  const int64_t* tokens, const float* temperature, float all_temperature,
                                  const float* stats, const float* entropies, const float* grad_logprobs,
                                  const float* grad_entropies, const float* scale, void* grad_logits, int64_t grad_ld,
                                  cudaStream_t stream) {
  int bad = check_rows(logits, type, rows, n, ld, tokens, temperature, all_temperature);
  if (bad != PROFK_OK) return bad;
  if (grad_entropies && !entropies && rows > 0) return PROFK_ERR_INVALID;
  if (rows > 0 && (!stats || !grad_logits)) return PROFK_ERR_INVALID;
  bad = check_gradient(logits, type, rows, n, ld, grad_logits, grad_ld);
  if (bad != PROFK_OK) return bad;
  if (!floats(entropies, grad_logprobs, grad_entropies, scale) || !aligned(stats, 8)) return PROFK_ERR_UNSUPPORTED;
  if (rows == 0) return PROFK_OK;
  const LogprobBackwardArgs a{logits, type, rows, n, ld, tokens, temperature, all_temperature,
                              reinterpret_cast<const float2*>(stats), entropies, grad_logprobs, grad_entropies, scale, grad_logits, grad_ld};
  return guarded([&] { return launch_token_logprobs_backward(a, stream); });
}

int profk_head_logprobs(const void* hidden, const void* weight, int type, int64_t rows, int64_t n, int64_t width,
                        int64_t hidden_ld, int64_t weight_ld, const int64_t* tokens, const float* temperature,
                        float all_temperature, float* out_logprobs, float* out_entropies, cudaStream_t stream) {
  if ((type != PROFK_BF16 && type != PROFK_F16) || rows < 0 || n < 1 || width < 1 || hidden_ld < width || weight_ld < width ||
      !temperature_ok(temperature, all_temperature))
    return PROFK_ERR_INVALID;
  if (n >= (int64_t(1) << 30) || rows >= (int64_t(1) << 24) || width >= (int64_t(1) << 20)) return PROFK_ERR_UNSUPPORTED;
  if ((rows / 128 + 1) * (n / 256 + 1) >= (int64_t(1) << 30)) return PROFK_ERR_UNSUPPORTED;
  if (hidden_ld >= (int64_t(1) << 38) || weight_ld >= (int64_t(1) << 38)) return PROFK_ERR_UNSUPPORTED;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || hidden_ld % 8 || weight_ld % 8 || !aligned(tokens, 8) ||
      !floats(temperature, out_logprobs, out_entropies))
    return PROFK_ERR_UNSUPPORTED;
  if (rows == 0) return PROFK_OK;
  if (!hidden || !weight || !tokens || !out_logprobs) return PROFK_ERR_INVALID;
  const HeadArgs a{hidden, weight, type, rows, n, width, hidden_ld, weight_ld, tokens, temperature, all_temperature,
                   out_logprobs, out_entropies};
  return guarded([&] { return launch_head_logprobs(a, stream); });
}

int profk_policy_loss(const void* logits, int type, int64_t rows, int64_t n, int64_t ld, const int64_t* tokens,
                      const float* temperature, float all_temperature, const profk_policy* how, float* out_loss,
                      float* out_sums, float* out_logprobs, float* out_entropies, float* out_stats, float* out_slopes,
                      float* out_entropy_slopes, void* grad_logits, int64_t grad_ld, cudaStream_t stream) {
  int bad = check_rows(logits, type, rows, n, ld, tokens, temperature, all_temperature);
  if (bad != PROFK_OK) return bad;
  if (!how || !out_loss || !out_sums) return PROFK_ERR_INVALID;
  if (!(how->clip_low >= 0.f) || !(how->clip_high >= 0.f) || !std::isfinite(how->kl) || !std::isfinite(how->entropy))
    return PROFK_ERR_INVALID;
  if (rows > 0 && (!how->old_logprobs || !how->advantages || !out_logprobs || !out_stats || !out_slopes)) return PROFK_ERR_INVALID;
  if (rows > 0 && how->entropy != 0.f && !out_entropies) return PROFK_ERR_INVALID;
  if (!floats(how->old_logprobs, how->advantages, how->ref_logprobs, how->weights, out_loss, out_sums, out_logprobs, out_entropies,
              out_slopes, out_entropy_slopes) ||
      !aligned(out_stats, 8))
    return PROFK_ERR_UNSUPPORTED;
  LogprobArgs a = row_args(logits, type, rows, n, ld, tokens, temperature, all_temperature, out_logprobs, out_entropies, out_stats);
  if (grad_logits) {
    bad = check_gradient(logits, type, rows, n, ld, grad_logits, grad_ld);
    if (bad != PROFK_OK) return bad;
    a.grad_logits = grad_logits;
    a.grad_ld = grad_ld;
  }
  a.weights = how->weights;
  const PolicyHow h{how->old_logprobs, how->advantages, how->ref_logprobs, how->weights, rows > 0 ? 1.f / static_cast<float>(rows) : 0.f,
                    how->clip_low, how->clip_high, how->kl, how->entropy};
  return guarded([&] { return launch_policy_loss(a, h, PolicyOut{out_loss, out_sums, out_slopes, out_entropy_slopes}, stream); });
}

int profk_preference_loss(const void* logits, int type, int64_t rows, int64_t n, int64_t ld, const int64_t* tokens,
                          const float* temperature, float all_temperature, const int64_t* offsets, int64_t pairs,
                          const profk_preference* how, float* out_loss, float* out_margins, float* out_logprobs,
                          float* out_stats, float* out_slopes, cudaStream_t stream) {
  const int bad = check_rows(logits, type, rows, n, ld, tokens, temperature, all_temperature);
  if (bad != PROFK_OK) return bad;
  if (!how || pairs < 0 || !offsets || !out_loss || (pairs > 0 && !out_margins)) return PROFK_ERR_INVALID;
  if (!std::isfinite(how->beta) || !std::isfinite(how->margin) || !(how->label_smoothing >= 0.f && how->label_smoothing <= 1.f))
    return PROFK_ERR_INVALID;
  if (rows > 0 && (!out_logprobs || !out_stats || !out_slopes)) return PROFK_ERR_INVALID;
  if (pairs >= (int64_t(1) << 28)) return PROFK_ERR_UNSUPPORTED;
  if (!aligned(offsets, 8) || !floats(how->ref_logprobs, out_loss, out_margins, out_logprobs, out_slopes) || !aligned(out_stats, 8))
    return PROFK_ERR_UNSUPPORTED;
  LogprobArgs a = row_args(logits, type, rows, n, ld, tokens, temperature, all_temperature, out_logprobs, nullptr, out_stats);
  a.lacks = out_slopes;  // until the slopes are there
  a.offsets = offsets;
  a.sequences = 2 * pairs;
  const PreferenceHow h{how->ref_logprobs, how->beta, how->label_smoothing, how->margin, how->average != 0};
  return guarded([&] { return launch_preference_loss(a, h, PreferenceOut{out_loss, out_margins, out_slopes}, stream); });
}

}  // extern "C"
