// Host side of the C ABI of layer norm, distillation on held logits and logit
// processing: argument checks and the stream-ordered launches.  No device
// memory is allocated and nothing synchronises.
#include "lmhead.h"

#include <cmath>
#include <cstdint>

#include "operators.h"

using namespace lmh;

namespace {

static_assert(kF32 == LMHEAD_F32 && kBF16 == LMHEAD_BF16 && kF16 == LMHEAD_F16, "element types");

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 256;
constexpr int32_t kMaxWidth = 1 << 20;   // of a layer norm's rows
constexpr int32_t kMaxVocab = INT32_MAX - 1024;   // columns, tails and mask words are counted in 32 bits

bool known_type(int type) { return type == kF32 || type == kBF16 || type == kF16; }

size_t element_bytes(int type) { return type == kF32 ? 4 : 2; }

// A pointer that is not aligned to its element cannot be read as one.
bool aligned_to(const void* p, int type) {
  return (reinterpret_cast<uintptr_t>(p) & (element_bytes(type) - 1)) == 0;
}

// A result over one of the call's inputs needs that input's layout: a CTA writes its
// rows while others still read theirs.
bool clash(const void* in, int64_t in_ld, const void* out, int64_t out_ld, int64_t rows) {
  return in && in == out && rows > 1 && in_ld != out_ld;
}

bool positive(float v) { return std::isfinite(v) && v > 0.f; }

lmhead_status status_of(cudaError_t e) { return e == cudaSuccess ? LMHEAD_OK : LMHEAD_ERR_CUDA; }

// Partial column sums, then (wide rows) the rows' own sums.
size_t norm_partials(int64_t H) {
  return (2 * sizeof(float) * kNormPartials * static_cast<size_t>(H) + 255) / 256 * 256;
}

size_t norm_workspace(int64_t N, int64_t H) {
  return norm_partials(H) + (H > kNormWide ? sizeof(float2) * static_cast<size_t>(N) : 0);
}

lmhead_status check_norm(int64_t N, int32_t H, int x_type, int other_type, int param_type,
                         int64_t x_ld, int64_t other_ld) {
  if (N < 0 || H <= 0 || !known_type(x_type) || !known_type(other_type) || !known_type(param_type))
    return LMHEAD_ERR_INVALID_ARG;
  if (x_ld < H || other_ld < H) return LMHEAD_ERR_INVALID_ARG;
  if (N >= kMaxRows || H > kMaxWidth || (param_type != kF32 && param_type != x_type)) return LMHEAD_ERR_UNSUPPORTED;
  return LMHEAD_OK;
}

lmhead_status check_distill(const void* logits, int type, int64_t ld, const int32_t* top_ids,
                            const float* top_logits, int64_t T, int32_t V, int32_t K, float tau,
                            float teacher_tau) {
  if (T < 0 || V <= 0 || K <= 0 || !known_type(type) || ld < V || !positive(tau) ||
      !positive(teacher_tau))
    return LMHEAD_ERR_INVALID_ARG;
  if (T >= kMaxRows || V > kMaxVocab || K > kMaxTeacher) return LMHEAD_ERR_UNSUPPORTED;
  if (T == 0) return LMHEAD_OK;
  if (!logits || !top_ids || !top_logits) return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(logits, type)) return LMHEAD_ERR_UNSUPPORTED;
  return LMHEAD_OK;
}

// Arguments that lmhead_process_logits_fwd and _bwd share.
lmhead_status check_process(const ProcessLogits& a) {
  if (a.R < 0 || a.V <= 0 || !known_type(a.type) || a.ld < a.V || a.out_ld < a.V ||
      a.n_tokens < 0 || a.n_bias < 0 || a.M < 0)
    return LMHEAD_ERR_INVALID_ARG;
  if (a.R >= kMaxRows || a.V > kMaxVocab) return LMHEAD_ERR_UNSUPPORTED;
  if (a.R == 0) return LMHEAD_OK;
  if (!a.logits || !a.out) return LMHEAD_ERR_INVALID_ARG;
  // an empty list may have no address
  if (a.tokens ? !a.spans : a.spans && a.n_tokens > 0) return LMHEAD_ERR_INVALID_ARG;
  if (!a.spans && (a.repetition || a.frequency || a.presence)) return LMHEAD_ERR_INVALID_ARG;
  if (a.bias_offsets && a.n_bias > 0 && (!a.bias_ids || !a.bias_values))
    return LMHEAD_ERR_INVALID_ARG;
  if (!a.bias_offsets && (a.bias_ids || a.bias_values)) return LMHEAD_ERR_INVALID_ARG;
  if (!a.allowed && a.allowed_rows && a.M > 0) return LMHEAD_ERR_INVALID_ARG;
  if (a.allowed && !a.allowed_rows && a.M < a.R) return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(a.logits, a.type) || !aligned_to(a.out, a.type)) return LMHEAD_ERR_UNSUPPORTED;
  if (clash(a.logits, a.ld, a.out, a.out_ld, a.R)) return LMHEAD_ERR_INVALID_ARG;
  return LMHEAD_OK;
}

}  // namespace

extern "C" {

size_t lmhead_layernorm_workspace_size(int64_t N, int32_t H) {
  return N < 0 || N >= kMaxRows || H <= 0 || H > kMaxWidth ? 0 : norm_workspace(N, H);
}

lmhead_status lmhead_layernorm_fwd(const void* x, int x_type, int64_t x_ld, const void* weight,
                                   const void* bias, int param_type, int64_t N, int32_t H,
                                   float eps, void* y, int y_type, int64_t y_ld, float* mean,
                                   float* rstd, lmhead_stream_t stream) {
  const lmhead_status rc = check_norm(N, H, x_type, y_type, param_type, x_ld, y_ld);
  if (rc != LMHEAD_OK) return rc;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return LMHEAD_ERR_INVALID_ARG;
  if (y_type != x_type && !(x_type == kF32 && y_type == kBF16)) return LMHEAD_ERR_UNSUPPORTED;
  if (N == 0) return LMHEAD_OK;
  if (!x || !weight || !y) return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(x, x_type) || !aligned_to(y, y_type) || !aligned_to(weight, param_type) ||
      !aligned_to(bias, param_type))
    return LMHEAD_ERR_UNSUPPORTED;
  if (clash(x, x_ld, y, y_ld, N) || (x == y && x_type != y_type)) return LMHEAD_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const NormFwd a{x, x_type, x_ld, weight, bias, param_type, N, H, eps, y, y_type, y_ld, mean, rstd};
  return status_of(traced_launch("layernorm_fwd", s, [&] { return launch_norm_fwd(a, s); }));
}

lmhead_status lmhead_layernorm_bwd(const void* dy, int dy_type, int64_t dy_ld, const void* x,
                                   int x_type, int64_t x_ld, const void* weight, int param_type,
                                   const float* mean, const float* rstd, int64_t N, int32_t H,
                                   void* dx, int64_t dx_ld, float* d_weight, float* d_bias,
                                   int accumulate, void* workspace, size_t workspace_bytes,
                                   lmhead_stream_t stream) {
  const lmhead_status rc = check_norm(N, H, x_type, dy_type, param_type, x_ld, dy_ld);
  if (rc != LMHEAD_OK) return rc;
  if (dx && dx_ld < H) return LMHEAD_ERR_INVALID_ARG;
  if (dy_type != x_type && dy_type != kF32 && !(x_type == kF32 && dy_type == kBF16))
    return LMHEAD_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) {
    for (float* g : {d_weight, d_bias})
      if (g && !accumulate && cudaMemsetAsync(g, 0, sizeof(float) * static_cast<size_t>(H), s) != cudaSuccess)
        return LMHEAD_ERR_CUDA;
    return LMHEAD_OK;
  }
  if (!dy || !x || !weight || !mean || !rstd || (!dx && !d_weight && !d_bias))
    return LMHEAD_ERR_INVALID_ARG;
  if ((d_weight || d_bias) && !workspace) return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(dy, dy_type) || !aligned_to(x, x_type) || !aligned_to(dx, x_type) ||
      !aligned_to(weight, param_type) || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return LMHEAD_ERR_UNSUPPORTED;
  if ((d_weight || d_bias) && workspace_bytes < norm_workspace(N, H))
    return LMHEAD_ERR_WORKSPACE_TOO_SMALL;
  if (clash(x, x_ld, dx, dx_ld, N) || clash(dy, dy_ld, dx, dx_ld, N) || (dx == dy && dy_type != x_type))
    return LMHEAD_ERR_INVALID_ARG;
  // a workspace given for dx alone is used if it is large enough
  const bool room = workspace && workspace_bytes >= norm_workspace(N, H);
  float2* sums = room && H > kNormWide
                     ? reinterpret_cast<float2*>(static_cast<char*>(workspace) + norm_partials(H))
                     : nullptr;
  const NormBwd a{dy, dy_type, dy_ld, x, x_type, x_ld, weight, param_type, mean, rstd, N, H,
                  dx, dx_ld, d_weight, d_bias, accumulate ? 1 : 0, static_cast<float*>(workspace), sums};
  return status_of(traced_launch("layernorm_bwd", s, [&] { return launch_norm_bwd(a, s); }));
}

lmhead_status lmhead_distill_logits_fwd(const void* logits, int type, int64_t ld,
                                        const int32_t* top_ids, const float* top_logits,
                                        const float* teacher_lse, const uint8_t* loss_mask,
                                        int64_t T, int32_t V, int32_t K, float temperature,
                                        float teacher_temperature, float* loss, float* lse,
                                        lmhead_stream_t stream) {
  const lmhead_status rc = check_distill(logits, type, ld, top_ids, top_logits, T, V, K,
                                         temperature, teacher_temperature);
  if (rc != LMHEAD_OK) return rc;
  if (T == 0) return LMHEAD_OK;
  if (!loss || !lse) return LMHEAD_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DistillLogits a{};
  a.logits = logits;
  a.type = type;
  a.ld = ld;
  a.teacher = {top_ids, top_logits, teacher_lse, K, teacher_temperature};
  a.mask = loss_mask;
  a.T = T;
  a.V = V;
  a.tau = temperature;
  a.loss = loss;
  a.lse = lse;
  return status_of(traced_launch("distill_logits_fwd", s, [&] { return launch_distill_logits_fwd(a, s); }));
}

lmhead_status lmhead_distill_logits_bwd(const void* logits, int type, int64_t ld,
                                        const int32_t* top_ids, const float* top_logits,
                                        const float* teacher_lse, const uint8_t* loss_mask,
                                        int64_t T, int32_t V, int32_t K, float temperature,
                                        float teacher_temperature, const float* grad_loss,
                                        const float* lse, void* d_logits, int64_t d_ld,
                                        lmhead_stream_t stream) {
  const lmhead_status rc = check_distill(logits, type, ld, top_ids, top_logits, T, V, K,
                                         temperature, teacher_temperature);
  if (rc != LMHEAD_OK) return rc;
  if (d_ld < V) return LMHEAD_ERR_INVALID_ARG;
  if (T == 0) return LMHEAD_OK;
  if (!grad_loss || !lse || !d_logits) return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(d_logits, type)) return LMHEAD_ERR_UNSUPPORTED;
  if (clash(logits, ld, d_logits, d_ld, T)) return LMHEAD_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DistillLogits a{};
  a.logits = logits;
  a.type = type;
  a.ld = ld;
  a.teacher = {top_ids, top_logits, teacher_lse, K, teacher_temperature};
  a.mask = loss_mask;
  a.T = T;
  a.V = V;
  a.tau = temperature;
  a.lse = const_cast<float*>(lse);   // read only in the backward
  a.grad = grad_loss;
  a.d_logits = d_logits;
  a.d_ld = d_ld;
  return status_of(traced_launch("distill_logits_bwd", s, [&] { return launch_distill_logits_bwd(a, s); }));
}

lmhead_status lmhead_process_logits_fwd(const void* logits, int type, int64_t ld, int64_t R,
                                        int32_t V, const int32_t* tokens, int64_t n_tokens,
                                        const int64_t* spans, const float* repetition,
                                        const float* frequency, const float* presence,
                                        const int64_t* bias_offsets, const int32_t* bias_ids,
                                        const float* bias_values, int64_t n_bias,
                                        const uint32_t* allowed, int64_t n_allowed,
                                        const int32_t* allowed_rows, void* out, int64_t out_ld,
                                        lmhead_stream_t stream) {
  const ProcessLogits a{logits, type, ld, R, V, tokens, n_tokens, spans, repetition, frequency,
                        presence, bias_offsets, bias_ids, bias_values, n_bias, allowed, n_allowed,
                        allowed_rows, nullptr, 0, out, out_ld};
  const lmhead_status rc = check_process(a);
  if (rc != LMHEAD_OK || R == 0) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return status_of(traced_launch("process_logits_fwd", s, [&] { return launch_process_logits(a, s); }));
}

lmhead_status lmhead_process_logits_bwd(const void* grad_out, int64_t grad_ld, const void* logits,
                                        int type, int64_t ld, int64_t R, int32_t V,
                                        const int32_t* tokens, int64_t n_tokens,
                                        const int64_t* spans, const float* repetition,
                                        const uint32_t* allowed, int64_t n_allowed,
                                        const int32_t* allowed_rows, void* d_logits, int64_t d_ld,
                                        lmhead_stream_t stream) {
  const ProcessLogits a{logits, type, ld, R, V, tokens, n_tokens, spans, repetition, nullptr,
                        nullptr, nullptr, nullptr, nullptr, 0, allowed, n_allowed, allowed_rows,
                        grad_out, grad_ld, d_logits, d_ld};
  const lmhead_status rc = check_process(a);
  if (rc != LMHEAD_OK) return rc;
  if (grad_ld < V) return LMHEAD_ERR_INVALID_ARG;
  if (R == 0) return LMHEAD_OK;
  if (!grad_out) return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(grad_out, type)) return LMHEAD_ERR_UNSUPPORTED;
  if (clash(grad_out, grad_ld, d_logits, d_ld, R)) return LMHEAD_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return status_of(traced_launch("process_logits_bwd", s, [&] { return launch_process_logits(a, s); }));
}

}  // extern "C"
