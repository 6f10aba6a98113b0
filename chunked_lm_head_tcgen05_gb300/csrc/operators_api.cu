// Host side of the C ABI of layer norm, distillation on held logits, logit
// processing, embedding, low-rank adapters and beam search: argument checks and the stream-ordered launches.  No device
// memory is allocated and nothing synchronises.
#include "lmhead.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <numeric>

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

// An operand: `rows` rows of `width` bytes, ld bytes apart, from `from` to `to`; empty where
// there is none of it.
struct Rows {
  uintptr_t from, to;
  int64_t rows, ld, width;
};
Rows matrix(const void* p, int type, int64_t rows, int64_t ld, int64_t cols) {
  const int64_t size = static_cast<int64_t>(element_bytes(type)), width = cols * size;
  const uintptr_t from = reinterpret_cast<uintptr_t>(p);
  if (!p || rows <= 0 || width <= 0) return Rows{from, from, 0, 0, 0};
  int64_t stride, last;      // a stride may be anything
  if (__builtin_mul_overflow(ld, size, &stride)) stride = INT64_MAX;
  if (__builtin_mul_overflow(rows - 1, stride, &last)) last = INT64_MAX;
  uintptr_t to;
  if (__builtin_add_overflow(from, static_cast<uintptr_t>(last) + static_cast<uintptr_t>(width), &to)) to = UINTPTR_MAX;
  return Rows{from, to, rows, stride, width};
}
Rows block(const void* p, size_t bytes) {
  const uintptr_t from = reinterpret_cast<uintptr_t>(p);
  return Rows{from, p ? from + bytes : from, 1, 0, static_cast<int64_t>(bytes)};
}

// Whether two operands share a byte.  Columns of one tensor beside each other do not: their
// rows' starts keep their distance, modulo the strides' common divisor, outside both widths.
// (Strides that differ may be found to share where they only might.)
bool share(const Rows& a, const Rows& b) {
  if (a.from >= b.to || b.from >= a.to || a.from == a.to || b.from == b.to) return false;
  const int64_t step = std::gcd(a.rows > 1 ? a.ld : 0, b.rows > 1 ? b.ld : 0);
  if (step == 0) return true;      // a row each
  int64_t d = b.from >= a.from ? static_cast<int64_t>((b.from - a.from) % static_cast<uintptr_t>(step))
                               : -static_cast<int64_t>((a.from - b.from) % static_cast<uintptr_t>(step));
  if (d < 0) d += step;
  return d < a.width || d > step - b.width;
}

// Whether what a call writes shares no byte with what it reads, nor with another of its results.
bool disjoint(std::initializer_list<Rows> written, std::initializer_list<Rows> read) {
  for (const Rows* w = written.begin(); w != written.end(); ++w) {
    for (const Rows* other = written.begin(); other != w; ++other)
      if (share(*w, *other)) return false;
    for (const Rows& r : read)
      if (share(*w, r)) return false;
  }
  return true;
}

// Arguments that both directions of the embedding share; `in` and `out` are its matrices.
lmhead_status check_embedding(int64_t N, int32_t V, int32_t H, float scale, int in_type, int64_t in_ld,
                              int out_type, int64_t out_ld) {
  if (N < 0 || V <= 0 || H <= 0 || !known_type(in_type) || !known_type(out_type) || in_ld < H || out_ld < H ||
      !std::isfinite(scale))
    return LMHEAD_ERR_INVALID_ARG;
  if (N >= kMaxRows || V > kMaxVocab || H > kMaxWidth) return LMHEAD_ERR_UNSUPPORTED;
  return LMHEAD_OK;
}

// Sizes, types and operands that both directions of the adapters share.
lmhead_status check_adapters(const Adapters& a, int type, int64_t ld) {
  if (a.T < 0 || a.H <= 0 || a.V <= 0 || a.rank <= 0 || a.n <= 0 || !known_type(type) || ld < a.V || a.x_ld < a.H)
    return LMHEAD_ERR_INVALID_ARG;
  if (a.T >= kMaxRows || a.H > kMaxVocab || a.V > kMaxVocab || a.rank > kMaxRank || a.n > kMaxAdapters ||
      !adapters_fit(a.T, a.H > a.V ? a.H : a.V, a.n))
    return LMHEAD_ERR_UNSUPPORTED;
  return LMHEAD_OK;
}

lmhead_status check_adapter_operands(const Adapters& a, size_t workspace_bytes, size_t needed) {
  if (!a.x || !a.down || !a.up || !a.workspace) return LMHEAD_ERR_INVALID_ARG;
  for (const void* p : {a.x, a.down, a.up})
    if (!aligned_to(p, kBF16)) return LMHEAD_ERR_UNSUPPORTED;
  if (!aligned_to(a.ids, kF32) || !aligned_to(a.scale, kF32) || (reinterpret_cast<uintptr_t>(a.workspace) & 255))
    return LMHEAD_ERR_UNSUPPORTED;
  return workspace_bytes < needed ? LMHEAD_ERR_WORKSPACE_TOO_SMALL : LMHEAD_OK;
}

// Whether the workspace and the results (NULL: not asked for) lie apart from each other and from
// what a call reads: `own`, and what both directions do.
bool adapters_disjoint(const Adapters& a, size_t needed, const Rows& own, const Rows& first, const Rows& second,
                       const Rows& third) {
  const int64_t factor_rows = int64_t{a.n} * a.rank;
  return disjoint({first, second, third, block(a.workspace, needed)},
                  {own, matrix(a.x, kBF16, a.T, a.x_ld, a.H), matrix(a.down, kBF16, factor_rows, a.H, a.H),
                   matrix(a.up, kBF16, factor_rows, a.V, a.V), matrix(a.ids, kF32, 1, 0, a.T),
                   matrix(a.scale, kF32, 1, 0, a.n)});
}

constexpr int32_t kMaxBeamVocab = 1 << 30;   // columns of the pieces past a row's end are counted too

// A strided block of bytes: up to three dimensions of `inner` contiguous bytes.
struct Block {
  int64_t size[3], stride[3], inner;
};

// The bytes from its first to its last, or -1 where that cannot be: sizes are small
// enough for memory, strides may be anything.
int64_t extent_of(const Block& b) {
  double end = static_cast<double>(b.inner);
  for (int i = 0; i < 3; ++i)
    if (b.size[i] > 1) end += static_cast<double>(b.size[i] - 1) * static_cast<double>(b.stride[i]);
  if (end > 9.0e18) return -1;
  int64_t n = b.inner;
  for (int i = 0; i < 3; ++i)
    if (b.size[i] > 1) n += (b.size[i] - 1) * b.stride[i];
  return n;
}

// Whether no two elements share a byte, judged from the strides in ascending order.
bool apart(Block b) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int x, int y) { return b.stride[x] < b.stride[y]; });
  int64_t within = b.inner;
  for (const int i : order) {
    if (b.size[i] <= 1) continue;
    if (b.stride[i] < within) return false;
    within += (b.size[i] - 1) * b.stride[i];
  }
  return true;
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

size_t lmhead_embedding_workspace_size(int64_t N, int32_t H) {
  return N < 0 || N >= kMaxRows || H <= 0 || H > kMaxWidth ? 0 : embed_workspace(N, H);
}

lmhead_status lmhead_embedding_fwd(const int32_t* ids, int64_t N, const void* weight, int type,
                                   int64_t w_ld, int32_t V, int32_t H, float scale, void* y,
                                   int y_type, int64_t y_ld, lmhead_stream_t stream) {
  const lmhead_status rc = check_embedding(N, V, H, scale, type, w_ld, y_type, y_ld);
  if (rc != LMHEAD_OK) return rc;
  if (y_type != type && !(type == kF32 && y_type == kBF16) && y_type != kF32) return LMHEAD_ERR_UNSUPPORTED;
  if (N == 0) return LMHEAD_OK;
  if (!ids || !weight || !y) return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(weight, type) || !aligned_to(y, y_type) || !aligned_to(ids, kF32)) return LMHEAD_ERR_UNSUPPORTED;
  if (!disjoint({matrix(y, y_type, N, y_ld, H)}, {matrix(weight, type, V, w_ld, H), matrix(ids, kF32, 1, 0, N)}))
    return LMHEAD_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const EmbedFwd a{ids, N, weight, type, w_ld, V, H, scale, y, y_type, y_ld};
  return status_of(traced_launch("embedding_fwd", s, [&] { return launch_embed_fwd(a, s); }));
}

lmhead_status lmhead_embedding_bwd(const void* dy, int dy_type, int64_t dy_ld, const int32_t* ids,
                                   int64_t N, int32_t V, int32_t H, float scale,
                                   int32_t padding_id, void* d_weight, int d_weight_type,
                                   int accumulate, void* workspace, size_t workspace_bytes,
                                   lmhead_stream_t stream) {
  const lmhead_status rc = check_embedding(N, V, H, scale, dy_type, dy_ld, d_weight_type, H);
  if (rc != LMHEAD_OK) return rc;
  int skip = -1;
  if (padding_id != LMHEAD_NO_PADDING) {
    if (padding_id < -V || padding_id >= V) return LMHEAD_ERR_INVALID_ARG;
    skip = padding_id < 0 ? padding_id + V : padding_id;
  }
  if (d_weight_type != kF32 && (d_weight_type != kBF16 || accumulate || N > kSortMost))
    return LMHEAD_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0 && accumulate) return LMHEAD_OK;
  if (!d_weight) return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(d_weight, d_weight_type)) return LMHEAD_ERR_UNSUPPORTED;
  if (N == 0) {
    const size_t bytes = element_bytes(d_weight_type) * static_cast<size_t>(V) * static_cast<size_t>(H);
    return status_of(cudaMemsetAsync(d_weight, 0, bytes, s));
  }
  if (!dy || !ids || !workspace) return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(dy, dy_type) || !aligned_to(ids, kF32) || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return LMHEAD_ERR_UNSUPPORTED;
  const size_t needed = embed_workspace(N, H);
  if (workspace_bytes < needed) return LMHEAD_ERR_WORKSPACE_TOO_SMALL;
  if (!disjoint({matrix(d_weight, d_weight_type, V, H, H), block(workspace, needed)},
             {matrix(dy, dy_type, N, dy_ld, H), matrix(ids, kF32, 1, 0, N)}))
    return LMHEAD_ERR_INVALID_ARG;
  const EmbedBwd a{dy, dy_type, dy_ld, ids, N, V, H, scale, skip, d_weight, d_weight_type,
                   accumulate ? 1 : 0, workspace};
  return status_of(launch_embed_bwd(a, s));
}

size_t lmhead_adapters_workspace_size(int64_t T, int32_t H, int32_t V, int32_t rank, int32_t n_adapters) {
  const Adapters a{nullptr, H, nullptr, nullptr, nullptr, nullptr, T, H, V, rank, n_adapters, nullptr};
  return check_adapters(a, kF32, V) == LMHEAD_OK ? adapters_workspace(T, H, V, rank, n_adapters) : 0;
}

lmhead_status lmhead_adapters_fwd(const void* base, int type, int64_t base_ld, const uint16_t* x,
                                  int64_t x_ld, const uint16_t* down, const uint16_t* up,
                                  const int32_t* adapter_ids, const float* scale, int64_t T,
                                  int32_t H, int32_t V, int32_t rank, int32_t n_adapters,
                                  void* out, int64_t out_ld, void* workspace,
                                  size_t workspace_bytes, lmhead_stream_t stream) {
  const Adapters a{x, x_ld, down, up, adapter_ids, scale, T, H, V, rank, n_adapters, workspace};
  lmhead_status rc = check_adapters(a, type, base_ld);
  if (rc != LMHEAD_OK) return rc;
  if (out_ld < V) return LMHEAD_ERR_INVALID_ARG;
  if (T == 0) return LMHEAD_OK;
  if (!base || !out) return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(base, type) || !aligned_to(out, type)) return LMHEAD_ERR_UNSUPPORTED;
  if (clash(base, base_ld, out, out_ld, T)) return LMHEAD_ERR_INVALID_ARG;
  const size_t needed = adapters_workspace(T, H, V, rank, n_adapters);
  rc = check_adapter_operands(a, workspace_bytes, needed);
  if (rc != LMHEAD_OK) return rc;
  const Rows none = block(nullptr, 0);
  if (!adapters_disjoint(a, needed, base == out ? none : matrix(base, type, T, base_ld, V),
                         matrix(out, type, T, out_ld, V), none, none))
    return LMHEAD_ERR_INVALID_ARG;
  const AdaptersFwd f{a, base, type, base_ld, out, out_ld};
  return status_of(launch_adapters_fwd(f, reinterpret_cast<cudaStream_t>(stream)));
}

lmhead_status lmhead_adapters_bwd(const void* grad_out, int type, int64_t grad_ld,
                                  const uint16_t* x, int64_t x_ld, const uint16_t* down,
                                  const uint16_t* up, const int32_t* adapter_ids,
                                  const float* scale, int64_t T, int32_t H, int32_t V,
                                  int32_t rank, int32_t n_adapters, float* dx, int64_t dx_ld,
                                  int accumulate_dx, float* d_down, float* d_up, int accumulate,
                                  void* workspace, size_t workspace_bytes,
                                  lmhead_stream_t stream) {
  const Adapters a{x, x_ld, down, up, adapter_ids, scale, T, H, V, rank, n_adapters, workspace};
  lmhead_status rc = check_adapters(a, type, grad_ld);
  if (rc != LMHEAD_OK) return rc;
  if (dx && dx_ld < H) return LMHEAD_ERR_INVALID_ARG;
  for (const float* p : {dx, d_down, d_up})
    if (!aligned_to(p, kF32)) return LMHEAD_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    const size_t factor = sizeof(float) * static_cast<size_t>(n_adapters) * static_cast<size_t>(rank);
    if (d_down && !accumulate && cudaMemsetAsync(d_down, 0, factor * static_cast<size_t>(H), s) != cudaSuccess)
      return LMHEAD_ERR_CUDA;
    if (d_up && !accumulate && cudaMemsetAsync(d_up, 0, factor * static_cast<size_t>(V), s) != cudaSuccess)
      return LMHEAD_ERR_CUDA;
    return LMHEAD_OK;
  }
  if (!grad_out || (!dx && !d_down && !d_up)) return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(grad_out, type)) return LMHEAD_ERR_UNSUPPORTED;
  const size_t needed = adapters_workspace(T, H, V, rank, n_adapters);
  rc = check_adapter_operands(a, workspace_bytes, needed);
  if (rc != LMHEAD_OK) return rc;
  const int64_t factor_rows = int64_t{n_adapters} * rank;
  if (!adapters_disjoint(a, needed, matrix(grad_out, type, T, grad_ld, V), matrix(dx, kF32, T, dx_ld, H),
                         matrix(d_down, kF32, factor_rows, H, H), matrix(d_up, kF32, factor_rows, V, V)))
    return LMHEAD_ERR_INVALID_ARG;
  const AdaptersBwd b{a, grad_out, type, grad_ld, dx, dx_ld, accumulate_dx ? 1 : 0, d_down, d_up, accumulate ? 1 : 0};
  return status_of(launch_adapters_bwd(b, s));
}

size_t lmhead_beam_workspace_size(int64_t R, int32_t V, int32_t take) {
  return R < 0 || R >= kMaxRows || V <= 0 || V > kMaxBeamVocab || take <= 0 || take > kMaxTake
             ? 0 : beam_workspace(R, V, take);
}

lmhead_status lmhead_beam_select(const void* logits, int type, int64_t ld, int64_t R, int32_t V,
                                 int32_t beams, int32_t take, const float* scores,
                                 const uint8_t* finished, int32_t eos_id, float temperature,
                                 float* out_scores, int32_t* parents, int32_t* tokens,
                                 uint8_t* next_finished, float* lse, void* workspace,
                                 size_t workspace_bytes, lmhead_stream_t stream) {
  if (R < 0 || V <= 0 || beams <= 0 || take <= 0 || !known_type(type) || ld < V || !positive(temperature) ||
      R % beams != 0 || eos_id < -1 || eos_id >= V || (finished && eos_id < 0))
    return LMHEAD_ERR_INVALID_ARG;
  if (R >= kMaxRows || V > kMaxBeamVocab || beams > kMaxBeams || take > kMaxTake) return LMHEAD_ERR_UNSUPPORTED;
  if (R == 0) return LMHEAD_OK;
  if (!logits || !scores || !out_scores || !parents || !tokens || !workspace) return LMHEAD_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(scores), static_cast<const void*>(out_scores),
                        static_cast<const void*>(parents), static_cast<const void*>(tokens),
                        static_cast<const void*>(lse)})
    if (!aligned_to(p, kF32)) return LMHEAD_ERR_UNSUPPORTED;
  if (!aligned_to(logits, type) || (reinterpret_cast<uintptr_t>(workspace) & 255)) return LMHEAD_ERR_UNSUPPORTED;
  // one group's results may lie over its own inputs, which it has read by then, not over another's
  const size_t rows = static_cast<size_t>(R), results = rows / beams * take;
  const bool own = take == beams;
  const Rows old_scores = block(own && scores == out_scores ? nullptr : scores, 4 * rows),
             old_finished = block(own && finished == next_finished ? nullptr : finished, rows),
             new_scores = block(out_scores, 4 * results), new_finished = block(next_finished, results);
  if (!disjoint({new_scores}, {old_scores}) || !disjoint({new_finished}, {old_finished})) return LMHEAD_ERR_INVALID_ARG;
  const size_t needed = beam_workspace(R, V, take);
  if (workspace_bytes < needed) return LMHEAD_ERR_WORKSPACE_TOO_SMALL;
  if (!disjoint({new_scores, new_finished, block(parents, 4 * results), block(tokens, 4 * results), block(lse, 4 * rows),
                 block(workspace, needed)},
                {matrix(logits, type, R, ld, V), old_scores, old_finished}))
    return LMHEAD_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const BeamSelect a{logits, type, ld, R, V, beams, take, scores, finished, eos_id, temperature,
                     out_scores, parents, tokens, next_finished, lse, workspace};
  return status_of(launch_beam_select(a, s));
}

lmhead_status lmhead_beam_reorder(const void* src, int64_t src_outer, int64_t src_row,
                                  int64_t src_mid, int64_t src_rows, void* dst,
                                  int64_t dst_outer, int64_t dst_row, int64_t dst_mid,
                                  const int32_t* parents, int64_t rows, int32_t beams,
                                  int64_t outer, int64_t mid, int64_t inner_bytes,
                                  int clear_missing, lmhead_stream_t stream) {
  if (rows < 0 || src_rows < 0 || outer < 0 || mid < 0 || inner_bytes < 0) return LMHEAD_ERR_INVALID_ARG;
  if (rows >= kMaxRows || src_rows >= kMaxRows) return LMHEAD_ERR_UNSUPPORTED;
  if (rows == 0 || outer == 0 || mid == 0 || inner_bytes == 0) return LMHEAD_OK;
  if ((!src && src_rows > 0) || !dst || !parents) return LMHEAD_ERR_INVALID_ARG;   // no rows may have no address
  // strides of dimensions of size 1 say nothing
  if (outer == 1) src_outer = dst_outer = 0;
  if (mid == 1) src_mid = dst_mid = 0;
  if (rows == 1) dst_row = 0;
  if (src_rows <= 1) src_row = 0;
  if (src_outer < 0 || src_row < 0 || src_mid < 0 || dst_outer < 0 || dst_row < 0 || dst_mid < 0)
    return LMHEAD_ERR_INVALID_ARG;
  const Block from{{outer, src_rows, mid}, {src_outer, src_row, src_mid}, inner_bytes};
  const Block to{{outer, rows, mid}, {dst_outer, dst_row, dst_mid}, inner_bytes};
  const int64_t from_bytes = extent_of(from), to_bytes = extent_of(to);
  if (from_bytes < 0 || to_bytes < 0 || !apart(to)) return LMHEAD_ERR_INVALID_ARG;
  if (src == dst) {
    if (src_rows != rows || src_outer != dst_outer || src_row != dst_row || src_mid != dst_mid || beams <= 0 ||
        rows % beams != 0)
      return LMHEAD_ERR_INVALID_ARG;
    if (beams > kMaxBeams) return LMHEAD_ERR_UNSUPPORTED;
  } else {
    const uintptr_t p = reinterpret_cast<uintptr_t>(src), q = reinterpret_cast<uintptr_t>(dst);
    if (src_rows > 0 && p < q + static_cast<uintptr_t>(to_bytes) && q < p + static_cast<uintptr_t>(from_bytes))
      return LMHEAD_ERR_INVALID_ARG;
  }
  if (!disjoint({block(dst, static_cast<size_t>(to_bytes))}, {block(parents, 4 * static_cast<size_t>(rows))}))
    return LMHEAD_ERR_INVALID_ARG;
  if (!aligned_to(parents, kF32)) return LMHEAD_ERR_UNSUPPORTED;
  const BeamReorder a{static_cast<const char*>(src), static_cast<char*>(dst), parents, rows, src_rows, beams,
                      outer, mid, inner_bytes, src_outer, src_row, src_mid, dst_outer, dst_row, dst_mid,
                      clear_missing};
  if (!beam_reorder_fits(a)) return LMHEAD_ERR_UNSUPPORTED;
  return status_of(launch_beam_reorder(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
