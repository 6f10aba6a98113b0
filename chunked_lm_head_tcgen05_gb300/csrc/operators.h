// Internal interface between the C ABI's argument checks (operators_api.cu,
// lmhead_api.cu) and the kernels of layer norm, distillation and logit
// processing.  Not part of the public C ABI.
#pragma once

#include "kernels.h"
#include "launch.h"

namespace lmh {

// Element types (same numbers as LMHEAD_F32 ... in lmhead.h).
constexpr int kF32 = 0;
constexpr int kBF16 = 1;
constexpr int kF16 = 2;

// ------------------------------------------------------------------ layer norm
// Most partial rows of the weight gradient's column sums (workspace bound).
constexpr int kNormPartials = 304;
// Rows wider than this may need their two sums (mean(h xh), mean(h)) beforehand.
constexpr int kNormWide = 4096;

struct NormFwd {
  const void* x;
  int x_type;
  int64_t x_ld;
  const void* weight;
  const void* bias;      // or NULL
  int param_type;
  int64_t N;
  int H;
  float eps;
  void* y;
  int y_type;            // x_type, or bf16 for fp32 rows
  int64_t y_ld;
  float* mean;           // or NULL
  float* rstd;           // or NULL
};

struct NormBwd {
  const void* dy;
  int dy_type;
  int64_t dy_ld;
  const void* x;
  int x_type;
  int64_t x_ld;
  const void* weight;
  int param_type;
  const float* mean;
  const float* rstd;
  int64_t N;
  int H;
  void* dx;              // x_type, or NULL
  int64_t dx_ld;
  float* d_weight;       // or NULL
  float* d_bias;         // or NULL
  int accumulate;
  float* partials;       // workspace: 2 * kNormPartials * H floats at most
  float2* sums;          // workspace [N], or NULL without one or at H <= kNormWide
};

cudaError_t launch_norm_fwd(const NormFwd& a, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormBwd& a, cudaStream_t s);

// ------------------------------------------------------------------ distillation
// The teacher's side of a call: K entries per token, row-major.
constexpr int kMaxTeacher = 1024;

struct Teacher {
  const int32_t* ids;    // [T, K]
  const float* logits;   // [T, K]; -inf marks an absent entry
  const float* lse;      // [T] or NULL (normalise over the K entries)
  int K;
  float tau;             // teacher's temperature
};

struct DistillLogits {
  const void* logits;    // [T, V], rows ld elements apart
  int type;
  int64_t ld;
  Teacher teacher;
  const uint8_t* mask;   // or NULL
  int64_t T;
  int V;
  float tau;
  float* loss;           // forward
  float* lse;            // forward: written; backward: read
  const float* grad;     // backward: cotangent of the loss
  void* d_logits;        // backward
  int64_t d_ld;
};

cudaError_t launch_distill_logits_fwd(const DistillLogits& a, cudaStream_t s);
cudaError_t launch_distill_logits_bwd(const DistillLogits& a, cudaStream_t s);

// Through the head.  The teacher's ids of each scored (compacted) row go to the
// GEMMs as ascending lists (RowIds: ids [T_alloc, K], start [T_alloc, tiles + 1]).
// Forward, before the GEMM: the lists, and the entry each id came from.
cudaError_t launch_distill_lists(const Teacher& teacher, int V, const int* idx, int T_alloc,
                                 const DeviceState* st, const RowIds& lists, int32_t* ids,
                                 uint16_t* start, uint16_t* order, cudaStream_t s);
// Forward, after it: loss, lse and z_top of the scored tokens from the vocabulary
// splits' statistics (as launch_fwd_merge reads them) and the picked accumulators.
cudaError_t launch_distill_loss(const Teacher& teacher, int V, float tau, const int* idx,
                                int T_alloc, DeviceState* st, const float4* partials, int n_splits,
                                int part_ld, const RowIds& lists, const uint16_t* order,
                                const float* picked, float* loss, float* lse, float* z_top,
                                cudaStream_t s);
// Unscored tokens' outputs.
cudaError_t launch_distill_zero(const uint8_t* mask, int T, int K, float* loss, float* lse,
                                float* z_top, cudaStream_t s);
// Backward: the epilogue's row coefficients (whose target term stays unused), the
// lists, and the cotangents that replace the dense ones at their ids.
cudaError_t launch_distill_prep(const Teacher& teacher, int V, float tau, const int* idx,
                                int T_alloc, const float* grad_loss, const float* lse,
                                const float* z_top, DeviceState* st, float4* coef,
                                const RowIds& lists, int32_t* ids, uint16_t* start, float* values,
                                cudaStream_t s);
// Writes those cotangents into a stored dz block: rows [t0, t0 + rows_cap) of the
// compacted order, vocabulary rows [v0, v0 + cols).
cudaError_t launch_distill_patch(const int32_t* ids, const float* values, int K,
                                 const DeviceState* st, int t0, int rows_cap, int v0, int cols,
                                 uint16_t* dz, int64_t dz_ld, cudaStream_t s);

// ------------------------------------------------------------------ logit processing
struct ProcessLogits {
  const void* logits;    // [R, V]
  int type;
  int64_t ld;
  int64_t R;
  int V;
  const int32_t* tokens; // [n_tokens] or NULL
  int64_t n_tokens;
  const int64_t* spans;  // [R, 3] prompt begin, output begin, output end
  const float* repetition;   // [R] or NULL, as the next two
  const float* frequency;
  const float* presence;
  const int64_t* bias_offsets;   // [R + 1] or NULL
  const int32_t* bias_ids;
  const float* bias_values;
  int64_t n_bias;
  const uint32_t* allowed;   // [M, (V + 31) / 32] or NULL
  int64_t M;
  const int32_t* allowed_rows;   // [R] or NULL (row r)
  const void* grad;      // backward: cotangent of the result, else NULL
  int64_t grad_ld;
  void* out;             // forward: processed logits; backward: d_logits
  int64_t out_ld;
};

cudaError_t launch_process_logits(const ProcessLogits& a, cudaStream_t s);

}  // namespace lmh
