// Distillation from a teacher's top logits.  Token t has K teacher entries
// (id_k, a_k); with the teacher's log-sum-exp L (given, or over the K entries),
//   p_k = exp(a_k / tau' - L),   P = sum_k p_k,
//   loss = sum_k p_k (log p_k - z_{id_k} + lse(z)),    z = logits / tau,
//   d loss / d logits_v = (g / tau) (P softmax(z)_v - sum_{k: id_k = v} p_k).
// So the gradient is dense only through softmax(z): one coefficient per row,
// and K places where something is subtracted.  An entry with a_k = -inf is
// absent (its id is not looked at); a token whose entries are all absent has
// loss 0 and no gradient; entries that repeat an id add up.
#include "element.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace lmh {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBwdCols = 16384;   // columns per CTA in the backward

// Row of the student's table that an entry names: negative ids wrap; -1 for
// an id outside [-V, V).
__device__ __forceinline__ int wrap_id(int id, int V) {
  if (id < 0) id += V;
  return (id >= 0 && id < V) ? id : -1;
}

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) t += red[w];
  return t;
}

__device__ __forceinline__ float block_max(float v, float* red) {
  v = warp_max(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) t = fmaxf(t, red[w]);
  return t;
}

// The teacher's distribution of one token, for the whole CTA: p[k] and the
// log-probability logp[k] in shared memory (0 and -inf where the entry is
// absent); returns P.  NaN entries make P NaN.
__device__ float teacher_row(const Teacher& te, int64_t t, float* p, float* logp, float* red) {
  const float* a = te.logits + t * te.K;
  // L = base + rest, kept apart so that a distant maximum does not cancel
  float base, rest = 0.f;
  if (te.lse) {
    base = te.lse[t];
  } else {
    float m = -INFINITY;
    for (int k = threadIdx.x; k < te.K; k += kThreads) m = fmaxf(m, a[k] / te.tau);
    m = block_max(m, red);
    float s = 0.f;
    base = m == -INFINITY ? 0.f : m;
    for (int k = threadIdx.x; k < te.K; k += kThreads) s += expf(a[k] / te.tau - base);
    rest = logf(block_sum(s, red));
  }
  float P = 0.f;
  for (int k = threadIdx.x; k < te.K; k += kThreads) {
    const bool absent = a[k] == -INFINITY;   // L is -inf where every entry is
    const float lp = absent ? -INFINITY : (a[k] / te.tau - base) - rest;
    const float q = absent ? 0.f : expf(lp);
    logp[k] = lp;
    p[k] = q;
    P += q;
  }
  return block_sum(P, red);
}

// One entry's part of the loss, relative to the row's maximum: p (log p - (z - m)).
// p = 0 adds nothing, whatever z is; a NaN z (an invalid id) always shows.
__device__ __forceinline__ float loss_term(float p, float logp, float z_rel) {
  return p == 0.f && z_rel == z_rel ? 0.f : p * (logp - z_rel);
}

// One CTA per row.
template <typename T>
__global__ void __launch_bounds__(kThreads) logits_fwd_kernel(DistillLogits a) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float red[kWarps], red_m[kWarps];
  __shared__ float p[kMaxTeacher], logp[kMaxTeacher];
  const float c = kLog2e / a.tau;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    if (a.mask && !a.mask[t]) {
      if (threadIdx.x == 0) {
        a.loss[t] = 0.f;
        a.lse[t] = 0.f;
      }
      continue;
    }
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    const float P = teacher_row(a.teacher, t, p, logp, red);
    // running maximum m (of the unscaled logits) and s = sum 2^((x - m) c)
    float m = -INFINITY, s = 0.f;
    for (int i = threadIdx.x; i < a.V; i += kThreads) {
      const float x = to_f32(row[i]);
      const float mn = fmaxf(m, x);
      const float base = mn == -INFINITY ? 0.f : mn;
      s = s * ex2_approx((m - base) * c) + ex2_approx((x - base) * c);
      m = mn;
    }
    const float M = block_max(m, red_m);
    const float base = M == -INFINITY ? 0.f : M;
    const float S = block_sum(s * ex2_approx((m - base) * c), red);
    // loss relative to the maximum, so that large logits do not cancel
    const float mz = M / a.tau, ln_s = logf(S);
    float term = 0.f;
    for (int k = threadIdx.x; k < a.teacher.K; k += kThreads) {
      if (logp[k] == -INFINITY) continue;
      const int v = wrap_id(a.teacher.ids[t * a.teacher.K + k], a.V);
      term += loss_term(p[k], logp[k], v < 0 ? __int_as_float(0x7fc00000)
                                             : (to_f32(row[v]) - M) / a.tau);
    }
    const float A = block_sum(term, red);
    if (threadIdx.x == 0) {
      a.lse[t] = mz + ln_s;
      a.loss[t] = P == 0.f ? 0.f : fmaf(P, ln_s, A);
    }
    __syncthreads();
  }
}

// g (P q_v - taken) / tau for one logit; non-finite logits get zero.
__device__ __forceinline__ float cotangent(float x, float inv_tau, float lse, float gP,
                                           float taken) {
  if (!isfinite(x)) return 0.f;
  const float q = ex2_approx(fmaf(x, inv_tau, -lse) * kLog2e);
  return fmaf(gP, q, -taken);
}

// CTA (row, column range).  The K places of the range are computed from the
// logits before the dense pass (d_logits may be the logits buffer) and
// written after it.
template <typename T>
__global__ void __launch_bounds__(kThreads) logits_bwd_kernel(DistillLogits a, int parts) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float red[kWarps];
  __shared__ float p[kMaxTeacher], logp[kMaxTeacher];
  __shared__ int id[kMaxTeacher];
  const int K = a.teacher.K;
  const float inv_tau = 1.f / a.tau;
  for (int64_t w = blockIdx.x; w < a.T * parts; w += gridDim.x) {
    const int64_t t = w / parts;
    const int c0 = static_cast<int>(w - t * parts) * kBwdCols;
    const int c1 = min(a.V, c0 + kBwdCols);
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    T* out = static_cast<T*>(a.d_logits) + t * a.d_ld;
    const bool scored = !a.mask || a.mask[t];
    const float P = scored ? teacher_row(a.teacher, t, p, logp, red) : 0.f;
    if (P == 0.f) {
      for (int i = c0 + threadIdx.x; i < c1; i += kThreads) out[i] = from_f32<T>(0.f);
      __syncthreads();
      continue;
    }
    for (int k = threadIdx.x; k < K; k += kThreads)
      id[k] = logp[k] == -INFINITY ? -1 : wrap_id(a.teacher.ids[t * K + k], a.V);
    __syncthreads();
    const float g = a.grad[t] * inv_tau, lse = a.lse[t], gP = g * P;
    float fixed[kMaxTeacher / kThreads];
#pragma unroll
    for (int j = 0; j < kMaxTeacher / kThreads; ++j) {
      const int k = threadIdx.x + j * kThreads;
      fixed[j] = 0.f;
      if (k < K && id[k] >= c0 && id[k] < c1) {
        float taken = 0.f;   // repeated ids add up; each writes the same value
        for (int i = 0; i < K; ++i) taken += id[i] == id[k] ? p[i] : 0.f;
        fixed[j] = cotangent(to_f32(row[id[k]]), inv_tau, lse, gP, g * taken);
      }
    }
    __syncthreads();
    for (int i = c0 + threadIdx.x; i < c1; i += kThreads)
      out[i] = from_f32<T>(cotangent(to_f32(row[i]), inv_tau, lse, gP, 0.f));
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMaxTeacher / kThreads; ++j) {
      const int k = threadIdx.x + j * kThreads;
      if (k < K && id[k] >= c0 && id[k] < c1) out[id[k]] = from_f32<T>(fixed[j]);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ through the head
// One CTA per token: z_k = hidden . weight[id_k] / tau for the K entries (one
// warp per entry), then the loss with the statistics of the whole vocabulary.
// The loss takes z_k - max in the statistics' own units, u = (h . w) scale
// with the scale the GEMM used: the rounding of log2(e) / tau then cancels
// (loss error against 64 bits 1.3e-6 with z_k = (h . w) / tau there instead).
__global__ void __launch_bounds__(kThreads)
    head_loss_kernel(const uint16_t* __restrict__ hidden, const uint16_t* __restrict__ weight,
                     int H, int V, Teacher te, const uint8_t* __restrict__ mask, int T, float tau,
                     const float4* __restrict__ stats, DeviceState* st, float* loss, float* lse,
                     float* z_top) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float red[kWarps];
  __shared__ float p[kMaxTeacher], logp[kMaxTeacher], z[kMaxTeacher];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int K = te.K;
  const float scale = kLog2e / tau;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    float* zt = z_top + static_cast<int64_t>(t) * K;
    if (mask && !mask[t]) {
      for (int k = threadIdx.x; k < K; k += kThreads) zt[k] = 0.f;
      if (threadIdx.x == 0) {
        loss[t] = 0.f;
        lse[t] = 0.f;
      }
      continue;
    }
    const float P = teacher_row(te, t, p, logp, red);
    const uint4* h = reinterpret_cast<const uint4*>(hidden + static_cast<int64_t>(t) * H);
    bool bad = false;
    for (int k = warp; k < K; k += kWarps) {
      const bool absent = logp[k] == -INFINITY;
      const int v = absent ? -1 : wrap_id(te.ids[static_cast<int64_t>(t) * K + k], V);
      float acc = 0.f;
      if (v >= 0) {
        const uint4* wr = reinterpret_cast<const uint4*>(weight + static_cast<int64_t>(v) * H);
        for (int i = lane; i < H / 8; i += 32) {
          const Pack<__nv_bfloat16, 8> x = *reinterpret_cast<const Pack<__nv_bfloat16, 8>*>(h + i);
          const Pack<__nv_bfloat16, 8> y = *reinterpret_cast<const Pack<__nv_bfloat16, 8>*>(wr + i);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc = fmaf(to_f32(x.v[j]), to_f32(y.v[j]), acc);
        }
      } else if (!absent) {
        bad = true;
      }
      acc = warp_sum(acc);
      if (lane == 0) {
        const float none = absent ? 0.f : __int_as_float(0x7fc00000);
        z[k] = v >= 0 ? acc * scale : none;
        zt[k] = v >= 0 ? acc / tau : none;
      }
    }
    if (bad && lane == 0) atomicCAS(&st->status, 0, STATUS_BAD_TARGET);
    __syncthreads();
    const float4 q = stats[t];
    const float ln_s = logf(q.y);
    float term = 0.f;
    for (int k = threadIdx.x; k < K; k += kThreads)
      term += loss_term(p[k], logp[k], (z[k] - q.x) * kLn2);
    const float A = block_sum(term, red);
    if (threadIdx.x == 0) {
      lse[t] = fmaf(q.x, kLn2, ln_s);
      loss[t] = P == 0.f ? 0.f : fmaf(P, ln_s, A);
    }
    __syncthreads();
  }
}

// One CTA per compacted row.
__global__ void __launch_bounds__(kThreads)
    distill_prep_kernel(Teacher te, int V, float tau, const int* __restrict__ idx, int T_alloc,
                        const float* __restrict__ grad_loss, const float* __restrict__ lse,
                        const float* __restrict__ z_top, DeviceState* st, float4* coef,
                        int32_t* patch_ids, uint16_t* patch_values) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float red[kWarps];
  __shared__ float p[kMaxTeacher], logp[kMaxTeacher];
  __shared__ int id[kMaxTeacher];
  const int K = te.K;
  const int rows = st->rows;
  for (int r = blockIdx.x; r < T_alloc; r += gridDim.x) {
    if (r >= rows) {
      if (threadIdx.x == 0) coef[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      continue;
    }
    const int t = idx ? idx[r] : r;
    const float P = teacher_row(te, t, p, logp, red);
    bool bad = false;
    for (int k = threadIdx.x; k < K; k += kThreads) {
      const bool absent = logp[k] == -INFINITY;
      id[k] = absent ? -1 : wrap_id(te.ids[static_cast<int64_t>(t) * K + k], V);
      bad |= id[k] < 0 && !absent;
    }
    if (bad) atomicCAS(&st->status, 0, STATUS_BAD_TARGET);
    __syncthreads();
    const float g = grad_loss[t] / tau, L = lse[t];
    const float gP = P == 0.f ? 0.f : g * P;
    if (threadIdx.x == 0) coef[r] = make_float4(L * kLog2e, 0.f, -gP, 0.f);
    for (int k = threadIdx.x; k < K; k += kThreads) {
      const int64_t at = static_cast<int64_t>(r) * K + k;
      patch_ids[at] = id[k];
      if (id[k] < 0) continue;
      float taken = 0.f;
      for (int i = 0; i < K; ++i) taken += id[i] == id[k] ? p[i] : 0.f;
      const float q = ex2_approx((z_top[static_cast<int64_t>(t) * K + k] - L) * kLog2e);
      const __nv_bfloat16 v = __float2bfloat16_rn(fmaf(gP, q, -g * taken));
      patch_values[at] = __bfloat16_as_ushort(v);
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kThreads)
    distill_patch_kernel(const int32_t* __restrict__ patch_ids,
                         const uint16_t* __restrict__ patch_values, int K, const DeviceState* st,
                         int t0, int rows_cap, int v0, int cols, uint16_t* dz, int64_t dz_ld) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int rows = min(st->rows - t0, rows_cap);
  const int64_t n = rows > 0 ? static_cast<int64_t>(rows) * K : 0;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t at = static_cast<int64_t>(t0) * K + i;
    const int v = patch_ids[at];
    if (v < v0 || v - v0 >= cols) continue;
    dz[(i / K) * dz_ld + (v - v0)] = patch_values[at];
  }
}

template <typename T>
cudaError_t logits_fwd(const DistillLogits& a, cudaStream_t s) {
  const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
  return launch_dependent(logits_fwd_kernel<T>, dim3(static_cast<int>(a.T < cap ? a.T : cap)),
                          kThreads, 0, 1, s, a);
}

template <typename T>
cudaError_t logits_bwd(const DistillLogits& a, cudaStream_t s) {
  const int parts = (a.V + kBwdCols - 1) / kBwdCols;
  const int64_t cap = static_cast<int64_t>(sm_count()) * 16, items = a.T * parts;
  return launch_dependent(logits_bwd_kernel<T>, dim3(static_cast<int>(items < cap ? items : cap)),
                          kThreads, 0, 1, s, a, parts);
}

}  // namespace

cudaError_t launch_distill_logits_fwd(const DistillLogits& a, cudaStream_t s) {
  if (a.type == kF32) return logits_fwd<float>(a, s);
  if (a.type == kBF16) return logits_fwd<__nv_bfloat16>(a, s);
  return logits_fwd<__half>(a, s);
}

cudaError_t launch_distill_logits_bwd(const DistillLogits& a, cudaStream_t s) {
  if (a.type == kF32) return logits_bwd<float>(a, s);
  if (a.type == kBF16) return logits_bwd<__nv_bfloat16>(a, s);
  return logits_bwd<__half>(a, s);
}

cudaError_t launch_distill_head_loss(const uint16_t* hidden, const uint16_t* weight, int H, int V,
                                     const Teacher& teacher, const uint8_t* mask, int T, float tau,
                                     const float4* stats, DeviceState* st, float* loss, float* lse,
                                     float* z_top, cudaStream_t s) {
  const int cap = sm_count() * 8;
  return launch_dependent(head_loss_kernel, dim3(T < cap ? T : cap), kThreads, 0, 1, s, hidden,
                          weight, H, V, teacher, mask, T, tau, stats, st, loss, lse, z_top);
}

cudaError_t launch_distill_prep(const Teacher& teacher, int V, float tau, const int* idx,
                                int T_alloc, const float* grad_loss, const float* lse,
                                const float* z_top, DeviceState* st, float4* coef,
                                int32_t* patch_ids, uint16_t* patch_values, cudaStream_t s) {
  const int cap = sm_count() * 8;
  return launch_dependent(distill_prep_kernel, dim3(T_alloc < cap ? T_alloc : cap), kThreads, 0, 1,
                          s, teacher, V, tau, idx, T_alloc, grad_loss, lse, z_top, st, coef,
                          patch_ids, patch_values);
}

cudaError_t launch_distill_patch(const int32_t* patch_ids, const uint16_t* patch_values, int K,
                                 const DeviceState* st, int t0, int rows_cap, int v0, int cols,
                                 uint16_t* dz, int64_t dz_ld, cudaStream_t s) {
  const int64_t blocks = (static_cast<int64_t>(rows_cap) * K + kThreads - 1) / kThreads;
  const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
  return launch_dependent(distill_patch_kernel, dim3(static_cast<int>(blocks < cap ? blocks : cap)),
                          kThreads, 0, 1, s, patch_ids, patch_values, K, st, t0, rows_cap, v0,
                          cols, dz, dz_ld);
}

}  // namespace lmh
