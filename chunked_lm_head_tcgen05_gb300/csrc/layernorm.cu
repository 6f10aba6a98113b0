// Layer norm of the rows the head reads, and its gradients.  With
// mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r:
//   y = xh w + b
//   dx = r (h - mean(h) - xh mean(h xh)),  h = dy w
//   dw = sum over rows of dy xh,  db = sum over rows of dy
// All sums are fp32; the variance is the mean square of x - mu (never
// mean(x^2) - mu^2, which cancels when |mu| is large).  Column sums go through
// per-CTA partial rows that are added in a fixed order (no atomics: the same
// inputs give the same bits).
#include "element.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace lmh {
namespace {

constexpr int kRowThreads = 256;
constexpr int kColThreads = 256;   // 32 columns x 8 row lanes
constexpr int kFinishRows = 8;

__device__ __forceinline__ float load_param(const void* p, int type, int64_t i) {
  if (type == kF32) return static_cast<const float*>(p)[i];
  if (type == kBF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(static_cast<const __half*>(p)[i]);
}

// Sum over the CTA, returned to every thread.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) t += red[w];
  return t;
}

// Any width and alignment: one CTA per row, the row read once per pass.
template <typename X, typename Y>
__global__ void __launch_bounds__(kRowThreads)
    norm_fwd_any_kernel(const X* __restrict__ x, int64_t x_ld, const void* __restrict__ w,
                        const void* __restrict__ b, int param_type, int64_t N, int H, float eps,
                        Y* __restrict__ y, int64_t y_ld, float* mean, float* rstd) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float red[kRowThreads / 32];
  for (int64_t t = blockIdx.x; t < N; t += gridDim.x) {
    const X* row = x + t * x_ld;
    float s = 0.f;
    for (int i = threadIdx.x; i < H; i += kRowThreads) s += to_f32(row[i]);
    const float mu = block_sum(s, red) / static_cast<float>(H);
    s = 0.f;
    for (int i = threadIdx.x; i < H; i += kRowThreads) {
      const float d = to_f32(row[i]) - mu;
      s = fmaf(d, d, s);
    }
    const float r = 1.f / sqrtf(block_sum(s, red) / static_cast<float>(H) + eps);
    Y* out = y + t * y_ld;
    for (int i = threadIdx.x; i < H; i += kRowThreads) {
      const float v = (to_f32(row[i]) - mu) * r * load_param(w, param_type, i);
      out[i] = from_f32<Y>(b ? v + load_param(b, param_type, i) : v);
    }
    if (threadIdx.x == 0) {
      if (mean) mean[t] = mu;
      if (rstd) rstd[t] = r;
    }
  }
}

template <typename X, typename D>
__global__ void __launch_bounds__(kRowThreads)
    norm_dx_any_kernel(const D* __restrict__ dy, int64_t dy_ld, const X* __restrict__ x,
                       int64_t x_ld, const void* __restrict__ w, int param_type,
                       const float* __restrict__ mean, const float* __restrict__ rstd, int64_t N,
                       int H, X* __restrict__ dx, int64_t dx_ld) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float red[kRowThreads / 32];
  for (int64_t t = blockIdx.x; t < N; t += gridDim.x) {
    const X* xr = x + t * x_ld;
    const D* gr = dy + t * dy_ld;
    const float mu = mean[t], r = rstd[t];
    float s1 = 0.f, s2 = 0.f;
    for (int i = threadIdx.x; i < H; i += kRowThreads) {
      const float h = to_f32(gr[i]) * load_param(w, param_type, i);
      s1 = fmaf(h, (to_f32(xr[i]) - mu) * r, s1);
      s2 += h;
    }
    const float c1 = block_sum(s1, red) / static_cast<float>(H);
    const float c2 = block_sum(s2, red) / static_cast<float>(H);
    X* out = dx + t * dx_ld;
    for (int i = threadIdx.x; i < H; i += kRowThreads) {
      const float h = to_f32(gr[i]) * load_param(w, param_type, i);
      const float xh = (to_f32(xr[i]) - mu) * r;
      out[i] = from_f32<X>((h - c2 - xh * c1) * r);
    }
  }
}

// Partial column sums: CTA (c, p) adds rows p, p + P, ... of columns
// [32 c, 32 c + 32) and writes row p of part_w / part_b [P][H].
template <typename X, typename D>
__global__ void __launch_bounds__(kColThreads)
    norm_columns_any_kernel(const D* __restrict__ dy, int64_t dy_ld, const X* __restrict__ x,
                            int64_t x_ld, const float* __restrict__ mean,
                            const float* __restrict__ rstd, int64_t N, int H,
                            float* __restrict__ part_w, float* __restrict__ part_b) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float sw[8][33], sb[8][33];
  const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int P = gridDim.y, p = blockIdx.y;
  const int c = blockIdx.x * 32 + lane;
  float aw = 0.f, ab = 0.f;
  if (c < H) {
    for (int64_t t = p + static_cast<int64_t>(sub) * P; t < N; t += 8ll * P) {
      const float g = to_f32(dy[t * dy_ld + c]);
      aw = fmaf(g, (to_f32(x[t * x_ld + c]) - mean[t]) * rstd[t], aw);
      ab += g;
    }
  }
  sw[sub][lane] = aw;
  sb[sub][lane] = ab;
  __syncthreads();
  if (sub == 0 && c < H) {
    for (int k = 1; k < 8; ++k) {
      aw += sw[k][lane];
      ab += sb[k][lane];
    }
    part_w[static_cast<int64_t>(p) * H + c] = aw;
    part_b[static_cast<int64_t>(p) * H + c] = ab;
  }
}

// out[c] (+)= sum over the partial rows, in row order within each of
// kFinishRows lanes and then over the lanes.
__global__ void __launch_bounds__(32 * kFinishRows)
    norm_finish_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b, int P,
                       int H, float* d_weight, float* d_bias, int accumulate) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float red[kFinishRows][33];
  const float* part = blockIdx.y ? part_b : part_w;
  float* out = blockIdx.y ? d_bias : d_weight;
  if (!out) return;
  const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < H)
    for (int p = sub; p < P; p += kFinishRows) a += part[static_cast<int64_t>(p) * H + c];
  red[sub][lane] = a;
  __syncthreads();
  if (sub == 0 && c < H) {
    for (int k = 1; k < kFinishRows; ++k) a += red[k][lane];
    out[c] = accumulate ? out[c] + a : a;
  }
}

template <typename X, typename Y>
cudaError_t fwd_typed(const NormFwd& a, cudaStream_t s) {
  const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
  const int grid = static_cast<int>(a.N < cap ? a.N : cap);
  return launch_dependent(norm_fwd_any_kernel<X, Y>, dim3(grid), kRowThreads, 0, 1, s,
                          static_cast<const X*>(a.x), a.x_ld, a.weight, a.bias, a.param_type, a.N,
                          a.H, a.eps, static_cast<Y*>(a.y), a.y_ld, a.mean, a.rstd);
}

template <typename X, typename D>
cudaError_t bwd_typed(const NormBwd& a, cudaStream_t s) {
  const X* x = static_cast<const X*>(a.x);
  const D* dy = static_cast<const D*>(a.dy);
  cudaError_t e = cudaSuccess;
  // the column sums first: dx may overwrite x or dy
  if (a.d_weight || a.d_bias) {
  const int P = static_cast<int>(a.N < 32 ? 1 : (a.N / 32 < kNormPartials ? a.N / 32 : kNormPartials));
  float* part_w = a.partials;
  float* part_b = a.partials + static_cast<int64_t>(P) * a.H;
  const int cols = (a.H + 31) / 32;
  e = launch_dependent(norm_columns_any_kernel<X, D>, dim3(cols, P), kColThreads, 0, 1,
                                   s, dy, a.dy_ld, x, a.x_ld, a.mean, a.rstd, a.N, a.H, part_w,
                                   part_b);
  if (e != cudaSuccess) return e;
  e = launch_dependent(norm_finish_kernel, dim3(cols, 2), 32 * kFinishRows, 0, 1, s,
                       static_cast<const float*>(part_w), static_cast<const float*>(part_b), P,
                       a.H, a.d_weight, a.d_bias, a.accumulate);
  if (e != cudaSuccess) return e;
  }
  if (a.dx) {
    const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
    const int grid = static_cast<int>(a.N < cap ? a.N : cap);
    e = launch_dependent(norm_dx_any_kernel<X, D>, dim3(grid), kRowThreads, 0, 1,
                                           s, dy, a.dy_ld, x, a.x_ld, a.weight, a.param_type,
                                           a.mean, a.rstd, a.N, a.H, static_cast<X*>(a.dx),
                                           a.dx_ld);
  }
  return e;
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwd& a, cudaStream_t s) {
  if (a.x_type == kF32)
    return a.y_type == kF32 ? fwd_typed<float, float>(a, s) : fwd_typed<float, __nv_bfloat16>(a, s);
  if (a.x_type == kBF16) return fwd_typed<__nv_bfloat16, __nv_bfloat16>(a, s);
  return fwd_typed<__half, __half>(a, s);
}

cudaError_t launch_norm_bwd(const NormBwd& a, cudaStream_t s) {
  if (a.x_type == kF32)
    return a.dy_type == kF32 ? bwd_typed<float, float>(a, s) : bwd_typed<float, __nv_bfloat16>(a, s);
  if (a.x_type == kBF16)
    return a.dy_type == kF32 ? bwd_typed<__nv_bfloat16, float>(a, s)
                             : bwd_typed<__nv_bfloat16, __nv_bfloat16>(a, s);
  return a.dy_type == kF32 ? bwd_typed<__half, float>(a, s) : bwd_typed<__half, __half>(a, s);
}

}  // namespace lmh
