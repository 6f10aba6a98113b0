// Penalties for repeated tokens, biases and grammar masks on logits, and the
// gradient through them.  For row r and id v, with c the occurrences of v in
// the row's outputs and `met` whether v occurs in its prompt or outputs:
//   x1 = met ? (x > 0 ? x / rho : x rho) : x
//   x2 = x1 - (f c + p [c > 0])
//   x3 = x2 + bias_v
//   out = allowed ? x3 : -inf
//   d x = allowed ? (met ? (x > 0 ? 1 / rho : rho) : 1) g : 0
// Each CTA owns a range of one row's columns and counts the row's history into
// a table in shared memory that covers just this range, so there is no
// counting workspace and no global atomic; integer counts do not depend on the
// order they are added in.
#include "element.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace lmh {
namespace {

constexpr int kThreads = 256;
constexpr int kRange = 8192;   // columns per CTA: 32 KB of counts, 32 KB of bias slots

template <typename T, bool kBackward>
__global__ void __launch_bounds__(kThreads) process_kernel(ProcessLogits a, int parts) {
  extern __shared__ uint32_t table[];   // [kRange] 2 * outputs + met, then [kRange] bias slots
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  uint32_t* count = table;
  int* slot = reinterpret_cast<int*>(table + kRange);
  const int words = (a.V + 31) / 32;
  for (int64_t item = blockIdx.x; item < a.R * parts; item += gridDim.x) {
    const int64_t r = item / parts;
    const int c0 = static_cast<int>(item - r * parts) * kRange;
    const int n = min(kRange, a.V - c0);
    // history of the row inside this range
    int64_t p0 = 0, p1 = 0, p2 = 0;
    if (a.tokens) {
      p0 = min(max(a.spans[3 * r], int64_t{0}), a.n_tokens);
      p1 = min(max(a.spans[3 * r + 1], p0), a.n_tokens);
      p2 = min(max(a.spans[3 * r + 2], p1), a.n_tokens);
    }
    int64_t b0 = 0, b1 = 0;
    if (!kBackward && a.bias_offsets) {
      b0 = min(max(a.bias_offsets[r], int64_t{0}), a.n_bias);
      b1 = min(max(a.bias_offsets[r + 1], b0), a.n_bias);
    }
    const bool history = p2 > p0, biased = b1 > b0;
    __syncthreads();   // the previous item's table is no longer read
    for (int i = threadIdx.x; i < n; i += kThreads) {
      count[i] = 0;
      if (biased) slot[i] = 0;
    }
    __syncthreads();
    for (int64_t i = p0 + threadIdx.x; i < p2; i += kThreads) {
      const int64_t v = static_cast<int64_t>(a.tokens[i]) - c0;
      if (v < 0 || v >= n) continue;
      if (i < p1)
        atomicOr(&count[v], 1u);
      else
        atomicAdd(&count[v], 2u);
    }
    // the last entry of an id wins
    for (int64_t i = b0 + threadIdx.x; i < b1; i += kThreads) {
      const int64_t v = static_cast<int64_t>(a.bias_ids[i]) - c0;
      if (v >= 0 && v < n) atomicMax(&slot[v], static_cast<int>(i - b0) + 1);
    }
    __syncthreads();
    const uint32_t* mask = nullptr;
    if (a.allowed) {
      const int64_t m = a.allowed_rows ? a.allowed_rows[r] : r;
      if (m >= 0 && m < a.M) mask = a.allowed + m * words;
    }
    const float rho = a.repetition ? a.repetition[r] : 1.f;
    const float fr = a.frequency ? a.frequency[r] : 0.f;
    const float pr = a.presence ? a.presence[r] : 0.f;
    const T* x = static_cast<const T*>(a.logits) + r * a.ld + c0;
    const T* g = static_cast<const T*>(a.grad) + r * a.grad_ld + c0;
    T* out = static_cast<T*>(a.out) + r * a.out_ld + c0;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int c = c0 + i;
      const bool on = !mask || (mask[c >> 5] >> (c & 31) & 1u);
      float v;
      if (!on) {
        v = kBackward ? 0.f : -INFINITY;
      } else {
        v = to_f32(kBackward ? g[i] : x[i]);
        const uint32_t met = history ? count[i] : 0u;
        if (met) {
          const bool positive = (kBackward ? to_f32(x[i]) : v) > 0.f;
          v = positive ? v / rho : v * rho;
          if (!kBackward && met > 1u) v -= fmaf(fr, static_cast<float>(met >> 1), pr);
        }
        if (!kBackward && biased && slot[i]) v += a.bias_values[b0 + slot[i] - 1];
      }
      out[i] = from_f32<T>(v);
    }
  }
}

template <typename T, bool kBackward>
cudaError_t run(const ProcessLogits& a, cudaStream_t s) {
  static std::atomic<int> ready[64];
  auto* kern = process_kernel<T, kBackward>;
  const cudaError_t e = allow_shared(ready, reinterpret_cast<const void*>(kern),
                                     2 * kRange * sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const int parts = (a.V + kRange - 1) / kRange;
  const int64_t items = a.R * parts;
  const int grid = static_cast<int>(items < (1 << 20) ? items : (1 << 20));
  const size_t smem = (a.bias_offsets ? 2 : 1) * kRange * sizeof(uint32_t);
  return launch_dependent(kern, dim3(grid), kThreads, smem, 1, s, a, parts);
}

template <typename T>
cudaError_t either(const ProcessLogits& a, cudaStream_t s) {
  return a.grad ? run<T, true>(a, s) : run<T, false>(a, s);
}

}  // namespace

cudaError_t launch_process_logits(const ProcessLogits& a, cudaStream_t s) {
  if (a.type == kF32) return either<float>(a, s);
  if (a.type == kBF16) return either<__nv_bfloat16>(a, s);
  return either<__half>(a, s);
}

}  // namespace lmh
