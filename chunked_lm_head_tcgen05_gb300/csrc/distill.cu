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
constexpr int kUnroll = 4;         // backward: 16-byte accesses in flight per thread
constexpr int kBwdBytes = 32768;   // backward: logits per CTA
constexpr int kFwdThreads = 512;   // forward on held logits
constexpr int kFwdUnroll = 4;
constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = kFwdThreads / 32;

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
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) t += red[w];
  return t;
}

__device__ __forceinline__ float block_max(float v, float* red) {
  v = warp_max(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = red[0];
  for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) t = fmaxf(t, red[w]);
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
    for (int k = threadIdx.x; k < te.K; k += static_cast<int>(blockDim.x)) m = fmaxf(m, a[k] / te.tau);
    m = block_max(m, red);
    float s = 0.f;
    base = m == -INFINITY ? 0.f : m;
    for (int k = threadIdx.x; k < te.K; k += static_cast<int>(blockDim.x)) s += expf(a[k] / te.tau - base);
    rest = logf(block_sum(s, red));
  }
  float P = 0.f;
  for (int k = threadIdx.x; k < te.K; k += static_cast<int>(blockDim.x)) {
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

// Running maximum m of the unscaled logits and s = sum 2^((x - m) c), over a
// chunk of N values: one maximum, one rescale, then the exponentials.  -inf adds
// exactly nothing; NaN and +inf turn s into NaN.
template <int N>
__device__ __forceinline__ void fold(float& m, float& s, const float (&x)[N], float c) {
  float top = m;
#pragma unroll
  for (int j = 0; j < N; ++j) top = fmaxf(top, x[j]);
  const float base = top == -INFINITY ? 0.f : top;
  if (top > m) {
    s *= ex2_approx((m - base) * c);
    m = top;
  }
  // subtracted first: x c and base c overflow for a mask of the type's lowest value
#pragma unroll
  for (int j = 0; j < N; ++j) s += ex2_approx((x[j] - base) * c);
}

// A cluster of CTAs per row (one CTA when there are rows enough), each with a
// range of its columns; ranks above 0 hand their maximum and sum to rank 0 in
// distributed shared memory, and rank 0 adds the teacher's side.
template <typename T>
__global__ void __launch_bounds__(kFwdThreads) logits_fwd_kernel(DistillLogits a) {
  extern __shared__ float teacher[];   // p [K], log p [K]
  __shared__ float red[kMaxWarps], red_m[kMaxWarps];
  __shared__ float joined[2][2 * kMaxCluster];   // by row parity: maxima, sums
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr int VEC = kVec<T>;
  uint32_t size;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  const uint32_t rank = cluster_cta_rank();
  const int K = a.teacher.K;
  float* const p = teacher;
  float* const logp = teacher + K;
  const float c = kLog2e / a.tau;
  int flip = 0;
  for (int64_t t = blockIdx.x / size; t < a.T; t += gridDim.x / size, flip ^= 1) {
    if (a.mask && !a.mask[t]) {
      if (rank == 0 && threadIdx.x == 0) {
        a.loss[t] = 0.f;
        a.lse[t] = 0.f;
      }
      continue;
    }
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    const float P = rank == 0 ? teacher_row(a.teacher, t, p, logp, red) : 0.f;
    float m = -INFINITY, s = 0.f;
    const int head = min(to_boundary(row), a.V), packs = (a.V - head) / VEC;
    const int k1 = static_cast<int>(static_cast<int64_t>(packs) * (rank + 1) / size);
    if (rank == 0) {   // before the first and after the last pack
      const int tail = head + packs * VEC;
      const int i = threadIdx.x < head ? threadIdx.x : tail + static_cast<int>(threadIdx.x) - head;
      if (i < a.V && static_cast<int>(threadIdx.x) < 2 * VEC) {
        const float x[1] = {to_f32(row[i])};
        fold(m, s, x, c);
      }
    }
    const Pack<T, VEC>* const from = reinterpret_cast<const Pack<T, VEC>*>(row + head);
    int k = static_cast<int>(static_cast<int64_t>(packs) * rank / size) + threadIdx.x;
    for (; k + (kFwdUnroll - 1) * kFwdThreads < k1; k += kFwdUnroll * kFwdThreads) {
      Pack<T, VEC> q[kFwdUnroll];
#pragma unroll
      for (int u = 0; u < kFwdUnroll; ++u) q[u] = from[k + u * kFwdThreads];
#pragma unroll
      for (int u = 0; u < kFwdUnroll; u += 8 / VEC > 1 ? 2 : 1) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = to_f32(q[u + j / VEC].v[j % VEC]);
        fold(m, s, x, c);
      }
    }
    for (; k < k1; k += kFwdThreads) {
      const Pack<T, VEC> q = from[k];
      float x[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[j] = to_f32(q.v[j]);
      fold(m, s, x, c);
    }
    float M = block_max(m, red_m);
    float base = M == -INFINITY ? 0.f : M;
    float S = block_sum(s * ex2_approx((m - base) * c), red);
    if (size > 1) {
      if (threadIdx.x == 0) {
        const uint32_t to = map_to_cta(smem_addr(&joined[flip][rank]), 0);
        st_shared_remote(to, __float_as_int(M));
        st_shared_remote(to + 4 * kMaxCluster, __float_as_int(S));
      }
      cluster_sync();
      if (rank) continue;
      M = -INFINITY;
      for (uint32_t j = 0; j < size; ++j) M = fmaxf(M, joined[flip][j]);
      base = M == -INFINITY ? 0.f : M;
      S = 0.f;
      for (uint32_t j = 0; j < size; ++j)
        S = fmaf(joined[flip][kMaxCluster + j], ex2_approx((joined[flip][j] - base) * c), S);
    }
    // loss relative to the maximum, so that large logits do not cancel
    const float ln_s = logf(S);
    float term = 0.f;
    for (int j = threadIdx.x; j < K; j += kFwdThreads) {
      if (logp[j] == -INFINITY) continue;
      const int v = wrap_id(a.teacher.ids[t * K + j], a.V);
      term += loss_term(p[j], logp[j], v < 0 ? __int_as_float(0x7fc00000)
                                             : (to_f32(row[v]) - M) / a.tau);
    }
    const float A = block_sum(term, red);
    if (threadIdx.x == 0) {
      a.lse[t] = M / a.tau + ln_s;
      a.loss[t] = P == 0.f ? 0.f : fmaf(P, ln_s, A);
    }
  }
}

// CTA (column range, row).  The K places of the range are computed from the
// logits before the dense pass (d_logits may be the logits buffer) and
// written after it.
template <typename T>
__global__ void __launch_bounds__(kThreads, 6) logits_bwd_kernel(DistillLogits a, int range) {
  extern __shared__ float teacher[];   // p [K], log p [K], id [K]
  __shared__ float red[kWarps];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr int VEC = kVec<T>;
  const int K = a.teacher.K;
  float* const p = teacher;
  float* const logp = teacher + K;
  int* const id = reinterpret_cast<int*>(teacher + 2 * K);
  const float inv_tau = 1.f / a.tau;
  // 1 / tau = inv_tau + inv_lo to 48 bits: the exponent is off by its own rounding only
  const float inv_lo = fmaf(-a.tau, inv_tau, 1.f) * inv_tau;
  const int c0 = blockIdx.x * range, n = min(range, a.V - c0);
  for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
    const T* const src = static_cast<const T*>(a.logits) + t * a.ld + c0;
    T* const dst = static_cast<T*>(a.d_logits) + t * a.d_ld + c0;
    const bool scored = !a.mask || a.mask[t];
    const float P = scored ? teacher_row(a.teacher, t, p, logp, red) : 0.f;
    const bool some = P != 0.f;   // NaN counts as some
    const float g = some ? a.grad[t] * inv_tau : 0.f, lse = some ? a.lse[t] : 0.f, gP = g * P;
    auto dense = [&](float x) {
      if (!(fabsf(x) < INFINITY)) return 0.f;   // NaN and infinities
      return gP * ex2_approx(fmaf(x, inv_tau, fmaf(x, inv_lo, -lse)) * kLog2e);
    };
    float fixed[kMaxTeacher / kThreads];
    if (some) {
      for (int k = threadIdx.x; k < K; k += kThreads) {
        const int v = logp[k] == -INFINITY ? -1 : wrap_id(a.teacher.ids[t * K + k], a.V);
        id[k] = v < c0 || v >= c0 + n ? -1 : v - c0;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kMaxTeacher / kThreads; ++j) {
        const int k = threadIdx.x + j * kThreads;
        if (k >= K || id[k] < 0) continue;
        float taken = 0.f;   // repeated ids add up; each writes the same value
        for (int i = 0; i < K; ++i) taken += id[i] == id[k] ? p[i] : 0.f;
        const float x = to_f32(src[id[k]]);
        fixed[j] = fabsf(x) < INFINITY ? fmaf(-g, taken, dense(x)) : 0.f;
      }
      __syncthreads();   // in place, the dense pass overwrites what was read
    }
    if (same_offset16(src, static_cast<const T*>(dst))) {
      const int head = min(to_boundary(src), n), packs = (n - head) / VEC;
      const int tail = head + packs * VEC;
      const int i = threadIdx.x < head ? threadIdx.x : tail + static_cast<int>(threadIdx.x) - head;
      if (i < n && static_cast<int>(threadIdx.x) < 2 * VEC)
        dst[i] = from_f32<T>(some ? dense(to_f32(src[i])) : 0.f);
      const Pack<T, VEC>* const from = reinterpret_cast<const Pack<T, VEC>*>(src + head);
      Pack<T, VEC>* const to = reinterpret_cast<Pack<T, VEC>*>(dst + head);
      if (!some) {
        Pack<T, VEC> zero;
#pragma unroll
        for (int e = 0; e < VEC; ++e) zero.v[e] = from_f32<T>(0.f);
        for (int k = threadIdx.x; k < packs; k += kThreads) to[k] = zero;
      } else {
        for (int k0 = threadIdx.x; k0 < packs; k0 += kUnroll * kThreads) {
          Pack<T, VEC> q[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u)
            if (k0 + u * kThreads < packs) q[u] = from[k0 + u * kThreads];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            if (k0 + u * kThreads >= packs) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) q[u].v[e] = from_f32<T>(dense(to_f32(q[u].v[e])));
            to[k0 + u * kThreads] = q[u];
          }
        }
      }
    } else {
      for (int i = threadIdx.x; i < n; i += kThreads)
        dst[i] = from_f32<T>(some ? dense(to_f32(src[i])) : 0.f);
    }
    __syncthreads();   // also: the teacher's arrays are free again
    if (!some) continue;
#pragma unroll
    for (int j = 0; j < kMaxTeacher / kThreads; ++j) {
      const int k = threadIdx.x + j * kThreads;
      if (k < K && id[k] >= 0) dst[id[k]] = from_f32<T>(fixed[j]);
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
  // Split rows while they are few: two CTAs per SM or more, and 8 KB or more of a
  // row for each.
  const int64_t bytes = static_cast<int64_t>(a.V) * static_cast<int64_t>(sizeof(T));
  int size = 1;
  while (size < kMaxCluster && a.T * size < 4ll * sm_count() && bytes / (2 * size) >= 8192) size *= 2;
  const int64_t rows = a.T < (1 << 20) ? a.T : (1 << 20);
  return launch_dependent(logits_fwd_kernel<T>, dim3(static_cast<unsigned>(rows * size)), kFwdThreads,
                          2 * sizeof(float) * a.teacher.K, size, s, a);
}

template <typename T>
cudaError_t logits_bwd(const DistillLogits& a, cudaStream_t s) {
  const int most = kBwdBytes / static_cast<int>(sizeof(T));
  const int ranges = static_cast<int>((static_cast<int64_t>(a.V) + most - 1) / most);
  const int range = ((a.V + ranges - 1) / ranges + 63) / 64 * 64;
  const unsigned rows = static_cast<unsigned>(a.T < 32768 ? a.T : 32768);
  return launch_dependent(logits_bwd_kernel<T>,
                          dim3(static_cast<unsigned>((a.V + range - 1) / range), rows), kThreads,
                          3 * sizeof(float) * a.teacher.K, 1, s, a, range);
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
