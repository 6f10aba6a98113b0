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
constexpr int kBwdMost = 65536;    // backward: bytes of logits per CTA, most and
constexpr int kBwdLeast = 16384;   // least (shorter rows aside)
constexpr int kFwdThreads = 256;   // forward on held logits
constexpr int kFwdDepth = 8;       // its packs in flight per thread (even)
constexpr int kMaxCluster = 8;

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

// The teacher's distribution of one token, formed by one warp: p[k] and the
// log-probability logp[k] in shared memory (0 and -inf where the entry is
// absent); returns P.  NaN entries make P NaN.  each(k, present) runs for every
// entry once its logit is there, for loads that belong to it.
template <class F>
__device__ __forceinline__ float teacher_row(const Teacher& te, int64_t t, float* p, float* logp,
                                             F&& each) {
  const float* a = te.logits + t * te.K;
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int k = lane; k < te.K; k += 32) {
    const float x = a[k];
    each(k, x != -INFINITY);
    logp[k] = x / te.tau;
    m = fmaxf(m, logp[k]);
  }
  // L = base + rest, kept apart so that a distant maximum does not cancel
  float base, rest = 0.f;
  if (te.lse) {
    base = te.lse[t];
  } else {
    m = warp_max(m);
    base = m == -INFINITY ? 0.f : m;
    float s = 0.f;
    for (int k = lane; k < te.K; k += 32) s += expf(logp[k] - base);
    rest = logf(warp_sum(s));
  }
  float P = 0.f;
  for (int k = lane; k < te.K; k += 32) {
    const bool absent = logp[k] == -INFINITY;   // L is -inf where every entry is
    const float lp = absent ? -INFINITY : (logp[k] - base) - rest;
    const float q = absent ? 0.f : expf(lp);
    logp[k] = lp;
    p[k] = q;
    P += q;
  }
  __syncwarp();
  return warp_sum(P);
}

__device__ __forceinline__ float teacher_row(const Teacher& te, int64_t t, float* p, float* logp) {
  return teacher_row(te, t, p, logp, [](int, bool) {});
}

// One entry's part of the loss, relative to the row's maximum: p (log p - (z - m)).
// p = 0 adds nothing, whatever z is; a NaN z (an invalid id) always shows.
__device__ __forceinline__ float loss_term(float p, float logp, float z_rel) {
  return p == 0.f && z_rel == z_rel ? 0.f : p * (logp - z_rel);
}

// Running maximum m of the unscaled logits and s = sum 2^((x - m) c), in two
// halves, over a chunk of N pairs: one maximum, one rescale, then the
// exponentials.  -inf adds exactly nothing; NaN and +inf turn s into NaN.  m is
// subtracted before c multiplies: x c and m c overflow for a mask of the type's
// lowest value.
template <int N>
__device__ __forceinline__ void fold(float& m, float2& s, const float2 (&x)[N], float c) {
  float top = m;
#pragma unroll
  for (int j = 0; j < N; ++j) top = fmaxf(top, fmaxf(x[j].x, x[j].y));
  const float base = top == -INFINITY ? 0.f : top;
  if (top > m) {
    const float w = ex2_approx((m - base) * c);
    s = mul2(s, make_float2(w, w));
    m = top;
  }
  const float2 minus = make_float2(-base, -base), c2 = make_float2(c, c);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float2 d = mul2(add2(x[j], minus), c2);
    s = add2(s, make_float2(ex2_approx(d.x), ex2_approx(d.y)));
  }
}

// A cluster of CTAs per row (one CTA when there are rows enough), each with a
// range of its columns; ranks above 0 hand their maximum and sum to rank 0 in
// distributed shared memory.  Packs come through a ring of asynchronous copies in
// shared memory.  Warp 0 of rank 0 forms the teacher's side while its first
// packs arrive, and the loss at the end.
template <typename T>
__global__ void __launch_bounds__(kFwdThreads) logits_fwd_kernel(DistillLogits a) {
  extern __shared__ __align__(16) float teacher[];   // ring of packs; p, log p, logits [K]
  __shared__ float red[2][kFwdThreads / 32];
  __shared__ float joined[2][2 * kMaxCluster];       // by row parity: maxima, sums
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr int VEC = kVec<T>;
  uint32_t size;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  const uint32_t rank = cluster_cta_rank();
  const int K = a.teacher.K, threads = blockDim.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool lead = rank == 0 && warp == 0;
  // a thread's packs in flight: it copies and reads only its own slots
  Pack<T, VEC>* const ring = reinterpret_cast<Pack<T, VEC>*>(teacher) + threadIdx.x;
  const uint32_t ring_addr = smem_addr(ring);
  float* const p = teacher + 4 * kFwdDepth * threads;
  float* const logp = p + K;
  float* const at_id = logp + K;
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
    const int head = min(to_boundary(row), a.V), packs = (a.V - head) / VEC;
    const Pack<T, VEC>* const from = reinterpret_cast<const Pack<T, VEC>*>(row + head);
    const int k0 = static_cast<int>(static_cast<int64_t>(packs) * rank / size) + threadIdx.x;
    const int k1 = static_cast<int>(static_cast<int64_t>(packs) * (rank + 1) / size);
    auto fetch = [&](int i) {   // the thread's i-th pack, if there is one
      const int k = k0 + i * threads;
      if (k < k1) copy_async<16>(ring_addr + (i % kFwdDepth) * 16 * threads, from + k);
      copy_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kFwdDepth; ++i) fetch(i);
    float P = 0.f;
    if (lead) {
      // the first 32 ids' logits are on their way while the teacher's side is formed
      const int32_t* const ids = a.teacher.ids + t * K;
      const int early = lane < K ? ids[lane] : 0;
      float first = __int_as_float(0x7fc00000);
      P = teacher_row(a.teacher, t, p, logp, [&](int k, bool present) {
        const int v = present ? wrap_id(k < 32 ? early : ids[k], a.V) : -1;
        const float x = v < 0 ? __int_as_float(0x7fc00000) : to_f32(row[v]);
        if (k < 32)
          first = x;
        else
          at_id[k] = x;
      });
      if (lane < K) at_id[lane] = first;
    }
    float m = -INFINITY;
    float2 s2 = make_float2(0.f, 0.f);
    if (rank == 0) {   // before the first and after the last pack
      const int tail = head + packs * VEC;
      const int i = threadIdx.x < head ? threadIdx.x : tail + static_cast<int>(threadIdx.x) - head;
      if (i < a.V && static_cast<int>(threadIdx.x) < 2 * VEC) {
        const float2 x[1] = {make_float2(to_f32(row[i]), -INFINITY)};
        fold(m, s2, x, c);
      }
    }
    const int mine = k0 < k1 ? (k1 - k0 + threads - 1) / threads : 0;
    for (int i = 0; i < mine; i += 2) {   // two packs at a time
      copy_async_wait<kFwdDepth - 2>();
      const Pack<T, VEC> q0 = ring[(i % kFwdDepth) * threads];
      if (i + 1 < mine) {
        const Pack<T, VEC> q1 = ring[((i + 1) % kFwdDepth) * threads];
        float2 x[VEC];
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          x[j] = pair_of(q0, j);
          x[VEC / 2 + j] = pair_of(q1, j);
        }
        fold(m, s2, x, c);
        fetch(i + kFwdDepth);   // into the slots just read
        fetch(i + kFwdDepth + 1);
      } else {
        float2 x[VEC / 2];
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) x[j] = pair_of(q0, j);
        fold(m, s2, x, c);
      }
    }
    copy_async_wait<0>();
    // the warp's, the CTA's and the cluster's maximum and sum
    float M = warp_max(m);
    float S = warp_sum((s2.x + s2.y) * ex2_approx((m - (M == -INFINITY ? 0.f : M)) * c));
    __syncthreads();   // the previous row's readers of red are done
    if (lane == 0) {
      red[0][warp] = M;
      red[1][warp] = S;
    }
    __syncthreads();
    if (warp == 0) {
      const bool have = lane < threads >> 5;
      const float mw = have ? red[0][lane] : -INFINITY;
      M = warp_max(mw);
      const float base = M == -INFINITY ? 0.f : M;
      S = warp_sum(have ? red[1][lane] * ex2_approx((mw - base) * c) : 0.f);
      if (size > 1 && lane == 0) {
        const uint32_t to = map_to_cta(smem_addr(&joined[flip][rank]), 0);
        st_shared_remote(to, __float_as_int(M));
        st_shared_remote(to + 4 * kMaxCluster, __float_as_int(S));
      }
    }
    if (size > 1) cluster_sync();
    if (!lead) continue;
    if (size > 1) {
      const bool have = lane < size;
      const float mw = have ? joined[flip][lane] : -INFINITY;
      M = warp_max(mw);
      const float base = M == -INFINITY ? 0.f : M;
      S = warp_sum(have ? joined[flip][kMaxCluster + lane] * ex2_approx((mw - base) * c) : 0.f);
    }
    // loss relative to the maximum, so that large logits do not cancel
    const float ln_s = logf(S);
    float term = 0.f;
    for (int k = lane; k < K; k += 32)
      if (logp[k] != -INFINITY) term += loss_term(p[k], logp[k], (at_id[k] - M) / a.tau);
    const float A = warp_sum(term);
    if (lane == 0) {
      a.lse[t] = M / a.tau + ln_s;
      a.loss[t] = P == 0.f ? 0.f : fmaf(P, ln_s, A);
    }
    __syncwarp();   // p, logp and at_id are read before the next row's are written
  }
}

// g P softmax(z) of two logits.  lse is subtracted before log2(e) multiplies (their
// product overflows for a row of the type's lowest value).  fp32 logits take
// 1 / tau to 48 bits; for 16-bit ones the product x / tau is off by 2^-23 of itself,
// far below the result's own rounding.
template <typename T>
struct Dense {
  float2 inv, lo, lse, gP;
  __device__ __forceinline__ Dense(float tau, float lse_, float gP_) {
    const float i = 1.f / tau, l = fmaf(-tau, i, 1.f) * i;
    inv = make_float2(i, i);
    lo = make_float2(l, l);
    lse = make_float2(-lse_, -lse_);
    gP = make_float2(gP_, gP_);
  }
  __device__ __forceinline__ float2 operator()(float2 x) const {
    const float2 d = mul2(fma2(x, inv, sizeof(T) == 4 ? fma2(x, lo, lse) : lse),
                          make_float2(kLog2e, kLog2e));
    return mul2(gP, make_float2(ex2_approx(d.x), ex2_approx(d.y)));
  }
  __device__ __forceinline__ float operator()(float x) const {   // non-finite logits get zero
    return fabsf(x) < INFINITY ? (*this)(make_float2(x, x)).x : 0.f;
  }
};

// CTA (column range, row).  Warp 0 forms the teacher's side while the others find
// the entries of this range and read their logits (d_logits may be the logits
// buffer); the dense pass follows, and the few exact cotangents are written last.
template <typename T>
__global__ void __launch_bounds__(kThreads, 5) logits_bwd_kernel(DistillLogits a, int range) {
  extern __shared__ float teacher[];   // p, log p, id, entries of the range, their cotangents [K]
  __shared__ float total;
  __shared__ int entries;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr int VEC = kVec<T>;
  const int K = a.teacher.K, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* const p = teacher;
  float* const logp = p + K;
  int* const id = reinterpret_cast<int*>(logp + K);
  int* const entry = id + K;
  float* const value = reinterpret_cast<float*>(entry + K);
  const int c0 = blockIdx.x * range, n = min(range, a.V - c0);
  for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
    const T* const src = static_cast<const T*>(a.logits) + t * a.ld + c0;
    T* const dst = static_cast<T*>(a.d_logits) + t * a.d_ld + c0;
    const bool scored = !a.mask || a.mask[t];
    const bool packed = same_offset16(src, static_cast<const T*>(dst));
    const int head = packed ? min(to_boundary(src), n) : n, packs = (n - head) / VEC;
    const int tail = head + packs * VEC;
    const Pack<T, VEC>* const from = reinterpret_cast<const Pack<T, VEC>*>(src + head);
    Pack<T, VEC>* const to = reinterpret_cast<Pack<T, VEC>*>(dst + head);
    Pack<T, VEC> q[kUnroll];
    if (scored) {   // the first packs, on their way meanwhile
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (threadIdx.x + u * kThreads < packs) q[u] = from[threadIdx.x + u * kThreads];
      if (threadIdx.x == 0) entries = 0;
      __syncthreads();   // also: the previous row's readers are done
      if (warp == 0) {
        const float sum = teacher_row(a.teacher, t, p, logp);
        if (lane == 0) total = sum;
      } else {
        for (int k = threadIdx.x - 32; k < K; k += kThreads - 32) {
          const int64_t at = t * K + k;
          const int v = a.teacher.logits[at] == -INFINITY ? -1 : wrap_id(a.teacher.ids[at], a.V);
          const bool here = v >= c0 && v < c0 + n;
          id[k] = here ? v - c0 : -1;
          if (here) {
            const int e = atomicAdd(&entries, 1);
            entry[e] = v - c0;
            value[e] = to_f32(src[v - c0]);
          }
        }
      }
      __syncthreads();
    }
    const float P = scored ? total : 0.f;
    if (P == 0.f) {   // unscored, or no teacher
      Pack<T, VEC> zero;
#pragma unroll
      for (int e = 0; e < VEC; ++e) zero.v[e] = from_f32<T>(0.f);
      for (int i = threadIdx.x; i < head; i += kThreads) dst[i] = from_f32<T>(0.f);
      for (int i = tail + threadIdx.x; i < n; i += kThreads) dst[i] = from_f32<T>(0.f);
      for (int k = threadIdx.x; k < packs; k += kThreads) to[k] = zero;
      continue;
    }
    const float g = a.grad[t] / a.tau;
    const Dense<T> dense(a.tau, a.lse[t], g * P);
    // a warp per entry: repeated ids add up, and each writes the same value
    const int here = entries;
    for (int e = warp; e < here; e += kWarps) {
      const int v = entry[e];
      float taken = 0.f;
      for (int i = lane; i < K; i += 32) taken += id[i] == v ? p[i] : 0.f;
      taken = warp_sum(taken);
      if (lane == 0) {
        const float x = value[e];
        value[e] = fabsf(x) < INFINITY ? fmaf(-g, taken, dense(x)) : 0.f;
      }
    }
#pragma unroll 4
    for (int i = threadIdx.x; i < head; i += kThreads) dst[i] = from_f32<T>(dense(to_f32(src[i])));
    for (int i = tail + threadIdx.x; i < n; i += kThreads) dst[i] = from_f32<T>(dense(to_f32(src[i])));
    for (int k0 = threadIdx.x; k0 < packs; k0 += kUnroll * kThreads) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int k = k0 + u * kThreads;
        if (k >= packs) continue;
        float2 zeros = make_float2(0.f, 0.f);   // 0 x: NaN once a logit is not finite
        Pack<T, VEC> o;
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          const float2 x = pair_of(q[u], j);
          zeros = fma2(x, make_float2(0.f, 0.f), zeros);
          set_pair(o, j, dense(x));
        }
        if (zeros.x != 0.f || zeros.y != 0.f) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) o.v[e] = from_f32<T>(dense(to_f32(q[u].v[e])));
        }
        to[k] = o;
        if (k + kUnroll * kThreads < packs) q[u] = from[k + kUnroll * kThreads];
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < here; e += kThreads) dst[entry[e]] = from_f32<T>(value[e]);
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
  __shared__ float red[kWarps], total;
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
    if (warp == 0) {
      const float sum = teacher_row(te, t, p, logp);
      if (lane == 0) total = sum;
    }
    __syncthreads();
    const float P = total;
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
  __shared__ float total;
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
    if (threadIdx.x < 32) {
      const float sum = teacher_row(te, t, p, logp);
      if (threadIdx.x == 0) total = sum;
    }
    __syncthreads();
    const float P = total;
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
  static std::atomic<int> ready[64];
  const cudaError_t e = allow_shared(ready, reinterpret_cast<const void*>(logits_fwd_kernel<T>),
                                     16 * kFwdDepth * kFwdThreads + 3 * sizeof(float) * kMaxTeacher);
  if (e != cudaSuccess) return e;
  const int64_t packs = static_cast<int64_t>(a.V) / kVec<T> + 1;
  int size = 1;
  // Few rows are split, up to two CTAs per SM: more CTAs only repeat the start and
  // end of a row (512 rows of 151,936 fp32: 57 us in one CTA each, 65 in four;
  // 152 rows: 24 us in two, 31 in four).
  while (size < kMaxCluster && a.T * size < 2ll * sm_count() && packs / (2 * size) >= 2 * kFwdThreads)
    size *= 2;
  int threads = kFwdThreads;
  while (threads > 64 && packs / size < threads * kFwdDepth) threads /= 2;
  const int64_t rows = a.T < (1 << 20) ? a.T : (1 << 20);
  return launch_dependent(logits_fwd_kernel<T>, dim3(static_cast<unsigned>(rows * size)), threads,
                          16 * static_cast<size_t>(kFwdDepth) * threads + 3 * sizeof(float) * a.teacher.K,
                          size, s, a);
}

template <typename T>
cudaError_t logits_bwd(const DistillLogits& a, cudaStream_t s) {
  // Long ranges repeat the teacher's side less often; shorter ones while there are
  // fewer than about four rounds of CTAs.
  const int64_t bytes = static_cast<int64_t>(a.V) * static_cast<int64_t>(sizeof(T));
  const int64_t least = (bytes + kBwdMost - 1) / kBwdMost, most = (bytes + kBwdLeast - 1) / kBwdLeast;
  int64_t ranges = (20ll * sm_count() + a.T - 1) / a.T;
  ranges = ranges < least ? least : ranges > most ? most : ranges;
  const int range = static_cast<int>(((a.V + ranges - 1) / ranges + 63) / 64 * 64);
  const unsigned rows = static_cast<unsigned>(a.T < 32768 ? a.T : 32768);
  return launch_dependent(logits_bwd_kernel<T>,
                          dim3(static_cast<unsigned>((static_cast<int64_t>(a.V) + range - 1) / range), rows),
                          kThreads, 5 * sizeof(float) * a.teacher.K, 1, s, a, range);
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
