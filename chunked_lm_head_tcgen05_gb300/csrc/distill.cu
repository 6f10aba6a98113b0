// Distillation from a teacher's top logits.  Token t has K teacher entries
// (id_k, a_k); with the teacher's log-sum-exp L (given, or over the K entries),
//   p_k = exp(a_k / tau' - L),   P = sum_k p_k,
//   loss = sum_k p_k (log p_k - z_{id_k} + lse(z)),    z = logits / tau,
//   d loss / d logits_v = (g / tau) (P softmax(z)_v - sum_{k: id_k = v} p_k).
// So the gradient is dense only through softmax(z): one coefficient per row,
// and K places where something is subtracted.  An entry with a_k = -inf is
// absent (its id is not looked at); a token whose entries are all absent has
// loss 0 and no gradient; entries that repeat an id add up.
// Exponentials over the vocabulary are the hardware's (ex2.approx, off by 2^-22 of
// the value): far below a 16-bit result's rounding, and no more than what an fp32 sum of
// that many terms is off by.  The teacher's K are expf.
#include "element.cuh"
#include "operators.h"
#include "ptx.cuh"

#include <climits>

namespace lmh {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 2;         // backward: 16-byte accesses in flight per thread
constexpr int kBwdMost = 65536;    // backward: bytes of logits per CTA, most and
constexpr int kBwdLeast = 16384;   // least (shorter rows aside)
constexpr int kFwdThreads = 256;   // forward on held logits
constexpr int kFwdDepth = 8;       // its packs in flight per thread (even)
constexpr int kMaxCluster = 8;
constexpr int kRowThreads = 128;   // lists of one row, through the head
constexpr int kLossWarps = 4;      // rows per CTA of the loss, through the head

// Row of the student's table that an entry names: negative ids wrap; -1 for
// an id outside [-V, V).
__device__ __forceinline__ int wrap_id(int id, int V) {
  if (id < 0) id += V;
  return (id >= 0 && id < V) ? id : -1;
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
// distributed shared memory.  Only single CTAs take further rows: a cluster has one
// (see the launch), so nothing guards the handed values against a next row's.  Packs come through a ring of asynchronous copies in
// shared memory.  Warp 0 of rank 0 forms the teacher's side while its first
// packs arrive, and the loss at the end.
// HBM-bound: 512 x 151936 fp32 55 us (5.6 TB/s), 2048 x 151936 bf16 6.1 TB/s.  Packs
// loaded into registers instead, by CTAs of 512: 72 us; the teacher's side formed by
// the whole CTA before the loads: 65.
template <typename T>
__global__ void __launch_bounds__(kFwdThreads) logits_fwd_kernel(DistillLogits a) {
  extern __shared__ __align__(16) float teacher[];   // ring of packs; p, log p, logits [K]
  __shared__ float red[2][kFwdThreads / 32];
  __shared__ float joined[2 * kMaxCluster];          // maxima, sums
  uint32_t size;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  if (size > 1) cluster_sync();   // every CTA runs before one writes to rank 0's memory
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr int VEC = kVec<T>;
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
  for (int64_t t = blockIdx.x / size; t < a.T; t += gridDim.x / size) {
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
        const uint32_t to = map_to_cta(smem_addr(&joined[rank]), 0);
        st_shared_remote(to, __float_as_int(M));
        st_shared_remote(to + 4 * kMaxCluster, __float_as_int(S));
      }
      __syncwarp();
    }
    if (size > 1) cluster_sync();
    if (!lead) continue;
    if (size > 1) {
      const bool have = lane < size;
      const float mw = have ? joined[lane] : -INFINITY;
      M = warp_max(mw);
      const float base = M == -INFINITY ? 0.f : M;
      S = warp_sum(have ? joined[kMaxCluster + lane] * ex2_approx((mw - base) * c) : 0.f);
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
// HBM-bound: 2048 x 151936 bf16, a quarter unscored, 168 us (6.5 TB/s).  Many warps with
// few loads each do best: eight CTAs per SM with two packs in flight per thread; five
// with four packs: 207 us.  K compares per entry by one thread instead of a warp, for
// repeated ids, cost as many instructions as the dense pass (285 us); with kBitmap a row
// without repeated ids makes none.
template <typename T, bool kBitmap>
__global__ void __launch_bounds__(kThreads, 8) logits_bwd_kernel(DistillLogits a, int range) {
  extern __shared__ float teacher[];   // p, log p, id, entries of the range, their cotangents [K]
  __shared__ uint32_t named[kBitmap ? kBwdMost / 2 / 32 : 1];   // a bit per column of the range
  __shared__ float total;
  __shared__ int entries, repeated;
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
  if constexpr (kBitmap)
    for (int i = threadIdx.x; i < range / 32; i += kThreads) named[i] = 0;   // and again after use
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
      if (threadIdx.x == 0) entries = repeated = 0;
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
            entry[e] = kBitmap ? v - c0 | k << 16 : v - c0;   // range <= 2^15 columns, K <= 2^10
            value[e] = to_f32(src[v - c0]);
            if constexpr (kBitmap) {
              const uint32_t bit = 1u << ((v - c0) & 31);
              if (atomicOr(&named[(v - c0) >> 5], bit) & bit) repeated = 1;
            }
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
      if (kBitmap && scored) {
        for (int e = threadIdx.x; e < entries; e += kThreads) named[(entry[e] & 0xffff) >> 5] = 0;
        __syncthreads();   // `entries` is read before the next row's is written
      }
      continue;
    }
    const float g = a.grad[t] / a.tau;
    const Dense<T> dense(a.tau, a.lse[t], g * P);
    const int here = entries;
    if (kBitmap && !repeated) {
      for (int e = threadIdx.x; e < here; e += kThreads) {
        const float x = value[e];
        value[e] = fabsf(x) < INFINITY ? fmaf(-g, p[entry[e] >> 16], dense(x)) : 0.f;
      }
    } else {   // a warp per entry: repeated ids add up, and each writes the same value
      for (int e = warp; e < here; e += kWarps) {
        const int v = kBitmap ? entry[e] & 0xffff : entry[e];
        float taken = 0.f;
        for (int i = lane; i < K; i += 32) taken += id[i] == v ? p[i] : 0.f;
        taken = warp_sum(taken);
        if (lane == 0) {
          const float x = value[e];
          value[e] = fabsf(x) < INFINITY ? fmaf(-g, taken, dense(x)) : 0.f;
        }
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
    for (int e = threadIdx.x; e < here; e += kThreads) {
      const int v = kBitmap ? entry[e] & 0xffff : entry[e];
      dst[v] = from_f32<T>(value[e]);
      if constexpr (kBitmap) named[v >> 5] = 0;
    }
  }
}

// ------------------------------------------------------------------ through the head
// A row's K ids in ascending order: position of entry k among them.  Entries
// without an id (absent, or outside [-V, V)) have key INT_MAX and come last, in
// entry order.  Ranks by counting: K compares per entry, all from shared memory.
__device__ __forceinline__ int id_key(const Teacher& te, int64_t at, int V) {
  if (te.logits[at] == -INFINITY) return INT_MAX;
  const int v = wrap_id(te.ids[at], V);
  return v < 0 ? INT_MAX : v;
}

__device__ __forceinline__ int rank_of(const int* key, int K, int k) {
  const int mine = key[k];
  int rank = 0;
  for (int j = 0; j < K; ++j) rank += key[j] < mine || (key[j] == mine && j < k);
  return rank;
}

// start[n] = entries whose id lies before 256-column tile n.
__device__ __forceinline__ void tile_starts(const int* sorted, int K, int n_tiles, uint16_t* start) {
  for (int n = threadIdx.x; n <= n_tiles; n += kRowThreads) {
    int lo = 0, hi = K;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sorted[mid] < n * BN)
        lo = mid + 1;
      else
        hi = mid;
    }
    start[n] = static_cast<uint16_t>(lo);
  }
}

// Lists of the forward, one CTA per compacted row: ids ascending, the entry each
// came from, and where each tile's begin.
__global__ void __launch_bounds__(kRowThreads)
    distill_lists_kernel(Teacher te, int V, const int* __restrict__ idx, const DeviceState* st,
                         int T_alloc, RowIds lists, int32_t* out_ids, uint16_t* out_start,
                         uint16_t* order) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ int key[kMaxTeacher], sorted[kMaxTeacher];
  const int K = te.K, rows = min(st->rows, T_alloc);
  for (int r = blockIdx.x; r < rows; r += gridDim.x) {
    const int64_t t = idx ? idx[r] : r;
    for (int k = threadIdx.x; k < K; k += kRowThreads) key[k] = id_key(te, t * K + k, V);
    __syncthreads();
    for (int k = threadIdx.x; k < K; k += kRowThreads) {
      const int at = rank_of(key, K, k);
      sorted[at] = key[k];
      out_ids[static_cast<int64_t>(r) * K + at] = key[k];
      order[static_cast<int64_t>(r) * K + at] = static_cast<uint16_t>(k);
    }
    __syncthreads();
    tile_starts(sorted, K, lists.start_ld - 1, out_start + static_cast<int64_t>(r) * lists.start_ld);
  }
}

// The loss, one warp per compacted row: the vocabulary splits' statistics joined,
// the picked logits put back in entry order.  z - max is taken in the statistics'
// own units, u = (h . w) scale with the scale the GEMM used, so that the rounding
// of log2(e) / tau cancels.
__global__ void __launch_bounds__(32 * kLossWarps)
    distill_loss_kernel(Teacher te, int V, float tau, const int* __restrict__ idx, DeviceState* st,
                        int T_alloc, const float4* __restrict__ partials, int n_splits, int part_ld,
                        const int32_t* __restrict__ sorted, const uint16_t* __restrict__ order,
                        const float* __restrict__ picked, float* loss, float* lse, float* z_top) {
  extern __shared__ float teacher[];   // per warp: p, log p, u [K]
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int K = te.K, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* const p = teacher + 3 * K * warp;
  float* const logp = p + K;
  float* const u = logp + K;
  const float scale = kLog2e / tau;
  const int rows = min(st->rows, T_alloc);
  for (int r = blockIdx.x * kLossWarps + warp; r < rows; r += gridDim.x * kLossWarps) {
    const int64_t t = idx ? idx[r] : r, at = static_cast<int64_t>(r) * K;
    const float4 q = lane < n_splits ? partials[static_cast<int64_t>(lane) * part_ld + r]
                                     : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    const float P = teacher_row(te, t, p, logp);
    bool bad = false;
    for (int j = lane; j < K; j += 32) {
      const int k = order[at + j];
      float z = 0.f, own = 0.f;
      if (sorted[at + j] != INT_MAX) {
        own = picked[at + j];
        z = own / tau;
      } else if (te.logits[t * K + k] != -INFINITY) {   // present, but no id of the vocabulary
        z = own = __int_as_float(0x7fc00000);
        bad = true;
      }
      u[k] = own * scale;
      z_top[t * K + k] = z;
    }
    if (bad) atomicCAS(&st->status, 0, STATUS_BAD_TARGET);
    __syncwarp();
    const float M = warp_max(q.x);
    const float ln_s = logf(warp_sum(q.y * exp2f(q.x - M)));
    float term = 0.f;
    for (int k = lane; k < K; k += 32)
      if (logp[k] != -INFINITY) term += loss_term(p[k], logp[k], (u[k] - M) * kLn2);
    const float A = warp_sum(term);
    if (lane == 0) {
      lse[t] = fmaf(M, kLn2, ln_s);
      loss[t] = P == 0.f ? 0.f : fmaf(P, ln_s, A);
    }
    __syncwarp();
  }
}

__global__ void distill_zero_kernel(const uint8_t* __restrict__ mask, int T, int K, float* loss,
                                    float* lse, float* z_top) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  for (int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; t < T; t += (gridDim.x * blockDim.x) >> 5) {
    if (mask[t]) continue;
    for (int k = lane; k < K; k += 32) z_top[static_cast<int64_t>(t) * K + k] = 0.f;
    if (lane == 0) loss[t] = lse[t] = 0.f;
  }
}

// The backward's side of a row, one CTA per compacted row: the GEMM epilogue's
// coefficients (dz = g P softmax(z) for every id) and, in ascending order of the
// teacher's ids, the cotangents that replace the dense ones there.  Either kind is formed
// in fp32 and rounded to bf16 once, in the dz block: both gradient products read it as a
// tensor-core operand, whose type is the other operand's.  2048 tokens, V 151936: gradients
// off by 1.7e-3 of their norm from that, and as much from a bf16 result's own rounding.
__global__ void __launch_bounds__(kRowThreads)
    distill_prep_kernel(Teacher te, int V, float tau, const int* __restrict__ idx, int T_alloc,
                        const float* __restrict__ grad_loss, const float* __restrict__ lse,
                        const float* __restrict__ z_top, DeviceState* st, float4* coef,
                        RowIds lists, int32_t* out_ids, uint16_t* out_start, float* out_values) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float total;
  __shared__ float p[kMaxTeacher], logp[kMaxTeacher];
  __shared__ int key[kMaxTeacher], sorted[kMaxTeacher];
  const int K = te.K;
  const int rows = st->rows;
  for (int r = blockIdx.x; r < T_alloc; r += gridDim.x) {
    if (r >= rows) {
      if (threadIdx.x == 0) coef[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      continue;
    }
    const int64_t t = idx ? idx[r] : r;
    if (threadIdx.x < 32) {
      const float sum = teacher_row(te, t, p, logp);
      if (threadIdx.x == 0) total = sum;
    }
    bool bad = false;
    for (int k = threadIdx.x; k < K; k += kRowThreads) {
      key[k] = id_key(te, t * K + k, V);
      bad |= key[k] == INT_MAX && te.logits[t * K + k] != -INFINITY;
    }
    if (bad) atomicCAS(&st->status, 0, STATUS_BAD_TARGET);
    __syncthreads();
    const float P = total, g = grad_loss[t] / tau, L = lse[t];
    const float gP = P == 0.f ? 0.f : g * P;   // a row without a teacher has no gradient
    if (threadIdx.x == 0) coef[r] = make_float4(L * kLog2e, 0.f, -gP, 0.f);
    for (int k = threadIdx.x; k < K; k += kRowThreads) {
      const int at = rank_of(key, K, k);
      float taken = 0.f;   // repeated ids add up, and each writes the same value
      for (int i = 0; i < K; ++i) taken += key[i] == key[k] ? p[i] : 0.f;
      const float q = ex2_approx((z_top[t * K + k] - L) * kLog2e);
      const float value = P == 0.f || key[k] == INT_MAX ? 0.f : fmaf(gP, q, -g * taken);
      sorted[at] = key[k];
      out_ids[static_cast<int64_t>(r) * K + at] = key[k];
      out_values[static_cast<int64_t>(r) * K + at] = value;
    }
    __syncthreads();
    tile_starts(sorted, K, lists.start_ld - 1, out_start + static_cast<int64_t>(r) * lists.start_ld);
    __syncthreads();
  }
}

// Two launches per block: the dz GEMM has stored the dense cotangents of rows
// [t0, t0 + rows_cap), vocabulary rows [v0, v0 + cols).
__global__ void __launch_bounds__(kThreads)
    distill_patch_kernel(const int32_t* __restrict__ ids, const float* __restrict__ values, int K,
                         const DeviceState* st, int t0, int rows_cap, int v0, int cols, uint16_t* dz,
                         int64_t dz_ld) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int rows = min(st->rows - t0, rows_cap);
  const int64_t n = rows > 0 ? static_cast<int64_t>(rows) * K : 0;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t at = static_cast<int64_t>(t0) * K + i;
    const int v = ids[at];
    if (v < v0 || v - v0 >= cols) continue;
    dz[(i / K) * dz_ld + (v - v0)] = __bfloat16_as_ushort(__float2bfloat16_rn(values[at]));
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
  // every row a CTA or cluster of its own, up to far more rows than are ever split
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
  // Comparing ids takes K compares for each of a range's about K range / V entries: with
  // many, a bitmap that shows whether a row repeats an id at all is faster (6,171 rows of
  // 2,491 fp16, K 213: 35 us against 146; 3,193 of 48,721 fp16, K 126: 115 against 126), with
  // few it is slower (2,048 of 151,936 bf16, K 128: 178 against 168).
  const int64_t K = a.teacher.K;
  auto* const kern = K * K * range >= 5000ll * a.V ? logits_bwd_kernel<T, true>
                                                   : logits_bwd_kernel<T, false>;
  return launch_dependent(kern,
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

cudaError_t launch_distill_lists(const Teacher& teacher, int V, const int* idx, int T_alloc,
                                 const DeviceState* st, const RowIds& lists, int32_t* ids,
                                 uint16_t* start, uint16_t* order, cudaStream_t s) {
  const int cap = sm_count() * 16;
  return launch_dependent(distill_lists_kernel, dim3(T_alloc < cap ? T_alloc : cap), kRowThreads, 0,
                          1, s, teacher, V, idx, st, T_alloc, lists, ids, start, order);
}

cudaError_t launch_distill_loss(const Teacher& teacher, int V, float tau, const int* idx,
                                int T_alloc, DeviceState* st, const float4* partials, int n_splits,
                                int part_ld, const RowIds& lists, const uint16_t* order,
                                const float* picked, float* loss, float* lse, float* z_top,
                                cudaStream_t s) {
  static std::atomic<int> ready[64];
  const cudaError_t e = allow_shared(ready, reinterpret_cast<const void*>(distill_loss_kernel),
                                     3 * sizeof(float) * kMaxTeacher * kLossWarps);
  if (e != cudaSuccess) return e;
  const int ctas = (T_alloc + kLossWarps - 1) / kLossWarps, cap = sm_count() * 16;
  return launch_dependent(distill_loss_kernel, dim3(ctas < cap ? ctas : cap), 32 * kLossWarps,
                          3 * sizeof(float) * teacher.K * kLossWarps, 1, s, teacher, V, tau, idx, st,
                          T_alloc, partials, n_splits, part_ld, lists.ids, order, picked, loss, lse,
                          z_top);
}

cudaError_t launch_distill_zero(const uint8_t* mask, int T, int K, float* loss, float* lse,
                                float* z_top, cudaStream_t s) {
  const int64_t ctas = (static_cast<int64_t>(T) * 32 + 255) / 256, cap = sm_count() * 16;
  return launch_dependent(distill_zero_kernel, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)),
                          256, 0, 1, s, mask, T, K, loss, lse, z_top);
}

cudaError_t launch_distill_prep(const Teacher& teacher, int V, float tau, const int* idx,
                                int T_alloc, const float* grad_loss, const float* lse,
                                const float* z_top, DeviceState* st, float4* coef,
                                const RowIds& lists, int32_t* ids, uint16_t* start, float* values,
                                cudaStream_t s) {
  const int cap = sm_count() * 16;
  return launch_dependent(distill_prep_kernel, dim3(T_alloc < cap ? T_alloc : cap), kRowThreads, 0,
                          1, s, teacher, V, tau, idx, T_alloc, grad_loss, lse, z_top, st, coef, lists,
                          ids, start, values);
}

cudaError_t launch_distill_patch(const int32_t* ids, const float* values, int K,
                                 const DeviceState* st, int t0, int rows_cap, int v0, int cols,
                                 uint16_t* dz, int64_t dz_ld, cudaStream_t s) {
  const int64_t blocks = (static_cast<int64_t>(rows_cap) * K + kThreads - 1) / kThreads;
  const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
  return launch_dependent(distill_patch_kernel, dim3(static_cast<int>(blocks < cap ? blocks : cap)),
                          kThreads, 0, 1, s, ids, values, K, st, t0, rows_cap, v0, cols, dz, dz_ld);
}

}  // namespace lmh
