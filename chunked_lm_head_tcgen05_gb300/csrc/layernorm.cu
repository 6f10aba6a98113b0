// Layer norm of the rows the head reads, and its gradients.  With
// mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r:
//   y = xh w + b
//   dx = r (h - mean(h) - xh mean(h xh)),  h = dy w
//   dw = sum over rows of dy xh,  db = sum over rows of dy
// All sums and statistics are fp32; the variance is the mean square of x - mu (never
// mean(x^2) - mu^2, which cancels when |mu| is large).  Column sums go through
// per-CTA partial rows that are added in a fixed order (no atomics: the same
// inputs give the same bits).
#include "element.cuh"
#include "operators.h"
#include "ptx.cuh"

#include <algorithm>

namespace lmh {
namespace {

constexpr int kFwdMaxThreads = 1024;   // forward, one CTA per row
constexpr int kFwdWarpRows = 4;        // forward, one warp per row: rows per CTA
constexpr int kStreamThreads = 768;    // forward with many rows: most threads per CTA (85 registers each)
constexpr int kBwdThreads = 512;       // backward: most threads per CTA
constexpr int kGroupThreads = 512;     // most threads of a row: 16 warps, half a warp reads their sums
static_assert(kBwdThreads <= kGroupThreads, "a row's warps");
constexpr int kRowThreads = 256;
constexpr int kFinishRows = 16;

__device__ __forceinline__ float load_param(const void* p, int type, int64_t i) {
  if (type == kF32) return static_cast<const float*>(p)[i];
  if (type == kBF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(static_cast<const __half*>(p)[i]);
}

// VEC parameters from index i (a multiple of VEC; 16-byte aligned base if VEC > 1).
template <int VEC>
__device__ __forceinline__ void load_params(const void* p, int type, int i, float (&v)[VEC]) {
  if (type == kF32) {
    constexpr int N = VEC < 4 ? VEC : 4;
#pragma unroll
    for (int j = 0; j < VEC; j += N) {
      const Pack<float, N> q = *reinterpret_cast<const Pack<float, N>*>(
          static_cast<const float*>(p) + i + j);
#pragma unroll
      for (int e = 0; e < N; ++e) v[j + e] = q.v[e];
    }
  } else if (type == kBF16) {
    const Pack<__nv_bfloat16, VEC> q = *reinterpret_cast<const Pack<__nv_bfloat16, VEC>*>(
        static_cast<const __nv_bfloat16*>(p) + i);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = to_f32(q.v[e]);
  } else {
    const Pack<__half, VEC> q =
        *reinterpret_cast<const Pack<__half, VEC>*>(static_cast<const __half*>(p) + i);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = to_f32(q.v[e]);
  }
}

// Element e of a row of pairs (e known at compile time).
template <int N>
__device__ __forceinline__ float& at(float2 (&v)[N], int e) {
  return e & 1 ? v[e >> 1].y : v[e >> 1].x;
}

// Sums of two values over a warp in one tree: lanes 0..15 return the first, lanes
// 16..31 the second.
__device__ __forceinline__ float warp_sum_halves(float a, float b) {
  const bool upper = threadIdx.x & 16;
  const float other = __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
  float v = (upper ? b : a) + other;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
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

// A row in the registers of one warp (kPerWarp, for short rows) or one CTA (few
// rows, or wide ones): read once, NV packs of VEC elements per thread.  Bound by
// the chain of load, two reductions and store, about 2 us (one row of 2560); short
// rows of many, 65536 x 512 bf16, reach 3.9 TB/s.  Warps form mean and squared deviations about
// their own mean; with one CTA per row those are joined by
//   M2 = sum_w M2_w + n_w (mean_w - mean)^2
// after a single barrier.
template <typename X, typename Y, int VEC, int NV, bool kPerWarp>
__global__ void __launch_bounds__(kPerWarp ? 32 * kFwdWarpRows : kFwdMaxThreads)
    norm_fwd_kernel(const X* __restrict__ x, int64_t x_ld, const void* __restrict__ w,
                    const void* __restrict__ b, int param_type, int64_t N, int H, float eps,
                    Y* __restrict__ y, int64_t y_ld, float* mean, float* rstd) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float red[3][kPerWarp ? 1 : kFwdMaxThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = kPerWarp ? 32 : blockDim.x;
  const int i = kPerWarp ? lane : threadIdx.x;
  const int64_t t = kPerWarp ? static_cast<int64_t>(blockIdx.x) * kFwdWarpRows + warp
                             : static_cast<int64_t>(blockIdx.x);
  if (t >= N) return;   // whole warps, and only where warps work alone
  const X* row = x + t * x_ld;
  const int n = H / VEC;
  Pack<X, VEC> raw[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (i + k * g < n) raw[k] = *reinterpret_cast<const Pack<X, VEC>*>(row + (i + k * g) * VEC);
  float s = 0.f;
  int cnt = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (i + k * g < n) {
      cnt += VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += to_f32(raw[k].v[e]);
    }
  cnt = __reduce_add_sync(0xffffffffu, cnt);
  float mu = cnt ? warp_sum(s) / static_cast<float>(cnt) : 0.f;
  float m2 = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (i + k * g < n) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = to_f32(raw[k].v[e]) - mu;
        m2 = fmaf(d, d, m2);
      }
    }
  m2 = warp_sum(m2);
  if (!kPerWarp && blockDim.x > 32) {
    if (lane == 0) {
      red[0][warp] = static_cast<float>(cnt);
      red[1][warp] = mu;
      red[2][warp] = m2;
    }
    __syncthreads();
    const int warps = blockDim.x >> 5;
    const float c = lane < warps ? red[0][lane] : 0.f;
    const float mw = lane < warps ? red[1][lane] : 0.f;
    mu = warp_sum(c * mw) / static_cast<float>(H);
    const float d = mw - mu;
    m2 = warp_sum(lane < warps ? fmaf(c * d, d, red[2][lane]) : 0.f);
  }
  const float r = 1.f / sqrtf(m2 / static_cast<float>(H) + eps);
  Y* out = y + t * y_ld;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (i + k * g < n) {
      const int c = (i + k * g) * VEC;
      float wv[VEC], bv[VEC];
      load_params<VEC>(w, param_type, c, wv);
      if (b) load_params<VEC>(b, param_type, c, bv);
      Pack<Y, VEC> o;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float v = (to_f32(raw[k].v[e]) - mu) * r * wv[e];
        o.v[e] = from_f32<Y>(b ? v + bv[e] : v);
      }
      *reinterpret_cast<Pack<Y, VEC>*>(out + c) = o;
    }
  if (i == 0) {
    if (mean) mean[t] = mu;
    if (rstd) rstd[t] = r;
  }
}

// Many rows: a group of g threads (a multiple of 32) takes row after row, each
// thread always the same columns, so that weight and bias stay in registers and
// rows arrive through a ring of asynchronous copies kDepth rows deep (kDepth = 0:
// units too small for such copies; a row's loads are issued a row ahead).  One
// barrier per row and group.  The statistics join by
//   mean = ref + sum n_j (m_j - ref) / n,  M2 = sum M2_j + n_j (m_j - ref)^2 - n (mean - ref)^2
// over threads and then warps, with one part's own mean as ref: both sums at once,
// and what cancels is no larger than that part's share of M2 times the parts.
// HBM-bound: 65536 x 2560 bf16 110 us, 6.1 TB/s (90% of the measured copy rate).  One
// warp per row, its weights from L1 each time: 154 us; four shuffle trees instead of
// two half ones: 133; 512 threads per CTA (three rows at once instead of four): 126.
template <typename X, typename Y, int VEC, int NV, int kDepth, bool kFull>
__global__ void __launch_bounds__(kStreamThreads)
    norm_fwd_stream_kernel(const X* __restrict__ x, int64_t x_ld, const void* __restrict__ w,
                           const void* __restrict__ b, int param_type, int64_t N, int H, float eps,
                           Y* __restrict__ y, int64_t y_ld, float* mean, float* rstd, int g) {
  extern __shared__ __align__(16) char ring_bytes[];
  __shared__ float red[2][3][kStreamThreads / 32];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int groups = blockDim.x / g;
  const int grp = threadIdx.x / g, i = threadIdx.x - grp * g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = g >> 5, w0 = grp * warps;
  constexpr bool kRing = kDepth > 0;
  const int n = H / VEC;
  auto in = [&](int k) { return kFull || i + k * g < n; };   // kFull: n = NV g
  const PackRing<X, VEC> ring(ring_bytes, blockDim.x, threadIdx.x);
  float2 wv[NV * VEC / 2], bv[NV * VEC / 2];
  int cnt = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float one[VEC] = {}, two[VEC] = {};
    if (in(k)) {
      cnt += VEC;
      load_params<VEC>(w, param_type, (i + k * g) * VEC, one);
      if (b) load_params<VEC>(b, param_type, (i + k * g) * VEC, two);
    } else if constexpr (kRing) {   // slots that are never filled read as zeros
#pragma unroll
      for (int d = 0; d < kDepth; ++d) ring.clear(d * NV + k);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      at(wv, k * VEC + e) = one[e];
      at(bv, k * VEC + e) = two[e];
    }
  }
  const float own_cnt = static_cast<float>(cnt), own_inv = cnt ? 1.f / own_cnt : 0.f;
  const float inv_H = 1.f / static_cast<float>(H);
  // columns of the group's (lane % 16)-th warp, which fills NV rounds of 32 packs
  float share = 0.f;
  for (int k = 0; k < NV; ++k)
    share += static_cast<float>(VEC * min(max(n - ((lane & 15) * 32 + k * g), 0), 32));
  const float share_inv = share > 0.f ? 1.f / share : 0.f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * groups + grp, next = t;
  int put = 0, get = 0;
  Pack<X, VEC> ahead[kRing ? 1 : NV];
  auto fetch = [&] {
    if (next < N) {
      const X* from = x + next * x_ld + i * VEC;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!in(k)) continue;
        if constexpr (kRing)
          ring.fetch(put * NV + k, from + k * g * VEC);
        else
          ahead[k] = *reinterpret_cast<const Pack<X, VEC>*>(from + k * g * VEC);
      }
    }
    if constexpr (kRing) {
      copy_async_commit();
      put = put + 1 == kDepth ? 0 : put + 1;
    }
    next += step;
  };
#pragma unroll
  for (int d = 0; d < (kRing ? kDepth : 1); ++d) fetch();
  for (int flip = 0; t < N; t += step, flip ^= 1) {
    if constexpr (kRing) copy_async_wait<kRing ? kDepth - 1 : 0>();
    // the thread's mean and squared deviations about it (pairs of columns: within a
    // pack, or of neighbouring packs of one element)
    constexpr int kPairs = NV * VEC / 2;
    float2 v[kPairs];
    float2 s2 = make_float2(0.f, 0.f), q2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      Pack<X, VEC> q;
      if constexpr (kRing)
        q = ring.read(get * NV + k);
      else
        q = ahead[k];
      if constexpr (VEC > 1) {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) v[k * VEC / 2 + e] = pair_of(q, e);
      } else {
        at(v, k) = in(k) ? to_f32(q.v[0]) : 0.f;
      }
    }
    if constexpr (kRing)
      get = get + 1 == kDepth ? 0 : get + 1;
    else
      fetch();
#pragma unroll
    for (int j = 0; j < kPairs; ++j) s2 = add2(s2, v[j]);
    const float own = (s2.x + s2.y) * own_inv;
    const float2 minus_own = make_float2(-own, -own);
    if constexpr (VEC > 1) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!in(k)) continue;
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          const float2 d = add2(v[k * VEC / 2 + e], minus_own);
          q2 = fma2(d, d, q2);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const float d = in(k) ? at(v, k) - own : 0.f;
        q2.x = fmaf(d, d, q2.x);
      }
    }
    // the warp's, about lane 0's mean: its two sums go to shared memory
    const float first = __shfl_sync(0xffffffffu, own, 0);
    const float d0 = own - first, d1 = own_cnt * d0;
    const float half = warp_sum_halves(d1, fmaf(d1, d0, q2.x + q2.y));
    if constexpr (kRing) fetch();   // into the slots just read, all of whose values are in the sums
    if ((lane & 15) == 0) red[flip][lane >> 4][warp] = half;
    if (lane == 1) red[flip][2][warp] = first;
    if (warps > 1)
      named_bar_sync(1 + grp, g);
    else
      __syncwarp();
    // the group's, about its first warp's mean
    const int wl = w0 + min(lane & 15, warps - 1);
    const bool have = (lane & 15) < warps;
    const float s1w = red[flip][0][wl], q1w = red[flip][1][wl], fw = red[flip][2][wl];
    const float mw = fmaf(s1w, share_inv, fw);
    const float ref = __shfl_sync(0xffffffffu, mw, 0);
    const float dw = mw - ref, nd = share * dw;
    const float part = lane < 16 ? nd : fmaf(nd, dw, fmaf(-s1w * share_inv, s1w, q1w));
    float sum = have ? part : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float e1 = __shfl_sync(0xffffffffu, sum, 0), e2 = __shfl_sync(0xffffffffu, sum, 16);
    const float mu = fmaf(e1, inv_H, ref);
    float var = fmaf(-e1 * inv_H, e1, e2) * inv_H;
    var = var < 0.f ? 0.f : var;   // rounding, where a row has no spread
    const float r = rsqrtf(var + eps);   // 2 units of the last place off at most; one value per row
    const float2 minus_mu = make_float2(-mu, -mu), r2 = make_float2(r, r);
    Y* out = y + t * y_ld + i * VEC;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) v[j] = fma2(mul2(add2(v[j], minus_mu), r2), wv[j], bv[j]);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!in(k)) continue;
      Pack<Y, VEC> o;
      if constexpr (VEC > 1) {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) set_pair(o, e, v[k * VEC / 2 + e]);
      } else {
        o.v[0] = from_f32<Y>(at(v, k));
      }
      *reinterpret_cast<Pack<Y, VEC>*>(out + k * g * VEC) = o;
    }
    if (i == 0) {
      if (mean) mean[t] = mu;
      if (rstd) rstd[t] = r;
    }
  }
  if constexpr (kRing) copy_async_wait<0>();
}

// Both gradients in one pass over x and dy.  A group of g threads (a multiple of
// 32) owns a row at a time and its threads fixed columns, so dw and db gather in
// registers over the group's rows; dx may be x or dy (each thread writes what it alone
// has read).  The CTA's groups are joined in shared memory at the end, and the CTA writes
// one partial row.  Rows of more than `cols` columns
// go in blocks of that many (blockIdx.y), their two sums having been formed before
// (`sums`); narrower ones in one block that forms them itself.  Rows arrive through a ring of
// asynchronous copies kDepth rows deep (kDepth = 0: units too small for such
// copies; a row's loads are then issued before the previous row's sums).
// HBM-bound with many rows: 65536 x 2560 bf16 6.0 TB/s.  4096 x 2560 with fp32 dy takes
// 20 us and 4 more for the join of the partial rows (floor 12): nine rows per group
// are too few to hide the first loads and the join.
template <typename X, typename D, int VEC, int NV, int kDepth, bool kFull>
__global__ void __launch_bounds__(kBwdThreads)
    norm_bwd_kernel(const D* dy, int64_t dy_ld, const X* x, int64_t x_ld,
                    const void* __restrict__ w, int param_type, const float* __restrict__ mean,
                    const float* __restrict__ rstd, int64_t N, int H, int cols,
                    const float2* __restrict__ sums, X* dx, int64_t dx_ld,
                    float* __restrict__ part_w, float* __restrict__ part_b, int g) {
  extern __shared__ __align__(16) char ring_bytes[];   // x and dy in flight; then [2][W] sums
  __shared__ float red[2][2][kBwdThreads / 32];
  constexpr bool kRing = kDepth > 0;
  constexpr int kRegs = kRing ? 1 : NV;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int c_first = blockIdx.y * cols, W = min(cols, H - c_first);
  x += c_first;
  dy += c_first;
  if (dx) dx += c_first;
  if (part_w) {
    part_w += c_first;
    part_b += c_first;
  }
  const int groups = blockDim.x / g;
  const int grp = threadIdx.x / g, i = threadIdx.x - grp * g;
  const int lane = threadIdx.x & 31, warps = g >> 5;
  const int n = W / VEC;
  auto in = [&](int k) { return kFull || i + k * g < n; };   // kFull: n = NV g
  const float inv = 1.f / static_cast<float>(H);
  const PackRing<X, VEC> x_ring(ring_bytes, blockDim.x, threadIdx.x);
  const PackRing<D, VEC> g_ring(ring_bytes + kDepth * NV * sizeof(X) * VEC * blockDim.x, blockDim.x,
                                threadIdx.x);
  // pairs of columns: within a pack, or of neighbouring packs of one element
  constexpr int kPairs = NV * VEC / 2;
  float2 aw[kPairs] = {}, ab[kPairs] = {}, wv[kPairs];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float one[VEC] = {};
    if (in(k)) load_params<VEC>(w, param_type, c_first + (i + k * g) * VEC, one);
#pragma unroll
    for (int e = 0; e < VEC; ++e) at(wv, k * VEC + e) = one[e];
  }
  Pack<X, VEC> xn[kRegs];
  Pack<D, VEC> gn[kRegs];
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * groups + grp, next = t;
  int put = 0, get = 0;
  float mn = 0.f, rn = 0.f;
  auto fetch = [&] {
    if (next < N) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!in(k)) continue;
        const X* xs = x + next * x_ld + (i + k * g) * VEC;
        const D* gs = dy + next * dy_ld + (i + k * g) * VEC;
        if constexpr (kRing) {
          x_ring.fetch(put * NV + k, xs);
          g_ring.fetch(put * NV + k, gs);
        } else {
          xn[k] = *reinterpret_cast<const Pack<X, VEC>*>(xs);
          gn[k] = *reinterpret_cast<const Pack<D, VEC>*>(gs);
        }
      }
    }
    if constexpr (kRing) {
      copy_async_commit();
      put = put + 1 == kDepth ? 0 : put + 1;
    }
    next += step;
  };
#pragma unroll
  for (int d = 0; d < (kRing ? kDepth : 1); ++d) fetch();
  if (t < N) {
    mn = mean[t];
    rn = rstd[t];
  }
  for (int flip = 0; t < N; t += step, flip ^= 1) {
    if constexpr (kRing) copy_async_wait<kRing ? kDepth - 1 : 0>();
    float2 xv[kPairs], gv[kPairs];   // columns past H count as zeros in dy
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      Pack<X, VEC> xq;
      Pack<D, VEC> gq;
      if constexpr (kRing) {
        xq = x_ring.read(get * NV + k);
        gq = g_ring.read(get * NV + k);
      } else {
        xq = xn[k];
        gq = gn[k];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        at(xv, k * VEC + e) = in(k) ? to_f32(xq.v[e]) : 0.f;
        at(gv, k * VEC + e) = in(k) ? to_f32(gq.v[e]) : 0.f;
      }
    }
    if constexpr (kRing) get = get + 1 == kDepth ? 0 : get + 1;
    const float2 minus_mu = make_float2(-mn, -mn), r2 = make_float2(rn, rn);
    if constexpr (!kRing) fetch();
    if (t + step < N) {
      mn = mean[t + step];
      rn = rstd[t + step];
    }
    float2 s1 = make_float2(0.f, 0.f), s2 = s1;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const float2 xh = mul2(add2(xv[j], minus_mu), r2), h = mul2(gv[j], wv[j]);
      s1 = fma2(h, xh, s1);
      s2 = add2(s2, h);
      aw[j] = fma2(gv[j], xh, aw[j]);
      ab[j] = add2(ab[j], gv[j]);
    }
    // into the slots just read, whose values are in the sums; fp32 dy, the longer rows,
    // gain from asking first (16384 x 4096: 115 us against 124), 16-bit ones lose
    // (65536 x 2560: 180 against 170)
    if constexpr (kRing && sizeof(D) == 4) fetch();
    float half = sums ? 0.f : warp_sum_halves(s1.x + s1.y, s2.x + s2.y);
    if constexpr (kRing && sizeof(D) != 4) fetch();
    if (dx) {
      if (!sums && warps > 1) {
        const int w0 = grp * warps, wl = lane & 15;
        if (wl == 0) red[flip][lane >> 4][threadIdx.x >> 5] = half;
        named_bar_sync(1 + grp, g);
        half = wl < warps ? red[flip][lane >> 4][w0 + wl] : 0.f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) half += __shfl_xor_sync(0xffffffffu, half, o);
      }
      float2 c;
      if (sums)
        c = sums[t];
      else
        c = make_float2(__shfl_sync(0xffffffffu, half, 0) * inv, __shfl_sync(0xffffffffu, half, 16) * inv);
      const float2 minus_c1 = make_float2(-c.x, -c.x), minus_c2 = make_float2(-c.y, -c.y);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const float2 xh = mul2(add2(xv[j], minus_mu), r2), h = mul2(gv[j], wv[j]);
        gv[j] = mul2(fma2(xh, minus_c1, add2(h, minus_c2)), r2);
      }
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!in(k)) continue;
        Pack<X, VEC> o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o.v[e] = from_f32<X>(at(gv, k * VEC + e));
        *reinterpret_cast<Pack<X, VEC>*>(dx + t * dx_ld + (i + k * g) * VEC) = o;
      }
    }
  }
  if constexpr (kRing) copy_async_wait<0>();
  if (!part_w) return;
  // groups join in order, in the memory of the ring
  float* const joined = reinterpret_cast<float*>(ring_bytes);
  for (int q = 0; q < groups; ++q) {
    if (groups > 1) __syncthreads();
    if (grp != q) continue;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (in(k)) {
        const int c = (i + k * g) * VEC;
        constexpr int N = VEC < 4 ? VEC : 4;
        using Some = Pack<float, N>;
        float* const to_w = q + 1 < groups ? joined : part_w + static_cast<int64_t>(blockIdx.x) * H;
        float* const to_b = q + 1 < groups ? joined + W : part_b + static_cast<int64_t>(blockIdx.x) * H;
#pragma unroll
        for (int e = 0; e < VEC; e += N) {
          Some a, b;
          if (q > 0) {
            a = *reinterpret_cast<const Some*>(joined + c + e);
            b = *reinterpret_cast<const Some*>(joined + W + c + e);
          }
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float own_w = at(aw, k * VEC + e + j), own_b = at(ab, k * VEC + e + j);
            a.v[j] = q > 0 ? a.v[j] + own_w : own_w;
            b.v[j] = q > 0 ? b.v[j] + own_b : own_b;
          }
          *reinterpret_cast<Some*>(to_w + c + e) = a;
          *reinterpret_cast<Some*>(to_b + c + e) = b;
        }
      }
  }
}

// dx of wide rows without a workspace for their sums; dx may be x or dy.
template <typename X, typename D>
__global__ void __launch_bounds__(kRowThreads)
    norm_dx_any_kernel(const D* dy, int64_t dy_ld, const X* x,
                       int64_t x_ld, const void* __restrict__ w, int param_type,
                       const float* __restrict__ mean, const float* __restrict__ rstd, int64_t N,
                       int H, X* dx, int64_t dx_ld) {
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

// The two sums of a row's gradient, for rows wider than a CTA keeps:
// sums[t] = (mean(h xh), mean(h)).
template <typename X, typename D, int VEC>
__global__ void __launch_bounds__(kRowThreads)
    norm_sums_kernel(const D* __restrict__ dy, int64_t dy_ld, const X* __restrict__ x, int64_t x_ld,
                     const void* __restrict__ w, int param_type, const float* __restrict__ mean,
                     const float* __restrict__ rstd, int64_t N, int H, float2* __restrict__ sums) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float red[kRowThreads / 32];
  for (int64_t t = blockIdx.x; t < N; t += gridDim.x) {
    const X* xr = x + t * x_ld;
    const D* gr = dy + t * dy_ld;
    const float mu = mean[t], r = rstd[t];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < H / VEC; i += kRowThreads) {
      const Pack<X, VEC> xq = *reinterpret_cast<const Pack<X, VEC>*>(xr + i * VEC);
      const Pack<D, VEC> gq = *reinterpret_cast<const Pack<D, VEC>*>(gr + i * VEC);
      float wl[VEC];
      load_params<VEC>(w, param_type, i * VEC, wl);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float h = to_f32(gq.v[e]) * wl[e];
        s1 = fmaf(h, (to_f32(xq.v[e]) - mu) * r, s1);
        s2 += h;
      }
    }
    s1 = block_sum(s1, red);
    s2 = block_sum(s2, red);
    if (threadIdx.x == 0)
      sums[t] = make_float2(s1 / static_cast<float>(H), s2 / static_cast<float>(H));
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
  if (c < H) {
#pragma unroll 8
    for (int p = sub; p < P; p += kFinishRows) a += part[static_cast<int64_t>(p) * H + c];
  }
  red[sub][lane] = a;
  __syncthreads();
  if (sub == 0 && c < H) {
    for (int k = 1; k < kFinishRows; ++k) a += red[k][lane];
    out[c] = accumulate ? out[c] + a : a;
  }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int round32(int n) { return (n + 31) / 32 * 32; }

template <typename X, typename Y, int VEC, int NV, bool kPerWarp>
cudaError_t fwd_rows(const NormFwd& a, cudaStream_t s) {
  const int n = a.H / VEC;
  const int threads = kPerWarp ? 32 * kFwdWarpRows : round32((n + NV - 1) / NV);
  const int64_t grid = kPerWarp ? (a.N + kFwdWarpRows - 1) / kFwdWarpRows : a.N;
  return launch_dependent(norm_fwd_kernel<X, Y, VEC, NV, kPerWarp>,
                          dim3(static_cast<unsigned>(grid)), threads, 0, 1, s, static_cast<const X*>(a.x), a.x_ld, a.weight, a.bias,
                          a.param_type, a.N, a.H, a.eps, static_cast<Y*>(a.y), a.y_ld, a.mean,
                          a.rstd);
}

template <typename X, typename Y, int VEC, int NV, int kDepth>
cudaError_t fwd_stream(const NormFwd& a, cudaStream_t s) {
  static std::atomic<int> ready_full[64], ready_part[64];
  const int n = a.H / VEC;
  const bool full = n % (32 * NV) == 0;
  auto* kern = full ? norm_fwd_stream_kernel<X, Y, VEC, NV, kDepth, true>
                    : norm_fwd_stream_kernel<X, Y, VEC, NV, kDepth, false>;
  constexpr size_t kPerThread = static_cast<size_t>(kDepth) * NV * sizeof(X) * VEC;
  const cudaError_t e = allow_shared(full ? ready_full : ready_part,
                                     reinterpret_cast<const void*>(kern),
                                     kPerThread * kStreamThreads);
  if (e != cudaSuccess) return e;
  const int g = round32((n + NV - 1) / NV), groups = kStreamThreads / g;
  const int64_t ctas = (a.N + groups - 1) / groups, sms = sm_count();
  return launch_dependent(kern, dim3(static_cast<unsigned>(ctas < sms ? ctas : sms)), g * groups,
                          kPerThread * g * groups, 1, s, static_cast<const X*>(a.x), a.x_ld,
                          a.weight, a.bias, a.param_type, a.N, a.H, a.eps, static_cast<Y*>(a.y),
                          a.y_ld, a.mean, a.rstd, g);
}

template <typename X, typename Y>
cudaError_t fwd_typed(const NormFwd& a, cudaStream_t s) {
  constexpr int VEC = kVec<X>;
  const bool packs = a.H % VEC == 0 && a.x_ld % VEC == 0 && a.y_ld % VEC == 0 &&
                     aligned(a.x, 16) && aligned(a.y, sizeof(Y) * VEC) && aligned(a.weight, 16) &&
                     aligned(a.bias, 16);
  if (packs) {
    const int n = a.H / VEC;
    if (a.N >= 4ll * sm_count()) {   // enough rows to give every warp its own
      if (n <= 32 * 2) return fwd_rows<X, Y, VEC, 2, true>(a, s);
      if (n <= 32 * 4) return fwd_rows<X, Y, VEC, 4, true>(a, s);
      constexpr int NV = 16 / VEC;
      if (n <= kGroupThreads * NV) return fwd_stream<X, Y, VEC, NV, NV == 2 ? 4 : 3>(a, s);
    }
    if (n <= kFwdMaxThreads) return fwd_rows<X, Y, VEC, 1, false>(a, s);
    if (n <= 4 * kFwdMaxThreads) return fwd_rows<X, Y, VEC, 4, false>(a, s);
  }
  if (a.N >= 4ll * sm_count() && a.H <= kGroupThreads * 8)
    return fwd_stream<X, Y, 1, 8, sizeof(X) == 4 ? 4 : 0>(a, s);
  if (a.H <= kFwdMaxThreads) return fwd_rows<X, Y, 1, 4, false>(a, s);
  if (a.H <= 8 * kFwdMaxThreads) return fwd_rows<X, Y, 1, 8, false>(a, s);
  const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
  const int grid = static_cast<int>(a.N < cap ? a.N : cap);
  return launch_dependent(norm_fwd_any_kernel<X, Y>, dim3(grid), kRowThreads, 0, 1, s,
                          static_cast<const X*>(a.x), a.x_ld, a.weight, a.bias, a.param_type, a.N,
                          a.H, a.eps, static_cast<Y*>(a.y), a.y_ld, a.mean, a.rstd);
}

cudaError_t finish(const NormBwd& a, int P, cudaStream_t s) {
  return launch_dependent(norm_finish_kernel, dim3((a.H + 31) / 32, 2), 32 * kFinishRows, 0, 1, s,
                          static_cast<const float*>(a.partials),
                          static_cast<const float*>(a.partials + static_cast<int64_t>(P) * a.H), P,
                          a.H, a.d_weight, a.d_bias, a.accumulate);
}

template <typename X, typename D, int VEC, int NV>
cudaError_t bwd_rows(const NormBwd& a, cudaStream_t s) {
  constexpr bool kRing = PackRing<X, VEC>::kAsync && PackRing<D, VEC>::kAsync;
  constexpr size_t kRow = NV * VEC * (sizeof(X) + sizeof(D));   // a thread's bytes of one row
  constexpr int kDepth = !kRing ? 0 : kRow <= 96 ? 4 : 3;
  constexpr int kCols = kBwdThreads * VEC * NV;
  const int sms = std::min(sm_count(), kNormPartials);
  const int blocks = (a.H + kCols - 1) / kCols;
  const int n = ((a.H + blocks - 1) / blocks + VEC - 1) / VEC;   // packs of a block
  const bool params = a.d_weight || a.d_bias;
  if (blocks > 1 && a.dx) {
    const int64_t cap = static_cast<int64_t>(sms) * 8;
    const cudaError_t e = launch_dependent(
        norm_sums_kernel<X, D, VEC>, dim3(static_cast<unsigned>(a.N < cap ? a.N : cap)), kRowThreads,
        0, 1, s, static_cast<const D*>(a.dy), a.dy_ld, static_cast<const X*>(a.x), a.x_ld, a.weight,
        a.param_type, a.mean, a.rstd, a.N, a.H, a.sums);
    if (e != cudaSuccess) return e;
  }
  const bool full = blocks == 1 && n % (32 * NV) == 0;
  const int g = round32((n + NV - 1) / NV);
  const int64_t most = sms / blocks > 1 ? sms / blocks : 1;   // CTAs per block of columns
  int groups = kBwdThreads / g;
  const int64_t per_cta = (a.N + most - 1) / most;
  if (groups > per_cta) groups = static_cast<int>(per_cta);
  const int64_t ctas = (a.N + groups - 1) / groups;
  const int P = static_cast<int>(ctas < most ? ctas : most);
  static std::atomic<int> ready_full[64], ready_part[64];
  auto* kern = full ? norm_bwd_kernel<X, D, VEC, NV, kDepth, true>
                    : norm_bwd_kernel<X, D, VEC, NV, kDepth, false>;
  constexpr size_t kMostRing = kDepth * kRow * kBwdThreads;
  constexpr size_t kMostJoin = 2 * sizeof(float) * kBwdThreads / 2 * VEC * NV;   // two groups or more
  cudaError_t e = allow_shared(full ? ready_full : ready_part, reinterpret_cast<const void*>(kern),
                               kMostRing > kMostJoin ? kMostRing : kMostJoin);
  if (e != cudaSuccess) return e;
  const size_t ring = kDepth * kRow * g * groups;
  const size_t join = groups > 1 && params ? 2 * sizeof(float) * static_cast<size_t>(n) * VEC : 0;
  float* part_w = params ? a.partials : nullptr;
  float* part_b = params ? a.partials + static_cast<int64_t>(P) * a.H : nullptr;
  e = launch_dependent(kern, dim3(P, blocks), g * groups, ring > join ? ring : join, 1, s,
                       static_cast<const D*>(a.dy), a.dy_ld, static_cast<const X*>(a.x), a.x_ld,
                       a.weight, a.param_type, a.mean, a.rstd, a.N, a.H, n * VEC,
                       static_cast<const float2*>(blocks > 1 ? a.sums : nullptr),
                       static_cast<X*>(a.dx), a.dx_ld, part_w, part_b, g);
  if (e != cudaSuccess || !params) return e;
  return finish(a, P, s);
}

template <typename X, typename D>
cudaError_t bwd_typed(const NormBwd& a, cudaStream_t s) {
  constexpr int VEC = kVec<X>;
  if (!a.sums && a.H > kNormWide) {   // dx alone, without a workspace for a wide row's sums
    const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
    return launch_dependent(norm_dx_any_kernel<X, D>, dim3(static_cast<unsigned>(a.N < cap ? a.N : cap)),
                            kRowThreads, 0, 1, s, static_cast<const D*>(a.dy), a.dy_ld,
                            static_cast<const X*>(a.x), a.x_ld, a.weight, a.param_type, a.mean,
                            a.rstd, a.N, a.H, static_cast<X*>(a.dx), a.dx_ld);
  }
  const bool packs = a.H % VEC == 0 && a.x_ld % VEC == 0 && a.dy_ld % VEC == 0 &&
                     a.dx_ld % VEC == 0 && aligned(a.x, 16) && aligned(a.dx, 16) &&
                     aligned(a.dy, sizeof(D) * VEC > 16 ? 16 : sizeof(D) * VEC) &&
                     aligned(a.weight, 16);
  return packs ? bwd_rows<X, D, VEC, 16 / VEC>(a, s) : bwd_rows<X, D, 1, 8>(a, s);
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
