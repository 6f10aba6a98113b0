// Low-rank adapters of many requests beside a shared projection, whose result
// `base` the caller holds.  Row t with adapter a (factors D [rank, H] and
// U [rank, V], both with the long side contiguous) gets
//   y_t = base_t + u_t U_a,          u_t = s_a x_t D_a^T
// and backwards, for the cotangent g of y,
//   du_t = s_a g_t U_a^T,   dx_t = du_t D_a,
//   dU_a = sum_t u_t^T g_t, dD_a = sum_t du_t^T x_t.
// With a rank of some tens the work is HBM-bound: the [T, V] matrices are read and
// written once (g twice, by two products), the rest is small.  Three products,
// each used with either factor:
//  narrow_kernel  u = wide F^T: long sums over the wide side, split over CTAs and
//                 over the warps of a CTA, joined in a fixed order (join_kernel);
//  widen_kernel   y = base + u F;
//  outer_kernel   dF_a = sum_t u_t^T wide_t.
// Rows are first sorted by adapter (sort_ids.cu) and cut into items of up to kRows
// rows of one adapter (plan_kernel), so requests with the same adapter share its
// factors, whatever their order.  Rows without an adapter come last.
// Matrix instructions take bf16 (mma.sync: at these ranks tensor throughput is not
// the bound, and fragments go straight to and from rows that lie apart).  Values
// with more bits -- u, fp32 and fp16 cotangents -- enter as sums of up to three
// bf16 parts, which together hold the 24 bits of fp32; products of parts whose
// result lies below 2^-24 of the whole are left out.  16-bit results take two
// parts of u (2^-17 of the adapter's share, against their own 2^-9 or 2^-12).
#include "element.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace lmh {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kRows = 64;        // of an item
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 256;      // columns of the wide side per CTA (widen, outer)
constexpr int kPad = 8;          // elements between rows in shared memory: no bank conflicts
constexpr int kParts = 3;        // bf16 parts of u
constexpr int kOuterRows = 32;   // rows of a step of outer_kernel

__host__ __device__ constexpr int round_rank(int r) { return (r + 15) / 16 * 16; }

// bf16 parts that hold every bit of a T.
template <typename T>
constexpr int kPartsOf = sizeof(T) == 4 ? 3 : 1;
template <>
constexpr int kPartsOf<__half> = 2;

struct Item {
  int adapter;     // n: rows without one
  int first;       // sorted place of its first row
  int count;
  int pad;
};

struct Plan {
  int* live;         // rows with an adapter
  int* n_items;
  int32_t* keys;     // [rows] adapters in order
  int32_t* pos;      // [rows] their rows
  int* starts;       // [n + 2] first sorted place of each adapter, of the rows without, and the end
  Item* items;
  int most;          // items at most
  int rows;
  int n;
};

// ------------------------------------------------------------------ matrix instructions
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(p)) : "memory");
}
__device__ __forceinline__ void load_matrices_turned(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(p)) : "memory");
}

// x = sum of its parts; the remainder of each rounding is exact.
template <int N>
__device__ __forceinline__ void split(float x, float (&part)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    part[i] = __bfloat162float(__float2bfloat16_rn(x));
    x -= part[i];
  }
  // an infinity or NaN is in the first part alone
  if (!isfinite(part[0])) {
#pragma unroll
    for (int i = 1; i < N; ++i) part[i] = 0.f;
  }
}

// Eight elements as bf16 pairs, part by part.
template <typename T>
__device__ __forceinline__ void to_parts(const Pack<T, 8>& q, uint4 (&part)[kPartsOf<T>]) {
  if constexpr (kPartsOf<T> == 1) {
    part[0] = *reinterpret_cast<const uint4*>(&q);
  } else {
    constexpr int N = kPartsOf<T>;
    uint32_t w[N][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = pair_of(q, e);
      float lo[N], hi[N];
      split(x.x, lo);
      split(x.y, hi);
#pragma unroll
      for (int i = 0; i < N; ++i) w[i][e] = pack_bf16x2(lo[i], hi[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) part[i] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
  }
}

// Elements [c, c + 8) of a row of `width`, zero behind its end; c >= 0.
template <typename T>
__device__ __forceinline__ Pack<T, 8> load8(const T* row, int c, int width) {
  Pack<T, 8> q;
  const T* const p = row + c;
  if (c + 8 <= width && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<uint4*>(&q)[0] = reinterpret_cast<const uint4*>(p)[0];
      reinterpret_cast<uint4*>(&q)[1] = reinterpret_cast<const uint4*>(p)[1];
    } else {
      *reinterpret_cast<uint4*>(&q) = *reinterpret_cast<const uint4*>(p);
    }
    return q;
  }
  if constexpr (sizeof(T) == 2) {
    if (c >= 8 && c + 16 <= width) {     // both blocks lie inside the row
      *reinterpret_cast<uint4*>(&q) = load_across(p);
      return q;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) q.v[e] = c + e < width ? p[e] : from_f32<T>(0.f);
  return q;
}

// ------------------------------------------------------------------ items
__global__ void __launch_bounds__(1024) plan_kernel(Plan p) {
  __shared__ int sums[32], total;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int g = tid; g <= p.rows; g += 1024) {
    const int before = g == 0 ? -1 : p.keys[g - 1], here = g == p.rows ? p.n + 1 : p.keys[g];
    for (int a = before + 1; a <= here; ++a) p.starts[a] = g;
  }
  if (tid == 0) total = 0;
  __syncthreads();
  for (int a0 = 0; a0 <= p.n; a0 += 1024) {
    const int a = a0 + tid;
    const int first = a <= p.n ? p.starts[a] : 0, count = a <= p.n ? p.starts[a + 1] - first : 0;
    const int mine = (count + kRows - 1) / kRows;
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    int at = total + scan - mine;
    for (int w = 0; w < warp; ++w) at += sums[w];
    for (int i = 0; i < mine; ++i)
      p.items[at + i] = Item{a, first + i * kRows, min(kRows, count - i * kRows), 0};
    __syncthreads();
    if (tid == 1023) total = at + mine;
    __syncthreads();
  }
  if (tid == 0) *p.n_items = total;
}

// ------------------------------------------------------------------ u = wide F^T
// Grid (items, splits of the wide side, blocks of 8 NT ranks).  A warp holds 32 rows;
// a thread reads 8 consecutive elements of its rows and of its ranks, so fragments
// need no shared memory: any order of the summed index serves, if it is the same on
// both sides.
template <typename X, int NT>
__global__ void __launch_bounds__(kThreads) narrow_kernel(const X* wide, int64_t ld, const bf16* factor, int width,
                                                          int rank, Plan p, float* part, int per_split) {
  constexpr int N = kPartsOf<X>;
  constexpr int kUnroll = N > 1 || NT > 4 ? 1 : 2;
  extern __shared__ float sums[];      // [warps][32][8 NT + 1]
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= *p.n_items) return;
  const Item it = p.items[blockIdx.x];
  if (it.adapter >= p.n) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int halves = it.count > 32 ? 2 : 1, slices = kWarps / halves, half = warp % halves, slice = warp / halves;
  const int rank0 = blockIdx.z * 8 * NT;
  const X* row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int local = half * 32 + i * 8 + g;
    row[i] = local < it.count ? wide + p.pos[it.first + local] * ld : nullptr;
  }
  const bf16* f[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    f[j] = rank0 + 8 * j + g < rank
               ? factor + (static_cast<int64_t>(it.adapter) * rank + rank0 + 8 * j + g) * width : nullptr;
  float acc[2][NT][4] = {};
  const int end = static_cast<int>(min(static_cast<int64_t>(blockIdx.y + 1) * per_split, static_cast<int64_t>(width)));
  for (int c0 = blockIdx.y * per_split + slice * 32 * kUnroll; c0 < end; c0 += slices * 32 * kUnroll) {
    Pack<X, 8> q[kUnroll][4];
    uint4 b[kUnroll][NT];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int c = c0 + u * 32 + t * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (row[i] && c < end)
          q[u][i] = load8(row[i], c, end);
        else
          q[u][i] = Pack<X, 8>{};
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        b[u][j] = make_uint4(0u, 0u, 0u, 0u);
        if (f[j] && c < end) {
          const Pack<bf16, 8> v = load8(f[j], c, width);
          b[u][j] = *reinterpret_cast<const uint4*>(&v);
        }
      }
    }
    // the sum of each stretch starts from zero, so that its small terms are not cut to
    // the last bit of a long sum
    float sum[2][NT][4] = {};
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      uint4 a[4][N];
#pragma unroll
      for (int i = 0; i < 4; ++i) to_parts(q[u][i], a[i]);
#pragma unroll
      for (int s = N - 1; s >= 0; --s)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint4 lo = a[2 * m][s], hi = a[2 * m + 1][s];
          const uint32_t first[4] = {lo.x, hi.x, lo.y, hi.y}, second[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma(sum[m][j], first, b[u][j].x, b[u][j].y);
            mma(sum[m][j], second, b[u][j].z, b[u][j].w);
          }
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][j][e] += sum[m][j][e];
  }
  constexpr int kStride = 8 * NT + 1;
  float* const own = sums + warp * 32 * kStride;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        own[(m * 16 + (e >> 1) * 8 + g) * kStride + 8 * j + 2 * t + (e & 1)] = acc[m][j][e];
  __syncthreads();
  const int wide_rank = round_rank(rank);
  for (int i = threadIdx.x; i < it.count * 8 * NT; i += kThreads) {
    const int local = i / (8 * NT), c = i % (8 * NT);
    if (rank0 + c >= rank) continue;
    float s = 0.f;
    for (int k = 0; k < slices; ++k)
      s += sums[((k * halves + local / 32) * 32 + local % 32) * kStride + c];
    part[(static_cast<int64_t>(blockIdx.y) * p.rows + it.first + local) * wide_rank + rank0 + c] = s;
  }
}

// u = scale * the sum of its splits, as bf16 parts [rows][kParts][round_rank(rank)].
__global__ void __launch_bounds__(kThreads) join_kernel(Plan p, const float* part, int splits, const float* scale,
                                                        int rank, bf16* u) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int wide_rank = round_rank(rank);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = i / wide_rank;
  const int c = static_cast<int>(i % wide_rank);
  if (row >= *p.live) return;
  float s = 0.f;
  if (c < rank) {
#pragma unroll 4
    for (int k = 0; k < splits; ++k) s += part[(static_cast<int64_t>(k) * p.rows + row) * wide_rank + c];
    if (scale) s *= scale[p.keys[row]];
  }
  float parts[kParts];
  split(s, parts);
#pragma unroll
  for (int k = 0; k < kParts; ++k) u[(row * kParts + k) * wide_rank + c] = __float2bfloat16_rn(parts[k]);
}

// ------------------------------------------------------------------ y = base + u F
// Shared memory: F's block [wide_rank][kBlock + kPad], u [parts][kRows][wide_rank + kPad],
// both bf16, and the share of 16 rows [16][kBlock + 4] in fp32.
size_t widen_shared(int wide_rank, int parts) {
  return 2 * (static_cast<size_t>(wide_rank) * (kBlock + kPad) + static_cast<size_t>(parts) * kRows * (wide_rank + kPad)) +
         4 * 16 * (kBlock + 4);
}

// CTA = (block of columns, item), items of one block next to each other: they share F.
template <typename Y, int VEC>
__global__ void __launch_bounds__(kThreads) widen_kernel(const Y* base, int64_t base_ld, Y* out, int64_t out_ld,
                                                         const bf16* factor, int width, int rank, const bf16* u,
                                                         int parts, Plan p, bool factor_wide) {
  constexpr int kEach = 16 * kBlock / kThreads / VEC;      // packs of 16 rows per thread
  extern __shared__ __align__(16) char shared[];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int item = blockIdx.x % p.most;
  if (item >= *p.n_items) return;
  const Item it = p.items[item];
  const bool bare = it.adapter >= p.n;
  if (bare && base == out) return;
  const int wide_rank = round_rank(rank), fs = kBlock + kPad, us = wide_rank + kPad;
  bf16* const F = reinterpret_cast<bf16*>(shared);
  bf16* const U = F + wide_rank * fs;
  float* const share = reinterpret_cast<float*>(U + parts * kRows * us);
  const int c0 = blockIdx.x / p.most * kBlock;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int my_row = tid / 16, my_col = tid % 16 * VEC;
  Pack<Y, VEC> q[kEach];
  auto fetch = [&](int r0) {
    if (r0 + my_row >= it.count) return;
    const Y* const src = base ? base + p.pos[it.first + r0 + my_row] * base_ld : nullptr;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int c = c0 + my_col + i * 16 * VEC;
      if (!src)
        q[i] = Pack<Y, VEC>{};
      else if (c + VEC <= width)
        q[i] = *reinterpret_cast<const Pack<Y, VEC>*>(src + c);
      else
        for (int e = 0; e < VEC; ++e)
          if (c + e < width) q[i].v[e] = src[c + e];
    }
  };
  fetch(0);
  if (!bare) {
    const bf16* const f = factor + static_cast<int64_t>(it.adapter) * rank * width;
    if (factor_wide) {
      for (int i = tid; i < wide_rank * (kBlock / 8); i += kThreads) {
        const int k = i / (kBlock / 8), c = i % (kBlock / 8) * 8;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (k < rank && c0 + c < width) v = *reinterpret_cast<const uint4*>(f + static_cast<int64_t>(k) * width + c0 + c);
        *reinterpret_cast<uint4*>(F + k * fs + c) = v;
      }
    } else {
      for (int i = tid; i < wide_rank * kBlock; i += kThreads) {
        const int k = i / kBlock, c = i % kBlock;
        F[k * fs + c] = k < rank && c0 + c < width ? f[static_cast<int64_t>(k) * width + c0 + c] : __float2bfloat16_rn(0.f);
      }
    }
    const int packs = wide_rank / 8;
    for (int i = tid; i < parts * kRows * packs; i += kThreads) {
      const int k = i / (kRows * packs), r = i / packs % kRows, c = i % packs * 8;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r < it.count)
        v = *reinterpret_cast<const uint4*>(u + (static_cast<int64_t>(it.first + r) * kParts + k) * wide_rank + c);
      *reinterpret_cast<uint4*>(U + (k * kRows + r) * us + c) = v;
    }
  }
  __syncthreads();
  for (int r0 = 0; r0 < it.count; r0 += 16) {
    if (!bare) {
      float acc[4][4] = {};
      for (int k = 0; k < wide_rank; k += 16) {
        uint32_t b[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          load_matrices_turned(b[h], F + (k + (lane >> 3 & 1) * 8 + (lane & 7)) * fs + warp * 32 + h * 16 + (lane >> 4) * 8);
        for (int s = parts - 1; s >= 0; --s) {
          uint32_t a[4];
          load_matrices(a, U + (s * kRows + r0 + (lane >> 3 & 1) * 8 + (lane & 7)) * us + k + (lane >> 4) * 8);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma(acc[j], a, b[j >> 1][(j & 1) * 2], b[j >> 1][(j & 1) * 2 + 1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(share + (h * 8 + g) * (kBlock + 4) + warp * 32 + j * 8 + 2 * t) =
              make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
    }
    __syncthreads();
    if (r0 + my_row < it.count) {
      Y* const dst = out + p.pos[it.first + r0 + my_row] * out_ld;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int at = my_col + i * 16 * VEC, c = c0 + at;
        if (!bare) {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            q[i].v[e] = from_f32<Y>(to_f32(q[i].v[e]) + share[my_row * (kBlock + 4) + at + e]);
        }
        if (c + VEC <= width)
          *reinterpret_cast<Pack<Y, VEC>*>(dst + c) = q[i];
        else
          for (int e = 0; e < VEC; ++e)
            if (c + e < width) dst[c + e] = q[i].v[e];
      }
    }
    fetch(r0 + 16);
    __syncthreads();
  }
}

// ------------------------------------------------------------------ dF = sum u^T wide
// CTA = (block of columns, adapter, block of 16 RT ranks).  Steps of kOuterRows rows;
// the next step's rows are fetched while the matrix instructions run.
template <typename X, int RT>
constexpr size_t outer_shared() {
  return 2 * (static_cast<size_t>(kPartsOf<X>) * kOuterRows * (kBlock + kPad) +
              static_cast<size_t>(kParts) * kOuterRows * (16 * RT + kPad));
}

template <typename X, int RT>
__global__ void __launch_bounds__(kThreads) outer_kernel(const X* wide, int64_t ld, int width, int rank, const bf16* u,
                                                         Plan p, float* grad, int accumulate) {
  constexpr int N = kPartsOf<X>, fs = kBlock + kPad, us = 16 * RT + kPad, kRowsEach = kOuterRows / kWarps;
  constexpr int kPacks = (kOuterRows * kParts * RT * 2 + kThreads - 1) / kThreads;   // of u per thread
  extern __shared__ __align__(16) char shared[];
  bf16* const W = reinterpret_cast<bf16*>(shared);     // [N][kOuterRows][fs]
  bf16* const U = W + N * kOuterRows * fs;             // [kParts][kOuterRows][us]
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int c0 = blockIdx.x * kBlock, adapter = blockIdx.y, rank0 = blockIdx.z * 16 * RT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int from = p.starts[adapter], to = p.starts[adapter + 1], wide_rank = round_rank(rank);
  Pack<X, 8> q[kRowsEach];
  uint4 uq[kPacks];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
      const int r = r0 + i * kWarps + warp, c = c0 + lane * 8;
      q[i] = Pack<X, 8>{};
      if (r < to && c < width) q[i] = load8(wide + p.pos[r] * ld, c, width);
    }
#pragma unroll
    for (int i = 0; i < kPacks; ++i) {
      const int at = i * kThreads + tid, k = at / (kOuterRows * RT * 2), r = at / (RT * 2) % kOuterRows,
                c = rank0 + at % (RT * 2) * 8;
      uq[i] = make_uint4(0u, 0u, 0u, 0u);
      if (k < kParts && r0 + r < to && c < wide_rank)
        uq[i] = *reinterpret_cast<const uint4*>(u + (static_cast<int64_t>(r0 + r) * kParts + k) * wide_rank + c);
    }
  };
  float acc[RT][4][4] = {};
  fetch(from);
  for (int r0 = from; r0 < to; r0 += kOuterRows) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
      uint4 part[N];
      to_parts(q[i], part);
#pragma unroll
      for (int s = 0; s < N; ++s)
        *reinterpret_cast<uint4*>(W + (s * kOuterRows + i * kWarps + warp) * fs + lane * 8) = part[s];
    }
#pragma unroll
    for (int i = 0; i < kPacks; ++i) {
      const int at = i * kThreads + tid, k = at / (kOuterRows * RT * 2), r = at / (RT * 2) % kOuterRows,
                c = at % (RT * 2) * 8;
      if (k < kParts) *reinterpret_cast<uint4*>(U + (k * kOuterRows + r) * us + c) = uq[i];
    }
    __syncthreads();
    fetch(r0 + kOuterRows);
    float sum[RT][4][4] = {};
#pragma unroll
    for (int k = 0; k < kOuterRows; k += 16) {
      uint32_t b[N][2][4];
#pragma unroll
      for (int s = 0; s < N; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          load_matrices_turned(b[s][h], W + (s * kOuterRows + k + (lane >> 3 & 1) * 8 + (lane & 7)) * fs + warp * 32 +
                                            h * 16 + (lane >> 4) * 8);
#pragma unroll
      for (int v = kParts - 1; v >= 0; --v)
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          uint32_t a[4];
          load_matrices_turned(a, U + (v * kOuterRows + k + (lane >> 4) * 8 + (lane & 7)) * us + m * 16 +
                                      (lane >> 3 & 1) * 8);
#pragma unroll
          for (int s = N - 1; s >= 0; --s)
            if (s + v < kParts) {
#pragma unroll
              for (int j = 0; j < 4; ++j) mma(sum[m][j], a, b[s][j >> 1][(j & 1) * 2], b[s][j >> 1][(j & 1) * 2 + 1]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][j][e] += sum[m][j][e];
  }
  if (accumulate && from == to) return;
#pragma unroll
  for (int m = 0; m < RT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = rank0 + m * 16 + h * 8 + g;
      if (r >= rank) continue;
      float* const dst = grad + (static_cast<int64_t>(adapter) * rank + r) * width;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = c0 + warp * 32 + j * 8 + 2 * t + e;
          if (c < width) dst[c] = accumulate ? dst[c] + acc[m][j][2 * h + e] : acc[m][j][2 * h + e];
        }
    }
}

// ------------------------------------------------------------------ host
size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

template <typename F>
auto by_type(int type, F&& f) {
  switch (type) {
    case kF32: return f(float{});
    case kBF16: return f(bf16{});
    default: return f(__half{});
  }
}

int64_t most_items(int64_t rows, int n) { return rows / kRows + (n + 1 < rows ? n + 1 : rows) + 1; }

// Splits of the wide side: CTAs enough for the GPU, at least 1,024 columns each.
int splits_of(int64_t rows, int width, int& per_split) {
  const int64_t items = (rows + kRows - 1) / kRows;
  int64_t splits = (608 + items - 1) / items;
  const int64_t most = (width + 1023) / 1024;
  if (splits > most) splits = most;
  per_split = static_cast<int>(((width + splits - 1) / splits + 255) / 256 * 256);
  return (width - 1) / per_split + 1;
}

struct Space {
  Plan plan;
  bf16 *u, *du;
  float* part;
  size_t bytes;
};

Space lay_out(void* workspace, int64_t T, int H, int V, int rank, int n) {
  const int64_t rows = T < kSortMost ? T : kSortMost;
  char* p = static_cast<char*>(workspace);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* const q = p + at;
    at += round_up(bytes);
    return q;
  };
  Space s{};
  s.plan.live = reinterpret_cast<int*>(take(256));
  s.plan.n_items = s.plan.live + 1;
  s.plan.keys = reinterpret_cast<int32_t*>(take(4 * static_cast<size_t>(rows)));
  s.plan.pos = reinterpret_cast<int32_t*>(take(4 * static_cast<size_t>(rows)));
  s.plan.starts = reinterpret_cast<int*>(take(4 * (static_cast<size_t>(n) + 2)));
  s.plan.most = static_cast<int>(most_items(rows, n));
  s.plan.items = reinterpret_cast<Item*>(take(sizeof(Item) * static_cast<size_t>(s.plan.most)));
  s.plan.n = n;
  const size_t wide_rank = static_cast<size_t>(round_rank(rank));
  s.u = reinterpret_cast<bf16*>(take(2 * kParts * wide_rank * rows));
  s.du = reinterpret_cast<bf16*>(take(2 * kParts * wide_rank * rows));
  int per;
  const int a = splits_of(rows > 0 ? rows : 1, H, per), b = splits_of(rows > 0 ? rows : 1, V, per);
  s.part = reinterpret_cast<float*>(take(4 * wide_rank * rows * static_cast<size_t>(a > b ? a : b)));
  // (a last part of fewer rows has more splits, of at most 64 * (608 + 607) rows in all)
  s.bytes = at;
  return s;
}

template <typename X, int NT>
cudaError_t narrow_of(const X* wide, int64_t ld, const bf16* factor, int width, int rank, const Plan& p, float* part,
                      int splits, int per_split, cudaStream_t s) {
  static std::atomic<int> ready[64];
  constexpr size_t smem = 4 * kWarps * 32 * (8 * NT + 1);
  const cudaError_t e = allow_shared(ready, reinterpret_cast<const void*>(narrow_kernel<X, NT>), smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(narrow_kernel<X, NT>, dim3(p.most, splits, (rank + 8 * NT - 1) / (8 * NT)), kThreads, smem, 1,
                          s, wide, ld, factor, width, rank, p, part, per_split);
}

// u (as parts) of every row with an adapter.
template <typename X>
cudaError_t narrow(const char* name, const X* wide, int64_t ld, const void* factor, int width, const Adapters& a,
                   const Space& z, bf16* u, cudaStream_t s) {
  int per_split;
  const int splits = splits_of(z.plan.rows, width, per_split);
  const bf16* const f = static_cast<const bf16*>(factor);
  cudaError_t e = traced_launch(name, s, [&] {
    if (a.rank <= 8) return narrow_of<X, 1>(wide, ld, f, width, a.rank, z.plan, z.part, splits, per_split, s);
    if (a.rank <= 16) return narrow_of<X, 2>(wide, ld, f, width, a.rank, z.plan, z.part, splits, per_split, s);
    if (a.rank <= 32) return narrow_of<X, 4>(wide, ld, f, width, a.rank, z.plan, z.part, splits, per_split, s);
    return narrow_of<X, 8>(wide, ld, f, width, a.rank, z.plan, z.part, splits, per_split, s);
  });
  if (e != cudaSuccess) return e;
  const int64_t n = static_cast<int64_t>(z.plan.rows) * round_rank(a.rank);
  return traced_launch("adapters_join", s, [&] {
    return launch_dependent(join_kernel, dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), kThreads, 0, 1, s,
                            z.plan, z.part, splits, a.scale, a.rank, u);
  });
}

template <typename Y, int VEC>
cudaError_t widen_of(const Y* base, int64_t base_ld, Y* out, int64_t out_ld, const bf16* factor, int width, int rank,
                     const bf16* u, int parts, const Plan& p, cudaStream_t s) {
  static std::atomic<int> ready[64];
  const cudaError_t e = allow_shared(ready, reinterpret_cast<const void*>(widen_kernel<Y, VEC>),
                                     widen_shared(round_rank(kMaxRank), kParts));
  if (e != cudaSuccess) return e;
  const int64_t blocks = (static_cast<int64_t>(width) + kBlock - 1) / kBlock;
  const bool factor_wide = reinterpret_cast<uintptr_t>(factor) % 16 == 0 && width % 8 == 0;
  return launch_dependent(widen_kernel<Y, VEC>, dim3(static_cast<unsigned>(blocks * p.most)), kThreads,
                          widen_shared(round_rank(rank), parts), 1, s, base, base_ld, out, out_ld, factor, width, rank, u,
                          parts, p, factor_wide);
}

template <typename Y>
cudaError_t widen(const char* name, const Y* base, int64_t base_ld, Y* out, int64_t out_ld, const void* factor, int width,
                  int rank, const bf16* u, const Plan& p, cudaStream_t s) {
  constexpr int VEC = kVec<Y>;
  const bf16* const f = static_cast<const bf16*>(factor);
  const bool packs = ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0 &&
                     base_ld % VEC == 0 && out_ld % VEC == 0;
  const int parts = sizeof(Y) == 4 ? kParts : 2;
  return traced_launch(name, s, [&] {
    return packs ? widen_of<Y, VEC>(base, base_ld, out, out_ld, f, width, rank, u, parts, p, s)
                 : widen_of<Y, 1>(base, base_ld, out, out_ld, f, width, rank, u, parts, p, s);
  });
}

template <typename X, int RT>
cudaError_t outer_of(const X* wide, int64_t ld, int width, int rank, const bf16* u, const Plan& p, float* grad,
                     int accumulate, cudaStream_t s) {
  static std::atomic<int> ready[64];
  constexpr size_t smem = outer_shared<X, RT>();
  const cudaError_t e = allow_shared(ready, reinterpret_cast<const void*>(outer_kernel<X, RT>), smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(outer_kernel<X, RT>, dim3((width + kBlock - 1) / kBlock, p.n, (rank + 16 * RT - 1) / (16 * RT)),
                          kThreads, smem, 1, s, wide, ld, width, rank, u, p, grad, accumulate);
}

template <typename X>
cudaError_t outer(const char* name, const X* wide, int64_t ld, int width, int rank, const bf16* u, const Plan& p,
                  float* grad, int accumulate, cudaStream_t s) {
  return traced_launch(name, s, [&] {
    if (rank <= 16) return outer_of<X, 1>(wide, ld, width, rank, u, p, grad, accumulate, s);
    if (rank <= 32) return outer_of<X, 2>(wide, ld, width, rank, u, p, grad, accumulate, s);
    return outer_of<X, 4>(wide, ld, width, rank, u, p, grad, accumulate, s);
  });
}

cudaError_t plan_rows(const Adapters& a, int64_t first, Space& z, cudaStream_t s) {
  z.plan.rows = static_cast<int>(a.T - first < kSortMost ? a.T - first : kSortMost);
  z.plan.most = static_cast<int>(most_items(z.plan.rows, a.n));
  const cudaError_t e = traced_launch("adapters_sort", s, [&] {
    return launch_sort_ids(a.ids ? a.ids + first : nullptr, z.plan.rows, a.n, false, -1, z.plan.keys, z.plan.pos,
                           z.plan.live, s);
  });
  if (e != cudaSuccess) return e;
  return traced_launch("adapters_plan", s, [&] { return launch_dependent(plan_kernel, dim3(1), 1024, 0, 1, s, z.plan); });
}

}  // namespace

size_t adapters_workspace(int64_t T, int H, int V, int rank, int n) {
  return lay_out(nullptr, T, H, V, rank, n).bytes;
}

bool adapters_fit(int64_t T, int width, int n) {
  const int64_t rows = T < kSortMost ? T : kSortMost;
  const int64_t blocks = (static_cast<int64_t>(width) + kBlock - 1) / kBlock;
  return blocks * most_items(rows, n) <= 0x7fffffff;
}

cudaError_t launch_adapters_fwd(const AdaptersFwd& f, cudaStream_t s) {
  const Adapters& a = f.a;
  Space z = lay_out(a.workspace, a.T, a.H, a.V, a.rank, a.n);
  for (int64_t first = 0; first < a.T; first += kSortMost) {
    cudaError_t e = plan_rows(a, first, z, s);
    if (e != cudaSuccess) return e;
    e = narrow("adapters_narrow", static_cast<const bf16*>(a.x) + first * a.x_ld, a.x_ld, a.down, a.H, a, z, z.u, s);
    if (e != cudaSuccess) return e;
    e = by_type(f.type, [&](auto t) {
      using Y = decltype(t);
      return widen("adapters_widen", static_cast<const Y*>(f.base) + first * f.base_ld, f.base_ld,
                   static_cast<Y*>(f.out) + first * f.out_ld, f.out_ld, a.up, a.V, a.rank, z.u, z.plan, s);
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_adapters_bwd(const AdaptersBwd& b, cudaStream_t s) {
  const Adapters& a = b.a;
  Space z = lay_out(a.workspace, a.T, a.H, a.V, a.rank, a.n);
  int accumulate = b.accumulate;
  for (int64_t first = 0; first < a.T; first += kSortMost) {
    const bf16* const x = static_cast<const bf16*>(a.x) + first * a.x_ld;
    cudaError_t e = plan_rows(a, first, z, s);
    if (e != cudaSuccess) return e;
    if (b.d_up) {
      e = narrow("adapters_narrow", x, a.x_ld, a.down, a.H, a, z, z.u, s);
      if (e != cudaSuccess) return e;
    }
    e = by_type(b.type, [&](auto t) {
      using G = decltype(t);
      const G* const g = static_cast<const G*>(b.grad) + first * b.grad_ld;
      cudaError_t r = cudaSuccess;
      if (b.dx || b.d_down) r = narrow("adapters_narrow_grad", g, b.grad_ld, a.up, a.V, a, z, z.du, s);
      if (r == cudaSuccess && b.d_up)
        r = outer("adapters_d_up", g, b.grad_ld, a.V, a.rank, z.u, z.plan, b.d_up, accumulate, s);
      return r;
    });
    if (e == cudaSuccess && b.d_down)
      e = outer("adapters_d_down", x, a.x_ld, a.H, a.rank, z.du, z.plan, b.d_down, accumulate, s);
    if (e == cudaSuccess && b.dx) {
      float* const dx = b.dx + first * b.dx_ld;
      e = widen("adapters_dx", b.accumulate_dx ? static_cast<const float*>(dx) : nullptr, b.dx_ld, dx, b.dx_ld, a.down,
                a.H, a.rank, z.du, z.plan, s);
    }
    if (e != cudaSuccess) return e;
    accumulate = 1;   // what follows is added to the first part's sums
  }
  return cudaSuccess;
}

}  // namespace lmh
