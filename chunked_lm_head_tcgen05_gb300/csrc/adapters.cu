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
// Matrix instructions take bf16 (mma.sync: at these ranks tensor throughput does not
// bind the forward, and fragments go straight to and from rows that lie apart; the
// two products with a cotangent keep the tensor pipe 27% and 53% busy).  Values
// with more bits -- u, fp32 and fp16 cotangents -- enter as sums of up to three
// bf16 parts, which together hold the 24 bits of fp32; products of parts whose
// result lies below 2^-24 of the whole are left out.  16-bit results take two
// parts of u (2^-17 of the adapter's share, against their own 2^-9 or 2^-12).
#include <type_traits>

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
constexpr int kFewAtOnce = 4;    // rows of a run that few_kernel takes
constexpr int kFewMean = 8;      // rows per adapter on average, up to which it may multiply
constexpr int kFewAlone = 128;   // rows up to which nothing else is launched then
constexpr int kFewRuns = 3;      // its runs per item, up to which it multiplies more rows
constexpr int kOuterRows = 32;   // rows of a step of outer_kernel
constexpr int kManyCtas = 608;   // four per SM
constexpr int kFewCtas = 304;    // two

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
  int* counts;       // of items, of runs and, where `choose`, of items that widen_kernel takes
  int32_t* keys;     // [rows] adapters in order
  int32_t* pos;      // [rows] their rows
  int* starts;       // [n + 2] first sorted place of each adapter, of the rows without, and the end
  Item* items;       // up to kRows rows of one adapter each
  Item* runs;        // up to run_rows rows each
  int most;          // items at most
  int run_rows;
  int rows;
  int n;
  bool choose;       // few_kernel (all runs) or widen_kernel (all items), by their numbers
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

// The nearest bf16 number, the largest one for what lies above it (fp32 numbers from 3.396e38 on
// would become infinite).
__device__ __forceinline__ float nearest_bf16(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
  return __uint_as_float(static_cast<uint32_t>(r) << 16);
}

// x = sum of its parts; the remainder of each rounding is exact.
template <int N>
__device__ __forceinline__ void split(float x, float (&part)[N]) {
  part[0] = nearest_bf16(x);
  x -= part[0];
#pragma unroll
  for (int i = 1; i < N; ++i) {
    part[i] = __bfloat162float(__float2bfloat16_rn(x));
    x -= part[i];
  }
  // an infinity is in the second part, beside the largest number; a NaN in the first two
  if (N > 2 && !isfinite(part[1])) {
#pragma unroll
    for (int i = 2; i < N; ++i) part[i] = 0.f;
  }
}

// Elements [c, c + 8) of a row.  A thread that knows which of these fits all of its loads
// has several of them in flight: a choice per load would make each wait for the one before.
enum class At {
  kAligned,    // on a 16-byte boundary, inside the row
  kInside,     // anywhere, with 8 elements of the row on either side
  kEdge        // anywhere, zeros behind the row's end
};
template <At kAt, typename T>
__device__ __forceinline__ Pack<T, 8> load8(const T* row, int c, int width) {
  Pack<T, 8> q;
  const T* const p = row + c;
  if constexpr (kAt == At::kAligned) {
#pragma unroll
    for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h)
      reinterpret_cast<uint4*>(&q)[h] = reinterpret_cast<const uint4*>(p)[h];
  } else if constexpr (kAt == At::kInside && sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(&q) = load_across(p);
  } else if constexpr (kAt == At::kInside) {
#pragma unroll
    for (int e = 0; e < 8; ++e) q.v[e] = p[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) q.v[e] = c + e < width ? p[e] : from_f32<T>(0.f);
  }
  return q;
}

// f(std::integral_constant<At, ...>) for loads of columns [c, c + 8).
template <typename F>
__device__ __forceinline__ void at_columns(bool aligned, int c, int width, F&& f) {
  if (aligned)
    f(std::integral_constant<At, At::kAligned>{});
  else if (c >= 8 && c + 16 <= width)
    f(std::integral_constant<At, At::kInside>{});
  else
    f(std::integral_constant<At, At::kEdge>{});
}

// ------------------------------------------------------------------ items
constexpr int kSmallRows = 1024, kSmallKeys = 512;

// kSmall: up to kSmallRows rows of fewer than kSmallKeys - 1 adapters, sorted here in one pass
// of sort_ids.cu's kind, whose digit is the adapter: a launch less.
template <bool kSmall>
__global__ void __launch_bounds__(1024) plan_kernel(Plan p, const int32_t* ids) {
  __shared__ int sums[2][32], total[2];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if constexpr (kSmall) {
    __shared__ uint16_t counts[32][kSmallKeys];
    __shared__ int base[kSmallKeys];
    int key = p.n + 1;         // places past the end
    if (tid < p.rows) {
      key = ids ? ids[tid] : 0;
      if (key < 0 || key >= p.n) key = p.n;
    }
    for (int k = lane; k < p.n + 2; k += 32) counts[warp][k] = 0;
    __syncwarp();
    const uint32_t peers = __match_any_sync(0xffffffffu, key);
    if (lane == __ffs(static_cast<int>(peers)) - 1) counts[warp][key] = static_cast<uint16_t>(__popc(peers));
    __syncthreads();
    int all = 0;
    if (tid < p.n + 2) {
#pragma unroll 8
      for (int w = 0; w < 32; ++w) {
        const int c = counts[w][tid];
        counts[w][tid] = static_cast<uint16_t>(all);
        all += c;
      }
    }
    int scan = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) sums[0][warp] = scan;
    __syncthreads();
    if (tid < p.n + 2) {
      int first = scan - all;
      for (int w = 0; w < warp; ++w) first += sums[0][w];
      base[tid] = first;
      p.starts[tid] = first;
      if (tid == p.n) *p.live = first;
    }
    __syncthreads();
    if (tid < p.rows) {
      const int to = base[key] + counts[warp][key] + __popc(peers & ((1u << lane) - 1u));
      p.keys[to] = key;
      p.pos[to] = tid;
    }
  } else {
    for (int g = tid; g <= p.rows; g += 1024) {
      const int before = g == 0 ? -1 : p.keys[g - 1], here = g == p.rows ? p.n + 1 : p.keys[g];
      for (int a = before + 1; a <= here; ++a) p.starts[a] = g;
    }
  }
  if (tid < 2) total[tid] = 0;
  __syncthreads();
  for (int a0 = 0; a0 <= p.n; a0 += 1024) {
    const int a = a0 + tid;
    const int first = a <= p.n ? p.starts[a] : 0, count = a <= p.n ? p.starts[a + 1] - first : 0;
    const int mine[2] = {(count + kRows - 1) / kRows, (count + p.run_rows - 1) / p.run_rows};
    int scan[2];
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      scan[l] = mine[l];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan[l], o);
        if (lane >= o) scan[l] += v;
      }
      if (lane == 31) sums[l][warp] = scan[l];
    }
    __syncthreads();
    int at[2];
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      at[l] = total[l] + scan[l] - mine[l];
      for (int w = 0; w < warp; ++w) at[l] += sums[l][w];
    }
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      Item* const list = l ? p.runs : p.items;
      const int each = l ? p.run_rows : kRows;
      const bool alone = mine[l] <= 4;      // longer ones by the whole warp, one adapter after the other
      for (int i = 0; alone && i < mine[l]; ++i) list[at[l] + i] = Item{a, first + i * each, min(each, count - i * each), 0};
      for (uint32_t left = __ballot_sync(0xffffffffu, !alone); left; left &= left - 1) {
        const int from = __ffs(static_cast<int>(left)) - 1;
        const int n = __shfl_sync(0xffffffffu, mine[l], from), to = __shfl_sync(0xffffffffu, at[l], from),
                  f = __shfl_sync(0xffffffffu, first, from), c = __shfl_sync(0xffffffffu, count, from);
        for (int i = lane; i < n; i += 32)
          list[to + i] = Item{a - lane + from, f + i * each, min(each, c - i * each), 0};
      }
    }
    __syncthreads();
    if (tid == 1023) {
#pragma unroll
      for (int l = 0; l < 2; ++l) total[l] = at[l] + mine[l];
    }
    __syncthreads();
  }
  if (tid == 0) {
    const bool few = total[1] <= kFewRuns * total[0];
    p.counts[0] = total[0];
    p.counts[1] = p.choose && !few ? 0 : total[1];
    p.counts[2] = few ? 0 : total[0];
  }
}

// ------------------------------------------------------------------ tiles in shared memory
// A tile's rows lie kPad elements apart more than they are long, so that the eight
// 16-byte rows of a matrix load fall into different banks.  fp32 tiles are read as
// pairs along their rows (narrow) or their columns (outer): 8 and 4 floats of padding.
template <typename X>
__device__ __forceinline__ void copy_chunk(X* dst, const X* src, bool on) {   // 16 bytes, or zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}

// Eight elements of a row (or zeros) into a tile by an asynchronous copy, both being
// aligned; `any`: an address that may be named where nothing is read.
template <typename X>
__device__ __forceinline__ void copy8(X* dst, const X* row, int c, int width, const X* any) {
  constexpr int n = 16 / sizeof(X);
#pragma unroll
  for (int h = 0; h < 8; h += n) {
    const bool on = row != nullptr && c + h < width;      // width is a multiple of n
    copy_chunk(dst + h, on ? row + c + h : any, on);
  }
}
template <typename X>
__device__ __forceinline__ void put8(X* dst, const Pack<X, 8>& q) {
  reinterpret_cast<uint4*>(dst)[0] = reinterpret_cast<const uint4*>(&q)[0];
  if constexpr (sizeof(X) == 4) reinterpret_cast<uint4*>(dst)[1] = reinterpret_cast<const uint4*>(&q)[1];
}

// A pair of numbers as bf16 pairs, part by part.
template <int N>
__device__ __forceinline__ void pair_parts(float2 x, uint32_t (&w)[N]) {
  float lo[N], hi[N];
  split(x.x, lo);
  split(x.y, hi);
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = pack_bf16x2(lo[i], hi[i]);
}

// ------------------------------------------------------------------ u = wide F^T
// Grid (items, splits of the wide side).  Both operands come tile by tile (kRows and
// 8 NT rows of kTile columns) through a ring of asynchronous copies.  Warp = (16 rows,
// half of the tile's columns); the halves meet at the end.  2,048 rows of 151,936 bf16
// columns and 32 ranks: 125 us, 5.3 TB/s, two CTAs per SM and waits at each tile's barrier.  A
// first form that read fragments straight from global memory, 64 bytes of each of 8 rows at a
// time, took 915 us.  Rows off 16-byte boundaries go by way of registers, one tile ahead.
constexpr int kTile = 128;

template <typename X, int NT>
struct NarrowShape {
  static constexpr int kStages = 3;
  static constexpr int xs = kTile + kPad, fs = kTile + kPad;
  static constexpr size_t stage = sizeof(X) * kRows * xs + 2 * size_t{8} * NT * fs;
  static constexpr size_t bytes(bool async) { return async ? kStages * stage : stage; }
  static_assert(sizeof(float) * 4 * 32 * NT * 4 <= stage, "the halves meet in one stage");
};

template <typename X, int NT, bool kAsync>
__global__ void __launch_bounds__(kThreads) narrow_kernel(const X* wide, int64_t ld, const bf16* factor, int width,
                                                          int rank, Plan p, float* part, int per_split) {
  using S = NarrowShape<X, NT>;
  constexpr int N = kPartsOf<X>, kStages = kAsync ? S::kStages : 1;
  constexpr int kX = kRows * kTile / 8 / kThreads, kF = NT * kTile / kThreads;
  static_assert(kF >= 1, "chunks per thread");
  extern __shared__ __align__(16) char shared[];
  __shared__ int64_t offset[kRows];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= p.counts[0]) return;
  const Item it = p.items[blockIdx.x];
  if (it.adapter >= p.n) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  if (tid < it.count) offset[tid] = p.pos[it.first + tid] * ld;
  __syncthreads();
  auto x_tile = [&](int s) { return reinterpret_cast<X*>(shared + s * S::stage); };
  auto f_tile = [&](int s) { return reinterpret_cast<bf16*>(shared + s * S::stage + sizeof(X) * kRows * S::xs); };
  const int begin = blockIdx.y * per_split;
  const int end = static_cast<int>(min(static_cast<int64_t>(begin) + per_split, static_cast<int64_t>(width)));
  const bf16* const f0 = factor + static_cast<int64_t>(it.adapter) * rank * width;
  Pack<X, 8> xq[kX];
  Pack<bf16, 8> fq[kF];
  // chunk i of a thread: row (i kThreads + tid) / 16, columns 8 (tid % 16)
  const int row0 = tid / 16, col = tid % 16 * 8;
  auto fetch = [&](int c0, int s) {
    if constexpr (kAsync) {
#pragma unroll
      for (int i = 0; i < kX; ++i) {
        const int r = row0 + i * 16;
        copy8(x_tile(s) + r * S::xs + col, r < it.count ? wide + offset[r] : nullptr, c0 + col, end, wide);
      }
#pragma unroll
      for (int i = 0; i < kF; ++i) {
        const int r = row0 + i * 16;
        copy8(f_tile(s) + r * S::fs + col, r < rank ? f0 + static_cast<int64_t>(r) * width : nullptr, c0 + col, width,
              factor);
      }
    } else {
      const int c = c0 + col;
      at_columns(false, c, end, [&](auto at) {
#pragma unroll
        for (int i = 0; i < kX; ++i) {
          const int r = row0 + i * 16;
          xq[i] = r < it.count && c < end ? load8<decltype(at)::value>(wide + offset[r], c, end) : Pack<X, 8>{};
        }
#pragma unroll
        for (int i = 0; i < kF; ++i) {
          const int r = row0 + i * 16;
          fq[i] = r < rank && c < end ? load8<decltype(at)::value>(f0 + static_cast<int64_t>(r) * width, c, end)
                                      : Pack<bf16, 8>{};
        }
      });
    }
  };
  const int m0 = (warp & 3) * 16, k0 = (warp >> 2) * (kTile / 2);
  const bool busy = m0 < it.count;
  float acc[NT][4] = {};
  if constexpr (kAsync) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      if (begin + s * kTile < end) fetch(begin + s * kTile, s);
      copy_async_commit();
    }
  } else {
    fetch(begin, 0);
  }
  int stage = 0;
  for (int c0 = begin; c0 < end; c0 += kTile) {
    if constexpr (kAsync) {
      copy_async_wait<kStages - 2>();
      __syncthreads();
      const int ahead = c0 + (kStages - 1) * kTile;
      if (ahead < end) fetch(ahead, (stage + kStages - 1) % kStages);
      copy_async_commit();
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kX; ++i) put8(x_tile(0) + (row0 + i * 16) * S::xs + col, xq[i]);
#pragma unroll
      for (int i = 0; i < kF; ++i) put8(f_tile(0) + (row0 + i * 16) * S::fs + col, fq[i]);
      __syncthreads();
      if (c0 + kTile < end) fetch(c0 + kTile, 0);
    }
    if (busy) {
      const X* const xt = x_tile(stage);
      const bf16* const ft = f_tile(stage);
      // a tile's sum starts from zero, so that its terms are not cut to the last bit of a long sum
      float sum[NT][4] = {};
#pragma unroll
      for (int k = k0; k < k0 + kTile / 2; k += 16) {
        uint32_t a[N][4];
        if constexpr (sizeof(X) == 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[N];
            pair_parts(*reinterpret_cast<const float2*>(xt + (m0 + (i & 1) * 8 + g) * S::xs + k + (i >> 1) * 8 + 2 * t), w);
#pragma unroll
            for (int s = 0; s < N; ++s) a[s][i] = w[s];
          }
        } else {
          uint32_t raw[4];
          load_matrices(raw, xt + (m0 + (lane >> 3 & 1) * 8 + (lane & 7)) * S::xs + k + (lane >> 4) * 8);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (N == 1) {
              a[0][i] = raw[i];
            } else {
              uint32_t w[N];
              pair_parts(__half22float2(*reinterpret_cast<const __half2*>(&raw[i])), w);
#pragma unroll
              for (int s = 0; s < N; ++s) a[s][i] = w[s];
            }
          }
        }
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          uint32_t b[4];   // two blocks of 8 ranks
          load_matrices(b, ft + (j * 8 + (lane >> 4) * 8 + (lane & 7)) * S::fs + k + (lane >> 3 & 1) * 8);
#pragma unroll
          for (int s = N - 1; s >= 0; --s) {
            mma(sum[j], a[s], b[0], b[1]);
            mma(sum[j + 1], a[s], b[2], b[3]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] += sum[j][e];
    }
    stage = (stage + 1) % kStages;
  }
  if constexpr (kAsync) copy_async_wait<0>();
  __syncthreads();
  float* const meet = reinterpret_cast<float*>(shared) + ((warp & 3) * 32 + lane);   // [NT * 4][4 * 32]
  if (warp >= 4) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) meet[(j * 4 + e) * 128] = acc[j][e];
  }
  __syncthreads();
  if (warp >= 4) return;
  const int wide_rank = round_rank(rank);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = m0 + (e >> 1) * 8 + g, c = j * 8 + 2 * t + (e & 1);
      if (r < it.count && c < rank)
        part[(static_cast<int64_t>(blockIdx.y) * p.rows + it.first + r) * wide_rank + c] =
            acc[j][e] + meet[(j * 4 + e) * 128];
    }
}

// u = scale * the sum of its splits, as bf16 parts [rows][kParts][round_rank(rank)].
struct Join {
  const float* part;
  int splits;
  bf16* u;
};

__global__ void __launch_bounds__(kThreads) join_kernel(Plan p, Join first, Join second, const float* scale, int rank) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const float* const part = blockIdx.y ? second.part : first.part;
  const int splits = blockIdx.y ? second.splits : first.splits;
  bf16* const u = blockIdx.y ? second.u : first.u;
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
// Persistent grids over units of work.  widen_kernel: (block of columns, run of up to
// `run_rows` rows of one adapter), runs of one block next to each other, so that they find F
// in the L2.  F's block stays in registers (ranks up to 64) or shared memory for the
// run, u comes 64 rows at a time, and y moves 16 rows at a time through a ring of
// asynchronous copies in which each thread reads back what it copied itself: no
// barrier but one per 64 rows.  2,048 x 151,936 bf16 and 32 ranks: 260 us, 4.9 TB/s; what is
// missing is the start of a unit (places, factor, ring), which only other CTAs cover.
// A warp has 32 columns.  Their order in shared memory is such that a thread's
// results in four 8-column tiles are 8 consecutive columns: word w (two columns) of
// the group of 32 lies at (w % 4) * 4 + w / 4.  So rows of y move 16 bytes a thread.
// Rows off 16-byte boundaries go column by column instead, their share by way of
// the warp's own corner of shared memory.
// few_kernel takes runs of up to four rows where adapters have few (one token per request),
// which have little to share: each thread multiplies its 8 columns of F, read once, by the rows' u (64 rows of 16
// adapters, rank 16, 151,936 columns: 31 us, 3.4 TB/s).
constexpr int kFewBlock = kThreads * 8;      // columns of such a unit
constexpr int kMostRun = 512;

template <typename Y>
constexpr int kPartsFor = sizeof(Y) == 4 ? kParts : 2;     // of u in a result of type Y

template <typename Y, int KT>
struct WidenShape {
  static constexpr int kStages = sizeof(Y) == 4 ? 3 : 4;
  static constexpr int kChunks = sizeof(Y) / 2;            // of 16 bytes: 8 columns of a row
  static constexpr int fs = kBlock + kPad, us = 16 * KT + kPad, u_size = kPartsFor<Y> * kRows * us;
  // F, two buffers of u, and the ring or the warps' corners
  static constexpr size_t bytes(bool packs) {
    return 2 * (size_t{16} * KT * fs + 2 * u_size) +
           (packs ? size_t{16} * 2 * kChunks * kThreads * kStages : sizeof(float) * kWarps * 16 * 33);
  }
};

template <typename Y, int KT, bool kPacks>
__global__ void __launch_bounds__(kThreads, KT <= 2 ? 3 : KT <= 4 ? 2 : 1)
widen_kernel(const Y* base, int64_t base_ld, Y* out, int64_t out_ld, const bf16* factor, int width, int rank,
             const bf16* u, Plan p, bool factor_wide) {
  using S = WidenShape<Y, KT>;
  constexpr int kStages = S::kStages, P = kPartsFor<Y>;
  constexpr bool kHold = KT <= 4;
  extern __shared__ __align__(16) char shared[];
  __shared__ int places[kMostRun];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int n_runs = p.counts[1];
  const int blocks = (width - 1) / kBlock + 1;
  // a narrow product takes its runs in pieces of kRows rows, to have enough units
  const int pieces = static_cast<int64_t>(n_runs) * blocks < 2 * static_cast<int64_t>(gridDim.x) ? p.run_rows / kRows : 1;
  const int64_t units = static_cast<int64_t>(n_runs) * blocks * pieces;
  const int wide_rank = round_rank(rank);
  bf16* const F = reinterpret_cast<bf16*>(shared);
  bf16* const U = F + 16 * KT * S::fs;                   // two buffers
  char* const ring = reinterpret_cast<char*>(U + 2 * S::u_size);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  float* const corner = reinterpret_cast<float*>(ring) + warp * 16 * 33;   // without kPacks
  char* const slots = ring + tid * 16;
  const int row8 = (lane >> 3 & 1) * 8 + (lane & 7), col8 = (lane >> 4) * 8;   // of a matrix load
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t piece = unit / n_runs;
    Item it = p.runs[unit % n_runs];
    const int c0 = static_cast<int>(piece / pieces) * kBlock;
    if (pieces > 1) {
      const int skip = static_cast<int>(piece % pieces) * kRows;
      it.first += skip;
      it.count = min(it.count - skip, kRows);
      if (it.count <= 0) continue;
    }
    const bool bare = it.adapter >= p.n;
    if (bare && base == out) continue;
    const bf16* const f = factor + static_cast<int64_t>(it.adapter) * rank * width;
    const int mine = c0 + warp * 32 + (kPacks ? 8 * t : lane);       // this thread's columns
    __syncthreads();     // the unit before has read its places, F and u
    for (int i = tid; i < it.count; i += kThreads) places[i] = p.pos[it.first + i];
    __syncthreads();
    const Y* const from = base ? base + mine : nullptr;
    Y* const to = out + mine;
    // stage s of the ring: 16 rows, this thread's chunk of two of them
    auto fetch = [&](int r0, int s) {
      if constexpr (kPacks) {
        if (!base || mine >= width) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = r0 + h * 8 + g;
          if (r >= it.count) continue;
          const Y* const src = from + places[r] * base_ld;
          const uint32_t dst = smem_addr(slots) + static_cast<uint32_t>((s * 2 + h) * S::kChunks * kThreads * 16);
          if (mine + 8 <= width) {
#pragma unroll
            for (int q = 0; q < S::kChunks; ++q)
              copy_async<16>(dst + q * kThreads * 16, src + q * kVec<Y>);
          } else {
#pragma unroll
            for (int q = 0; q < S::kChunks; ++q) {
              constexpr int n = kVec<Y>;
              const int left = max(0, min(width - mine - q * n, n)) * static_cast<int>(sizeof(Y));
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + q * kThreads * 16),
                           "l"(left ? src + q * n : base), "r"(left)
                           : "memory");
            }
          }
        }
      }
    };
    auto fetch_u = [&](int r0, int buffer) {
      constexpr int packs = 2 * KT;
      bf16* const dst = U + buffer * S::u_size;
#pragma unroll
      for (int i0 = 0; i0 < P * kRows * packs; i0 += kThreads) {
        const int i = i0 + tid, k = i / (kRows * packs), r = i / packs % kRows, c = i % packs * 8;
        if (P * kRows * packs % kThreads && i >= P * kRows * packs) break;
        const bool on = r0 + r < it.count && c < wide_rank;
        copy_chunk(dst + (k * kRows + r) * S::us + c,
                   on ? u + (static_cast<int64_t>(it.first + r0 + r) * kParts + k) * wide_rank + c : u, on);
      }
    };
    if (!bare) fetch_u(0, 0);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      if (s * 16 < it.count) fetch(s * 16, s);
      copy_async_commit();
    }
    uint32_t held[kHold ? KT : 1][2][4];
    if (!bare) {
      // this thread's 8 columns of every eighth rank
      const int c = tid % (kBlock / 8) * 8, first = tid / (kBlock / 8);
      constexpr int kAtOnce = KT <= 2 ? 2 * KT : 4;
      at_columns(factor_wide, c0 + c, width, [&](auto at) {
#pragma unroll
        for (int k0 = 0; k0 < 16 * KT; k0 += 8 * kAtOnce) {
          Pack<bf16, 8> v[kAtOnce];
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const int k = k0 + i * 8 + first;
            v[i] = k < rank && c0 + c < width ? load8<decltype(at)::value>(f + static_cast<int64_t>(k) * width, c0 + c, width)
                                              : Pack<bf16, 8>{};
          }
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const int k = k0 + i * 8 + first;
            const uint4 w = *reinterpret_cast<const uint4*>(&v[i]);
            if constexpr (kPacks) {
              uint32_t* const dst = reinterpret_cast<uint32_t*>(F + k * S::fs + c / 32 * 32) + c % 32 / 8;
              dst[0] = w.x;
              dst[4] = w.y;
              dst[8] = w.z;
              dst[12] = w.w;
            } else {
              *reinterpret_cast<uint4*>(F + k * S::fs + c) = w;
            }
          }
        }
      });
      if constexpr (kHold) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            load_matrices_turned(held[k][h], F + (k * 16 + row8) * S::fs + warp * 32 + h * 16 + col8);
      }
    }
    int stage = 0;
    for (int r0 = 0; r0 < it.count; r0 += 16) {
      // all but the last kStages - 2 groups are here: this stage, and u of these rows before it
      copy_async_wait<kStages - 2>();
      if (r0 % kRows == 0 && !bare) {
        __syncthreads();
        if (r0 + kRows < it.count) fetch_u(r0 + kRows, (r0 / kRows + 1) & 1);
      }
      const int ahead = r0 + (kStages - 1) * 16;
      if (ahead < it.count) fetch(ahead, stage == 0 ? kStages - 1 : stage - 1);
      copy_async_commit();
      Y single[16];
      if constexpr (!kPacks) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          single[r] = from_f32<Y>(0.f);
          if (r0 + r < it.count && base && mine < width) single[r] = from[places[r0 + r] * base_ld];
        }
      }
      float acc[4][4] = {};
      if (!bare) {
        const bf16* const own = U + (r0 / kRows & 1) * S::u_size + (r0 % kRows + row8) * S::us + col8;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          uint32_t b[2][4];
          if constexpr (!kHold) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              load_matrices_turned(b[h], F + (k * 16 + row8) * S::fs + warp * 32 + h * 16 + col8);
          }
#pragma unroll
          for (int s = P - 1; s >= 0; --s) {
            uint32_t a[4];
            load_matrices(a, own + s * kRows * S::us + k * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if constexpr (kHold)
                mma(acc[j], a, held[k][j >> 1][(j & 1) * 2], held[k][j >> 1][(j & 1) * 2 + 1]);
              else
                mma(acc[j], a, b[j >> 1][(j & 1) * 2], b[j >> 1][(j & 1) * 2 + 1]);
            }
          }
        }
      }
      if constexpr (kPacks) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = r0 + h * 8 + g;
          if (r >= it.count) continue;
          Pack<Y, 8> y{};
          if (base) {
#pragma unroll
            for (int q = 0; q < S::kChunks; ++q)
              reinterpret_cast<uint4*>(&y)[q] =
                  *reinterpret_cast<const uint4*>(slots + ((stage * 2 + h) * S::kChunks + q) * kThreads * 16);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) set_pair(y, j, add2(pair_of(y, j), make_float2(acc[j][2 * h], acc[j][2 * h + 1])));
          Y* const dst = to + places[r] * out_ld;
          if (mine + 8 <= width) {
            *reinterpret_cast<Pack<Y, 8>*>(dst) = y;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (mine + e < width) dst[e] = y.v[e];
          }
        }
      } else {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) corner[((e >> 1) * 8 + g) * 33 + j * 8 + 2 * t + (e & 1)] = acc[j][e];
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (r0 + r < it.count && mine < width)
            to[places[r0 + r] * out_ld] = from_f32<Y>(to_f32(single[r]) + corner[r * 33 + lane]);
      }
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    copy_async_wait<0>();
  }
}

template <typename Y, bool kPacks>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(const Y* base, int64_t base_ld, Y* out, int64_t out_ld,
                                                          const bf16* factor, int width, int rank, const bf16* u, Plan p,
                                                          bool factor_wide) {
  constexpr int kAhead = 8;      // ranks in flight
  __shared__ float4 us[kMaxRank];      // of four rows
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int n_runs = p.counts[1], blocks = (width - 1) / kFewBlock + 1, wide_rank = round_rank(rank);
  const int64_t units = static_cast<int64_t>(n_runs) * blocks;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const Item it = p.runs[unit / blocks];
    const bool bare = it.adapter >= p.n;
    if (bare && base == out) continue;
    const int ranks = bare ? 0 : rank;
    const int c = static_cast<int>(unit % blocks) * kFewBlock + threadIdx.x * 8;
    const bf16* const f = factor + static_cast<int64_t>(it.adapter) * rank * width;
    __syncthreads();     // the unit before has read its u
    for (int i = threadIdx.x; !bare && i < kFewAtOnce * wide_rank; i += kThreads) {
      const int r = i / wide_rank, k = i % wide_rank;      // 0 behind the rank
      const bf16* const q = u + static_cast<int64_t>(it.first + r) * kParts * wide_rank + k;
      reinterpret_cast<float*>(us)[k * 4 + r] =
          r < it.count ? __bfloat162float(q[0]) + (__bfloat162float(q[wide_rank]) + __bfloat162float(q[2 * wide_rank])) : 0.f;
    }
    __syncthreads();
    Pack<Y, 8> y[kFewAtOnce];
    Y* dst[kFewAtOnce];
    float2 acc[kFewAtOnce][4] = {};
    at_columns(factor_wide && c < width, c, width, [&](auto at) {
      Pack<bf16, 8> q[kAhead];
      auto fetch = [&](int k0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          q[k] = Pack<bf16, 8>{};
          if (k0 + k < ranks && c < width) q[k] = load8<decltype(at)::value>(f + static_cast<int64_t>(k0 + k) * width, c, width);
        }
      };
      fetch(0);      // before all that waits for the rows' places
#pragma unroll
      for (int r = 0; r < kFewAtOnce; ++r) {
        if (r >= it.count || c >= width) continue;
        const int64_t row = p.pos[it.first + r];
        dst[r] = out + row * out_ld + c;
        y[r] = Pack<Y, 8>{};
        if (!base) continue;
        const Y* const src = base + row * base_ld + c;
        if (kPacks && c + 8 <= width) {
          y[r] = *reinterpret_cast<const Pack<Y, 8>*>(src);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < width) y[r].v[e] = src[e];
        }
      }
      for (int k0 = 0; k0 < ranks; k0 += kAhead) {
        if (k0) fetch(k0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float4 w = us[k0 + k];
          const float each[kFewAtOnce] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = pair_of(q[k], e);
#pragma unroll
            for (int r = 0; r < kFewAtOnce; ++r) acc[r][e] = fma2(x, make_float2(each[r], each[r]), acc[r][e]);
          }
        }
      }
    });
    if (c >= width) continue;
#pragma unroll
    for (int r = 0; r < kFewAtOnce; ++r) {
      if (r >= it.count) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) set_pair(y[r], e, add2(pair_of(y[r], e), acc[r][e]));
      if (kPacks && c + 8 <= width) {
        *reinterpret_cast<Pack<Y, 8>*>(dst[r]) = y[r];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < width) dst[r][e] = y[r].v[e];
      }
    }
  }
}

// ------------------------------------------------------------------ dF = sum u^T wide
// CTA = (block of columns, adapter and part of its rows, block of 16 RT ranks).  Steps of
// kOuterRows rows come through a ring of asynchronous copies; the rows' places are read a
// step ahead.  A warp has 32 columns of the block.  2,048 x 151,936 bf16 and 32 ranks: 188 us,
// 3.7 TB/s with the tensor pipe 53% busy on three parts of u.
template <typename X, int RT>
struct OuterShape {
  static constexpr int kStages = 3;
  static constexpr int fs = kBlock + (sizeof(X) == 4 ? 4 : kPad), us = 16 * RT + kPad;
  static constexpr size_t x_bytes = sizeof(X) * kOuterRows * fs;
  static constexpr size_t stage = x_bytes + 2 * size_t{kParts} * kOuterRows * us;
  static constexpr size_t bytes(bool async) { return async ? kStages * stage : stage; }
};

// One element of dF from whole numbers, for sums that are no finite number: a part of u or of g is not the
// number itself where the other factor is infinite (it may be 0 or have the other sign, and 0 x inf or
// inf - inf would make a NaN of an infinity).  Once the sum is NaN it stays so.
template <typename X>
__device__ __noinline__ float outer_element(const X* wide, int64_t ld, const bf16* u, int wide_rank, const int32_t* pos,
                                            int from, int to) {
  constexpr int kAtOnce = 4;      // more would make the kernels spill
  float s = 0.f;
  for (int r0 = from; r0 < to && s == s; r0 += kAtOnce) {
    float all[kAtOnce], g[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int r = min(r0 + i, to - 1);
      const bf16* const q = u + static_cast<int64_t>(r) * kParts * wide_rank;
      all[i] = to_f32(q[0]) + (to_f32(q[wide_rank]) + to_f32(q[2 * wide_rank]));
      g[i] = to_f32(wide[pos[r] * ld]);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (r0 + i < to) s = fmaf(all[i], g[i], s);
  }
  return s;
}

template <typename X, int RT, bool kAsync>
__global__ void __launch_bounds__(kThreads, kAsync && sizeof(X) == 2 && RT <= 2 ? 3 : 1) outer_kernel(const X* wide, int64_t ld, int width, int rank, const bf16* u,
                                                         Plan p, float* grad, int accumulate, int row_splits,
                                                         int64_t split_size) {
  using S = OuterShape<X, RT>;
  constexpr int N = kPartsOf<X>, kStages = kAsync ? S::kStages : 1, kRowsEach = kOuterRows / kWarps;
  constexpr int kPacks = (kOuterRows * kParts * RT * 2 + kThreads - 1) / kThreads;   // of u per thread
  extern __shared__ __align__(16) char shared[];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int c0 = blockIdx.x * kBlock, adapter = blockIdx.y / row_splits, part = blockIdx.y % row_splits;
  const int rank0 = blockIdx.z * 16 * RT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int wide_rank = round_rank(rank);
  const int all_from = p.starts[adapter], all_to = p.starts[adapter + 1];
  const int each = ((all_to - all_from + row_splits - 1) / row_splits + kOuterRows - 1) / kOuterRows * kOuterRows;
  const int from = min(all_from + part * each, all_to), to = min(from + each, all_to);
  auto x_tile = [&](int s) { return reinterpret_cast<X*>(shared + s * S::stage); };
  auto u_tile = [&](int s) { return reinterpret_cast<bf16*>(shared + s * S::stage + S::x_bytes); };
  Pack<X, 8> xq[kRowsEach];
  Pack<bf16, 8> uq[kPacks];
  int place[kRowsEach];        // of the next step's rows
  auto look = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
      const int r = r0 + i * kWarps + warp;
      place[i] = r < to ? p.pos[r] : -1;
    }
  };
  auto fetch = [&](int r0, int s) {
    const int c = c0 + lane * 8;
    if constexpr (kAsync) {
#pragma unroll
      for (int i = 0; i < kRowsEach; ++i)
        copy8(x_tile(s) + (i * kWarps + warp) * S::fs + lane * 8, place[i] >= 0 ? wide + place[i] * ld : nullptr, c, width,
              wide);
    } else {
      at_columns(false, c, width, [&](auto at) {
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i)
          xq[i] = place[i] >= 0 && c < width ? load8<decltype(at)::value>(wide + place[i] * ld, c, width) : Pack<X, 8>{};
      });
    }
#pragma unroll
    for (int i = 0; i < kPacks; ++i) {
      const int at = i * kThreads + tid, k = at / (kOuterRows * RT * 2), r = at / (RT * 2) % kOuterRows,
                cu = at % (RT * 2) * 8;
      if (k >= kParts) continue;
      const bool on = r0 + r < to && rank0 + cu < wide_rank;
      const bf16* const src = on ? u + (static_cast<int64_t>(r0 + r) * kParts + k) * wide_rank + rank0 + cu : u;
      if constexpr (kAsync)
        copy_chunk(u_tile(s) + (k * kOuterRows + r) * S::us + cu, src, on);
      else
        uq[i] = on ? load8<At::kAligned>(src, 0, 8) : Pack<bf16, 8>{};
    }
    look(r0 + kOuterRows);
  };
  float acc[RT][4][4] = {};
  look(from);
  if constexpr (kAsync) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      if (from + s * kOuterRows < to) fetch(from + s * kOuterRows, s);
      copy_async_commit();
    }
  } else {
    fetch(from, 0);
  }
  int stage = 0;
  for (int r0 = from; r0 < to; r0 += kOuterRows) {
    if constexpr (kAsync) {
      copy_async_wait<kStages - 2>();
      __syncthreads();
      const int ahead = r0 + (kStages - 1) * kOuterRows;
      if (ahead < to) fetch(ahead, (stage + kStages - 1) % kStages);
      copy_async_commit();
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kRowsEach; ++i) put8(x_tile(0) + (i * kWarps + warp) * S::fs + lane * 8, xq[i]);
#pragma unroll
      for (int i = 0; i < kPacks; ++i) {
        const int at = i * kThreads + tid, k = at / (kOuterRows * RT * 2), r = at / (RT * 2) % kOuterRows,
                  c = at % (RT * 2) * 8;
        if (k < kParts) put8(u_tile(0) + (k * kOuterRows + r) * S::us + c, uq[i]);
      }
      __syncthreads();
      fetch(r0 + kOuterRows, 0);
    }
    const X* const W = x_tile(stage);
    const bf16* const U = u_tile(stage);
    // a step's sum starts from zero, so that its terms are not cut to the last bit of a long sum
    float sum[RT][4][4] = {};
#pragma unroll
    for (int k = 0; k < kOuterRows; k += 16) {
      uint32_t b[N][4][2];
      if constexpr (sizeof(X) == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const X* const at = W + (k + h * 8 + 2 * t) * S::fs + warp * 32 + j * 8 + g;
            uint32_t w[N];
            pair_parts(make_float2(at[0], at[S::fs]), w);
#pragma unroll
            for (int s = 0; s < N; ++s) b[s][j][h] = w[s];
          }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t raw[4];
          load_matrices_turned(raw, W + (k + (lane >> 3 & 1) * 8 + (lane & 7)) * S::fs + warp * 32 + h * 16 + (lane >> 4) * 8);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (N == 1) {
              b[0][2 * h + (i >> 1)][i & 1] = raw[i];
            } else {
              uint32_t w[N];
              pair_parts(__half22float2(*reinterpret_cast<const __half2*>(&raw[i])), w);
#pragma unroll
              for (int s = 0; s < N; ++s) b[s][2 * h + (i >> 1)][i & 1] = w[s];
            }
          }
        }
      }
#pragma unroll
      for (int v = kParts - 1; v >= 0; --v)
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          uint32_t a[4];
          load_matrices_turned(a, U + (v * kOuterRows + k + (lane >> 4) * 8 + (lane & 7)) * S::us + m * 16 +
                                      (lane >> 3 & 1) * 8);
#pragma unroll
          for (int s = N - 1; s >= 0; --s)
            if (s + v < kParts) {
#pragma unroll
              for (int j = 0; j < 4; ++j) mma(sum[m][j], a, b[s][j][0], b[s][j][1]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][j][e] += sum[m][j][e];
    stage = (stage + 1) % kStages;
  }
  if constexpr (kAsync) copy_async_wait<0>();
  if (accumulate && all_from == all_to) return;
  float* const result = grad + part * split_size;
#pragma unroll
  for (int m = 0; m < RT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = rank0 + m * 16 + h * 8 + g;
      if (r >= rank) continue;
      float* const dst = result + (static_cast<int64_t>(adapter) * rank + r) * width;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = c0 + warp * 32 + j * 8 + 2 * t + e;
          if (c >= width) continue;
          float sum = acc[m][j][2 * h + e];
          if (!isfinite(sum)) sum = outer_element(wide + c, ld, u + r, wide_rank, p.pos, from, to);
          dst[c] = accumulate ? dst[c] + sum : sum;
        }
    }
}

// dF = the sum of its row splits.
__global__ void __launch_bounds__(kThreads) add_splits_kernel(const float* part, int splits, int64_t size, float* grad,
                                                              int accumulate) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= size) return;
  float s = 0.f;
#pragma unroll 4
  for (int k = 0; k < splits; ++k) s += part[k * size + i];
  grad[i] = accumulate ? grad[i] + s : s;
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

// Items, or runs of `each` rows, that lists of rows of n adapters (and of none) are cut into.
int64_t most_items(int64_t rows, int n, int each = kRows) { return rows / each + (n + 1 < rows ? n + 1 : rows) + 1; }

// Splits of the wide side: one wave of two CTAs per SM (at 2,048 x 151,936 bf16 and rank 32
// 2.4 waves took 155 us, one takes 130), at least 512 columns each.  Adapters' last items are part full.
int splits_of(int64_t rows, int width, int n, int& per_split) {
  const int64_t items = (rows + kRows - 1) / kRows, partial = (n + 1) / 2;
  int64_t splits = kFewCtas / (items + (partial < items ? partial : items));
  const int64_t most = (width + 511) / 512;
  if (splits > most) splits = most;
  if (splits < 1) splits = 1;
  per_split = static_cast<int>(((width + splits - 1) / splits + kTile - 1) / kTile * kTile);
  return (width - 1) / per_split + 1;
}

// Splits of an adapter's rows, where columns and adapters alone leave SMs idle.
int row_splits_of(int64_t rows, int width, int n) {
  const int64_t ctas = (static_cast<int64_t>(width) + kBlock - 1) / kBlock * n;
  int64_t splits = kFewCtas / ctas;
  const int64_t most = rows / n / (8 * kOuterRows);   // 8 steps each: the splits cost a launch to join
  if (splits > most) splits = most;
  return splits < 1 ? 1 : static_cast<int>(splits);
}

// Whether few_kernel may multiply: where adapters have few rows on average.  Forward passes of
// rank 16 and 151,936 columns by few_kernel | widen_kernel: 64 rows of 16 adapters 49 | 72 us, 256
// of 64 127 | 231, 512 of 64 189 | 248, 256 of 16 96 | 90, 1,024 of 64 323 | 288.  At 10,240 columns
// 64 of 16 20 | 22, 256 of 64 28 | 35, 512 of 64 32 | 37, 1,024 of 64 45 | 41, 2,048 of 512 105 | 160; at
// 4,096 22 | 20, 24 | 26, 24 | 27, 32 | 30, 72 | 93.  If all rows have
// the same one of them, widen_kernel is faster: 64 rows 34 | 30, 256 86 | 53, 2,048 567 | 231 (10,240
// columns: 20 | 20, 24 | 22, 66 | 48).  So
// for more than kFewAlone rows the plan chooses and both are launched, one of them without work.
bool use_few(int64_t rows, int n) { return rows <= int64_t{kFewMean} * n; }

struct Space {
  Plan plan;
  bf16 *u, *du;
  float* part;       // splits of u and du, or of dF
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
  s.plan.counts = s.plan.live + 1;
  s.plan.keys = reinterpret_cast<int32_t*>(take(4 * static_cast<size_t>(rows)));
  s.plan.pos = reinterpret_cast<int32_t*>(take(4 * static_cast<size_t>(rows)));
  s.plan.starts = reinterpret_cast<int*>(take(4 * (static_cast<size_t>(n) + 2)));
  s.plan.most = static_cast<int>(most_items(rows, n));
  s.plan.items = reinterpret_cast<Item*>(take(sizeof(Item) * static_cast<size_t>(s.plan.most)));
  // the last part of a long list may have runs of few rows
  s.plan.runs = reinterpret_cast<Item*>(take(sizeof(Item) * static_cast<size_t>(most_items(rows, n, kFewAtOnce))));
  s.plan.n = n;
  const size_t wide_rank = static_cast<size_t>(round_rank(rank));
  s.u = reinterpret_cast<bf16*>(take(2 * kParts * wide_rank * rows));
  s.du = reinterpret_cast<bf16*>(take(2 * kParts * wide_rank * rows));
  // a last part of fewer rows has more splits of the wide side (those of at most kRows kFewCtas
  // rows in all) and no more of its rows
  size_t most = 0, narrow = 0;
  for (const int width : {H, V}) {
    int per;
    narrow += wide_rank * rows * static_cast<size_t>(splits_of(rows > 0 ? rows : 1, width, n, per));
    const int splits = row_splits_of(rows, width, n);
    const size_t outer = splits > 1 ? static_cast<size_t>(splits) * n * rank * width : 0;
    most = narrow > most ? narrow : most;
    most = outer > most ? outer : most;
  }
  s.part = reinterpret_cast<float*>(take(sizeof(float) * most));
  s.bytes = at;
  return s;
}

// Whether rows can be copied 16 bytes at a time.
template <typename X>
bool whole_chunks(const X* p, int64_t ld, int width) {
  constexpr int n = kVec<X>;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % n == 0 && width % n == 0;
}

template <typename X, int NT, bool kAsync>
cudaError_t narrow_of(const X* wide, int64_t ld, const bf16* factor, int width, int rank, const Plan& p, float* part,
                      int splits, int per_split, cudaStream_t s) {
  static std::atomic<int> ready[64];
  constexpr size_t smem = NarrowShape<X, NT>::bytes(kAsync);
  const cudaError_t e = allow_shared(ready, reinterpret_cast<const void*>(narrow_kernel<X, NT, kAsync>), smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(narrow_kernel<X, NT, kAsync>, dim3(p.most, splits), kThreads, smem, 1, s, wide, ld, factor,
                          width, rank, p, part, per_split);
}

// The splits of u of every row with an adapter, at `at` of the workspace's part, which moves on.
template <typename X>
cudaError_t narrow(const char* name, const X* wide, int64_t ld, const void* factor, int width, const Adapters& a,
                   const Space& z, float*& at, Join& join, cudaStream_t s) {
  int per_split;
  const int splits = splits_of(z.plan.rows, width, a.n, per_split);
  const bf16* const f = static_cast<const bf16*>(factor);
  const bool async = whole_chunks(wide, ld, width) && whole_chunks(f, width, width);
  float* const part = at;
  at += static_cast<size_t>(splits) * z.plan.rows * round_rank(a.rank);
  join.part = part;
  join.splits = splits;
  auto run = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    return async ? narrow_of<X, NT, true>(wide, ld, f, width, a.rank, z.plan, part, splits, per_split, s)
                 : narrow_of<X, NT, false>(wide, ld, f, width, a.rank, z.plan, part, splits, per_split, s);
  };
  return traced_launch(name, s, [&] {
    if (a.rank <= 16) return run(std::integral_constant<int, 2>{});
    if (a.rank <= 32) return run(std::integral_constant<int, 4>{});
    if (a.rank <= 64) return run(std::integral_constant<int, 8>{});
    return run(std::integral_constant<int, 16>{});
  });
}

// u, or u and du, from their splits.
cudaError_t join(const Join* joins, int n, const Adapters& a, const Plan& p, cudaStream_t s) {
  const int64_t size = static_cast<int64_t>(p.rows) * round_rank(a.rank);
  return traced_launch("adapters_join", s, [&] {
    return launch_dependent(join_kernel, dim3(static_cast<unsigned>((size + kThreads - 1) / kThreads), n), kThreads, 0, 1,
                            s, p, joins[0], joins[n - 1], a.scale, a.rank);
  });
}

template <typename Y, int KT, bool kPacks>
cudaError_t widen_of(const Y* base, int64_t base_ld, Y* out, int64_t out_ld, const bf16* factor, int width, int rank,
                     const bf16* u, const Plan& p, int sms, cudaStream_t s) {
  static std::atomic<int> ready[64];
  constexpr size_t smem = WidenShape<Y, KT>::bytes(kPacks);
  const cudaError_t e = allow_shared(ready, reinterpret_cast<const void*>(widen_kernel<Y, KT, kPacks>), smem);
  if (e != cudaSuccess) return e;
  constexpr int by_shared = static_cast<int>(size_t{220} * 1024 / (smem + 4096)), by_registers = KT <= 2 ? 3 : KT <= 4 ? 2 : 1;
  constexpr int fit = by_shared < 1 ? 1 : by_shared < by_registers ? by_shared : by_registers;
  const int64_t units = (static_cast<int64_t>(width - 1) / kBlock + 1) * p.most * (p.run_rows / kRows);
  const int64_t resident = static_cast<int64_t>(sms) * fit;
  return launch_dependent(widen_kernel<Y, KT, kPacks>, dim3(static_cast<unsigned>(units < resident ? units : resident)),
                          kThreads, smem, 1, s, base, base_ld, out, out_ld, factor, width, rank, u, p,
                          whole_chunks(factor, width, width));
}

template <typename Y>
cudaError_t widen(const char* name, const Y* base, int64_t base_ld, Y* out, int64_t out_ld, const void* factor, int width,
                  int rank, const bf16* u, const Plan& p, cudaStream_t s) {
  constexpr int VEC = kVec<Y>;
  const bf16* const f = static_cast<const bf16*>(factor);
  const bool packs = ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0 &&
                     base_ld % VEC == 0 && out_ld % VEC == 0;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  Plan wide = p;
  auto run = [&](auto kt) {
    constexpr int KT = decltype(kt)::value;
    return packs ? widen_of<Y, KT, true>(base, base_ld, out, out_ld, f, width, rank, u, wide, sms, s)
                 : widen_of<Y, KT, false>(base, base_ld, out, out_ld, f, width, rank, u, wide, sms, s);
  };
  if (use_few(p.rows, p.n)) {
    const cudaError_t e = traced_launch("adapters_few", s, [&] {
      auto kern = packs ? few_kernel<Y, true> : few_kernel<Y, false>;
      const int64_t units = most_items(p.rows, p.n, kFewAtOnce) * ((static_cast<int64_t>(width) - 1) / kFewBlock + 1);
      const int64_t resident = 2 * static_cast<int64_t>(sms);
      return launch_dependent(kern, dim3(static_cast<unsigned>(units < resident ? units : resident)), kThreads, 0, 1, s,
                              base, base_ld, out, out_ld, f, width, rank, u, p, whole_chunks(f, width, width));
    });
    if (e != cudaSuccess || !p.choose) return e;
    wide.runs = p.items;
    wide.run_rows = kRows;
    wide.counts = p.counts + 1;      // the third of them in the place of the second
  }
  return traced_launch(name, s, [&] {
    if (rank <= 16) return run(std::integral_constant<int, 1>{});
    if (rank <= 32) return run(std::integral_constant<int, 2>{});
    if (rank <= 64) return run(std::integral_constant<int, 4>{});
    return run(std::integral_constant<int, 8>{});
  });
}

template <typename X, int RT, bool kAsync>
cudaError_t outer_of(const char* name, const X* wide, int64_t ld, int width, int rank, const bf16* u, const Space& z, float* grad,
                     int accumulate, cudaStream_t s) {
  static std::atomic<int> ready[64];
  constexpr size_t smem = OuterShape<X, RT>::bytes(kAsync);
  const cudaError_t e = allow_shared(ready, reinterpret_cast<const void*>(outer_kernel<X, RT, kAsync>), smem);
  if (e != cudaSuccess) return e;
  const int splits = row_splits_of(z.plan.rows, width, z.plan.n);
  const int64_t size = static_cast<int64_t>(z.plan.n) * rank * width;
  const dim3 grid((width + kBlock - 1) / kBlock, z.plan.n * splits, (rank + 16 * RT - 1) / (16 * RT));
  const bool whole = splits == 1;
  const cudaError_t r = traced_launch(name, s, [&] {
    return launch_dependent(outer_kernel<X, RT, kAsync>, grid, kThreads, smem, 1, s, wide, ld, width, rank, u, z.plan,
                            whole ? grad : z.part, whole ? accumulate : 0, splits, size);
  });
  if (r != cudaSuccess || whole) return r;
  return traced_launch("adapters_add_splits", s, [&] {
    return launch_dependent(add_splits_kernel, dim3(static_cast<unsigned>((size + kThreads - 1) / kThreads)), kThreads,
                            0, 1, s, static_cast<const float*>(z.part), splits, size, grad, accumulate);
  });
}

template <typename X>
cudaError_t outer(const char* name, const X* wide, int64_t ld, int width, int rank, const bf16* u, const Space& z,
                  float* grad, int accumulate, cudaStream_t s) {
  const bool async = whole_chunks(wide, ld, width);
  auto run = [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    return async ? outer_of<X, RT, true>(name, wide, ld, width, rank, u, z, grad, accumulate, s)
                 : outer_of<X, RT, false>(name, wide, ld, width, rank, u, z, grad, accumulate, s);
  };
  if (rank <= 16) return run(std::integral_constant<int, 1>{});
  if (rank <= 32) return run(std::integral_constant<int, 2>{});
  return run(std::integral_constant<int, 4>{});
}

cudaError_t plan_rows(const Adapters& a, int64_t first, Space& z, cudaStream_t s) {
  z.plan.rows = static_cast<int>(a.T - first < kSortMost ? a.T - first : kSortMost);
  z.plan.most = static_cast<int>(most_items(z.plan.rows, a.n));
  // runs as long as keeps some units per CTA of the widest product
  const int64_t units = static_cast<int64_t>(a.V > a.H ? a.V : a.H) / kBlock * ((z.plan.rows + kRows - 1) / kRows);
  const int64_t run = units / (7 * kManyCtas);
  z.plan.run_rows = kRows * static_cast<int>(run < 1 ? 1 : run > kMostRun / kRows ? kMostRun / kRows : run);
  z.plan.choose = false;
  if (use_few(z.plan.rows, a.n)) {
    z.plan.run_rows = kFewAtOnce;
    z.plan.choose = z.plan.rows > kFewAlone;
  }
  const int32_t* const ids = a.ids ? a.ids + first : nullptr;
  const bool small = z.plan.rows <= kSmallRows && a.n + 2 <= kSmallKeys;
  if (!small) {
    const cudaError_t e = traced_launch("adapters_sort", s, [&] {
      return launch_sort_ids(ids, z.plan.rows, a.n, false, -1, z.plan.keys, z.plan.pos, z.plan.live, s);
    });
    if (e != cudaSuccess) return e;
  }
  return traced_launch("adapters_plan", s, [&] {
    return launch_dependent(small ? plan_kernel<true> : plan_kernel<false>, dim3(1), 1024, 0, 1, s, z.plan, ids);
  });
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
    float* at = z.part;
    Join u{nullptr, 0, z.u};
    e = narrow("adapters_narrow", static_cast<const bf16*>(a.x) + first * a.x_ld, a.x_ld, a.down, a.H, a, z, at, u, s);
    if (e == cudaSuccess) e = join(&u, 1, a, z.plan, s);
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
    float* at = z.part;
    Join joins[2];
    int n = 0;
    if (b.d_up) {
      joins[n] = Join{nullptr, 0, z.u};
      e = narrow("adapters_narrow", x, a.x_ld, a.down, a.H, a, z, at, joins[n++], s);
      if (e != cudaSuccess) return e;
    }
    e = by_type(b.type, [&](auto t) {
      using G = decltype(t);
      const G* const g = static_cast<const G*>(b.grad) + first * b.grad_ld;
      cudaError_t r = cudaSuccess;
      if (b.dx || b.d_down) {
        joins[n] = Join{nullptr, 0, z.du};
        r = narrow("adapters_narrow_grad", g, b.grad_ld, a.up, a.V, a, z, at, joins[n++], s);
      }
      if (r == cudaSuccess) r = join(joins, n, a, z.plan, s);
      if (r == cudaSuccess && b.d_up)
        r = outer("adapters_d_up", g, b.grad_ld, a.V, a.rank, z.u, z, b.d_up, accumulate, s);
      return r;
    });
    if (e == cudaSuccess && b.d_down)
      e = outer("adapters_d_down", x, a.x_ld, a.H, a.rank, z.du, z, b.d_down, accumulate, s);
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
