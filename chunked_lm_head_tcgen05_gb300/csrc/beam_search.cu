// One step of beam search.  Row r = group * beams + j of the logits belongs to
// beam j of its group, with score_r so far.  With z = x / tau,
//   lse_r = log sum_v exp(z_v),   candidate (j, v): score_r + z_v - lse_r,
// and a group's best `take` candidates go on, ties to the lowest j, then to the larger logit,
// then to the lowest v.
// HBM-bound: one read of the logits, two kernels.
//  1. scan_kernel, one CTA per piece of a row, tile by tile with the next one in flight:
//     maximum and exponential sum of the piece, and its best `take` logits.  In the first
//     tile, at least `take` groups of threads have a largest element, so the least of these
//     is at most the tile's take-th largest element: what is not below it (some
//     take * ln(take) of the elements) goes to shared memory and is ranked there.  From
//     then on only elements above the take-th best so far go there, and are ranked again
//     when they are many.  When a tile has more than fit (equal or ascending logits), its
//     take-th largest is found by halving intervals instead.  256 x 151,936 bf16: 25 us, 3.1
//     TB/s.  Some 12 us of that are instructions (12 per element); the rest is the tiles'
//     barriers and waits, which the three CTAs that fit on an SM (59,008 bytes of shared
//     memory each) do not cover, and the last CTAs of two waves.
//  2. best_kernel, one CTA per group, joins the pieces: lse, then the candidates.
//     An fp32 score with its error bound on either side sorts out most of them;
//     the rest are compared in 64 bits, where fp32 could confuse two that are
//     close (and 64-bit arithmetic for all of them would take longer than the
//     scan: a few operations per clock and SM).  7 us, all of it latency.
// Order among one row's logits is by the logit itself, as an integer that grows
// with it, then by the id.
//
// beam_reorder moves states to the beams that go on: row r takes over row parents[r].  In
// place a thread (or, for rows off 16-byte boundaries, a CTA) holds one stretch of a group's
// rows, reads what other rows need and then writes; rows that keep their place cost nothing
// (393 MB of 16 x 4 beams, half of which move: 62 us, 6.3 TB/s).
#include <type_traits>

#include "element.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace lmh {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Elements per thread and tile of many rows: 64 bytes, so tiles of 8,192 16-bit elements.
template <typename T>
constexpr int kManyElements = 64 / static_cast<int>(sizeof(T));
constexpr int kFewElements = 8;      // of few rows: pieces of one tile of 2,048
constexpr int64_t kManyTiles = 304;  // the long tiles from which on they fill the GPU
constexpr int64_t kManyPieces = 608; // CTAs that many rows are cut into, at most (456 are resident)
constexpr int kRoom = 1024;          // elements ranked in shared memory
constexpr int kBestThreads = 512;
constexpr int kBestWarps = kBestThreads / 32;

// An integer that grows with x (no NaN); 0 is below every number's.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);   // one zero
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kMinusInf = 0x007fffffu;      // order_of(-inf)
constexpr uint32_t kMinusZero = 0x7fffffffu;     // no number's: zero's is the next

// Larger logit first, then the lower id.
__device__ __forceinline__ uint64_t entry_of(uint32_t order, int v) {
  return static_cast<uint64_t>(order) << 32 | static_cast<uint32_t>(~v);
}

// log2(e) / tau, finite for every tau
__device__ __forceinline__ float steps(float tau) { return fminf(1.4426950408889634f / tau, 3.0e38f); }

// Tiles in flight; a short piece is one tile.
template <int ELEMS>
constexpr int kStagesOf = ELEMS == kFewElements ? 2 : 3;
template <typename T, int ELEMS>
constexpr size_t kRingBytes = sizeof(T) * ELEMS * kThreads * kStagesOf<ELEMS>;

struct Pieces {
  float2* stats;      // [R][pieces] maximum of x, sum of exp((x - maximum) / tau)
  uint64_t* best;     // [R][pieces][take] descending, 0 behind the last
  int pieces;
  int length;         // packs of a row per piece
};

// The number of `on` in the CTA.
__device__ __forceinline__ int count_all(int on, int* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = __reduce_add_sync(0xffffffffu, on);
  __syncthreads();
  if (lane == 0) scratch[warp] = w;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) sum += scratch[i];
  return sum;
}

// The `take` best of found[0, n), n <= kRoom, in falling order; every thread gets their number.
__device__ __noinline__ int keep_best(uint64_t* found, int n, int take) {
  constexpr int kEach = kRoom / kThreads;
  uint64_t me[kEach];
  int rank[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = i * kThreads + threadIdx.x;
    rank[i] = take;
    if (at >= n) continue;
    me[i] = found[at];
    int above = 0;
    for (int j = 0; j < n; ++j) above += found[j] > me[i];
    rank[i] = above;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (rank[i] < take) found[rank[i]] = me[i];
  __syncthreads();
  return min(n, take);
}

// The best `take` of a tile's elements above `low` (there are more than that), added to found:
// their take-th largest order, by halving intervals, then the ids up to which its equals are
// taken.  Reads the tile again each time: this is rare, and its registers are needed elsewhere.
template <typename T, int PACKS>
__device__ __noinline__ void add_best_of_tile(uint64_t* found, int* n_found, int* scratch, const T* row, int from, int p1,
                                              int skip, int V, uint32_t low, int take) {
  constexpr int VEC = kVec<T>;
  auto each = [&](auto&& f) {
    for (int i = 0; i < PACKS * VEC; ++i) {
      const int p = from + i / VEC * kThreads + threadIdx.x, v = p * VEC - skip + i % VEC;
      if (p >= p1 || v < 0 || v >= V) continue;
      const float x = to_f32(row[v]);
      if (x == x) f(order_of(x), v);       // a row with a NaN offers nothing in the end
    }
  };
  auto count = [&](auto&& f) {
    int c = 0;
    each([&](uint32_t o, int v) { c += f(o, v); });
    return count_all(c, scratch);
  };
  uint32_t lo = low + 1, hi = 0xff800000u;      // order_of(inf): no number is above it
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    if (count([&](uint32_t o, int) { return o >= mid; }) >= take) lo = mid; else hi = mid - 1;
  }
  const int larger = count([&](uint32_t o, int) { return o > lo; });
  int first = 0, last = V - 1;
  while (first < last) {
    const int mid = first + (last - first) / 2;
    if (count([&](uint32_t o, int v) { return o == lo && v <= mid; }) >= take - larger) last = mid; else first = mid + 1;
  }
  each([&](uint32_t o, int v) {
    if (o > lo || (o == lo && v <= first)) {
      const int n = atomicAdd(n_found, 1);
      if (n < kRoom) found[n] = entry_of(o, v);
    }
  });
  __syncthreads();
}

// The largest of a pack; NaN is passed over.
template <typename T, int VEC>
__device__ __forceinline__ float largest(const Pack<T, VEC>& q) {
  if constexpr (sizeof(T) == 4) {
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < VEC; ++e) top = fmaxf(top, q.v[e]);
    return top;
  } else {
    using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
    const T2* const v = reinterpret_cast<const T2*>(&q);
    T2 top = v[0];
#pragma unroll
    for (int e = 1; e < VEC / 2; ++e) top = __hmax2(top, v[e]);
    return fmaxf(fmaxf(to_f32(top.x), to_f32(top.y)), -INFINITY);       // of NaN alone: -inf
  }
}

// 64 registers, though shared memory holds three CTAs of the long tiles, not four: the fp32
// form spills 40 bytes for it.
template <typename T, int ELEMS>
__global__ void __launch_bounds__(kThreads, 4) scan_kernel(BeamSelect a, Pieces z, int groups) {
  constexpr int VEC = kVec<T>, PACKS = ELEMS / VEC, kStages = kStagesOf<ELEMS>;
  extern __shared__ __align__(16) char ring_memory[];
  __shared__ uint64_t found[kRoom];
  __shared__ uint32_t group_max[kMaxTake];
  __shared__ float2 warp_sums[kWarps];
  // elements that tiles t, t + 1 and t + 2 find: a thread that is ahead counts its next tile's
  // while others still read this one's, and the counter after that is cleared meanwhile
  __shared__ int added[3];
  __shared__ int scratch[kWarps], n_best;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int64_t r = blockIdx.x / z.pieces;
  const int piece = static_cast<int>(blockIdx.x % z.pieces);
  if (a.finished && a.finished[r]) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 3) added[tid] = 0;
  if (tid < kMaxTake) group_max[tid] = 0;
  __syncthreads();
  // packs are counted from the 16-byte boundary at or before the row's start
  const T* const row = static_cast<const T*>(a.logits) + r * a.ld;
  const int skip = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
  const int p0 = piece * z.length, p1 = min(p0 + z.length, (a.V + skip + VEC - 1) / VEC);
  // Whole packs come through a ring of asynchronous copies, each thread reading what it copied
  // itself; packs that reach over the row's ends are read element by element.
  const PackRing<T, VEC> ring(ring_memory, kThreads, tid);
  const int whole0 = skip ? 1 : 0, whole1 = min(p1, (a.V + skip) / VEC);
  constexpr int kTile = kThreads * PACKS;
  auto fetch = [&](int from, int stage) {
    const T* const src = row + (static_cast<int64_t>(from) + tid) * VEC - skip;
    if (from >= whole0 && from + kTile <= whole1) {
#pragma unroll
      for (int i = 0; i < PACKS; ++i) ring.fetch(stage * PACKS + i, src + i * kThreads * VEC);
    } else {
#pragma unroll
      for (int i = 0; i < PACKS; ++i) {
        const int p = from + i * kThreads + tid;
        if (p >= whole0 && p < whole1) ring.fetch(stage * PACKS + i, src + i * kThreads * VEC);
      }
    }
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (p0 + s * kTile < p1) fetch(p0 + s * kTile, s);
    copy_async_commit();
  }
  const float k = steps(a.tau);
  float m = -INFINITY, sum = 0.f;      // of this thread's elements: sum of 2^((x - m) k)
  uint32_t low = kMinusInf;            // what is found lies above it
  int before = 0, stage = 0, turn = 0;   // found in earlier tiles
  for (int from = p0; from < p1; from += kTile) {
    copy_async_wait<kStages - 2>();
    Pack<T, VEC> q[PACKS];
#pragma unroll
    for (int i = 0; i < PACKS; ++i) q[i] = ring.read(stage * PACKS + i);
    if (from < whole0 || from + kTile > whole1) {
#pragma unroll
      for (int i = 0; i < PACKS; ++i) {
        const int p = from + i * kThreads + tid, v = p * VEC - skip;
        if (p >= whole0 && p < whole1) continue;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          q[i].v[e] = p < p1 && v + e >= 0 && v + e < a.V ? row[v + e] : from_f32<T>(-INFINITY);
      }
    }
    const int ahead = from + (kStages - 1) * kTile;
    if (ahead < p1) fetch(ahead, stage == 0 ? kStages - 1 : stage - 1);
    copy_async_commit();
    float tops[PACKS], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PACKS; ++i) {
      tops[i] = largest(q[i]);
      top = fmaxf(top, tops[i]);
    }
    if (from == p0) {
      // the least of the largest elements of `groups` groups of threads: those with the same
      // number modulo that, so that a short tile leaves none empty
      uint32_t least = order_of(top);
      for (int o = 16; o >= groups; o >>= 1) least = max(least, __shfl_xor_sync(0xffffffffu, least, o));
      if (lane < groups) atomicMax(&group_max[tid & (groups - 1)], least);
      __syncthreads();
      least = ~0u;
      for (int g = lane; g < groups; g += 32) least = min(least, group_max[g]);
      least = __reduce_min_sync(0xffffffffu, least);
      low = max(least - 1, kMinusInf);
      low -= low == kMinusZero;      // not below zero, as a number
    }
    const float above = from_order(low);
    const float to = fmaxf(m, top), base = to == -INFINITY ? 0.f : to;
    const float shrink = ex2_approx((m - base) * k);
    // a tile's sum starts from zero: equal terms added to one long sum would all be rounded the
    // same way (1,000 rows of 151,936 equal logits below one: lse off by 1.6e-5)
    float2 sums = make_float2(0.f, 0.f);
    m = to;
    const float2 down = make_float2(-base, -base), kk = make_float2(k, k);
#pragma unroll
    for (int i = 0; i < PACKS; ++i)
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) {
        const float2 d = mul2(add2(pair_of(q[i], e), down), kk);
        sums = add2(sums, make_float2(ex2_approx(d.x), ex2_approx(d.y)));
      }
    sum = sum * shrink + (sums.x + sums.y);
    if (top > above) {
#pragma unroll
      for (int i = 0; i < PACKS; ++i) {
        if (!(tops[i] > above)) continue;
        const int v = (from + i * kThreads + tid) * VEC - skip;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float x = to_f32(q[i].v[e]);
          if (x > above) {
            const int n = before + atomicAdd(&added[turn], 1);
            if (n < kRoom) found[n] = entry_of(order_of(x), v + e);
          }
        }
      }
    }
    __syncthreads();
    int n = before + added[turn];
    if (tid == 0) added[turn == 0 ? 2 : turn - 1] = 0;
    turn = turn == 2 ? 0 : turn + 1;
    if (n > kRoom) {
      n = keep_best(found, before, a.take);
      if (tid == 0) n_best = n;
      __syncthreads();
      add_best_of_tile<T, PACKS>(found, &n_best, scratch, row, from, p1, skip, a.V, low, a.take);
      n = n_best;       // 2 take at most
    }
    if (from == p0 || n > 2 * a.take + 16) {
      n = keep_best(found, n, a.take);
      // later elements have higher ids: those equal to the last one kept come behind it
      if (n == a.take) low = static_cast<uint32_t>(found[n - 1] >> 32);
    }
    before = n;
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
  copy_async_wait<0>();
  const float most = warp_max(m), at = most == -INFINITY ? 0.f : most;
  sum = warp_sum(sum * ex2_approx((m - at) * k));
  if (lane == 0) warp_sums[warp] = make_float2(most, sum);
  const int n = keep_best(found, before, a.take);
  const int64_t slot = r * z.pieces + piece;
  uint64_t* const out = z.best + slot * a.take;
  for (int i = tid; i < a.take; i += kThreads) out[i] = i < n ? found[i] : 0;
  if (tid == 0) {
    float top = -INFINITY, s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, warp_sums[w].x);
    const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += warp_sums[w].y * ex2_approx((warp_sums[w].x - from) * k);
    // a NaN is in the sum, and an infinity minus itself is one
    z.stats[slot] = s != s ? make_float2(NAN, NAN) : make_float2(top, s);
  }
}

// ------------------------------------------------------------------ the group's best
enum : uint8_t { kLive, kEnded, kNone };   // a beam; kNone offers nothing

// Different logits may share a 64-bit score (a large temperature or score): one beam's then
// stay in the order that chose the best of its pieces, so that the pieces do not matter.
struct Ranked {
  uint64_t score;  // an integer that grows with the 64-bit score (comparing those themselves
                   // is slow here: 600 candidates took 190 us)
  uint64_t entry;  // entry_of the logit and its id v
  int64_t beam;    // j
};

__device__ __forceinline__ uint64_t order_of(double x) {
  const int64_t u = __double_as_longlong(x + 0.0);
  return static_cast<uint64_t>(u ^ ((u >> 63) | static_cast<int64_t>(uint64_t{1} << 63)));
}
__device__ __forceinline__ double from_order(uint64_t k) {
  return __longlong_as_double(static_cast<int64_t>(k >> 63 ? k ^ (uint64_t{1} << 63) : ~k));
}

__device__ __forceinline__ bool first_of_equals(const Ranked& x, const Ranked& y) {
  return x.beam < y.beam || (x.beam == y.beam && x.entry > y.entry);
}
__device__ __forceinline__ bool ahead(const Ranked& x, const Ranked& y) {
  return x.score > y.score || (x.score == y.score && first_of_equals(x, y));
}

// inv = 1 / tau, formed by the host: a 64-bit division by every thread here takes 4 us.
__global__ void __launch_bounds__(kBestThreads) best_kernel(BeamSelect a, Pieces z, double inv) {
  __shared__ Ranked found[kRoom];
  // lse = top / tau + log s, so score(j, v) = (score_j - log s) + (x_v - top) / tau: a row
  // whose logits are all near the type's lowest value keeps its differences
  __shared__ double bias[kMaxBeams];       // score - log s of each beam
  __shared__ float rough[kMaxBeams];       // the same in fp32
  __shared__ float tops[kMaxBeams];
  __shared__ uint8_t kind[kMaxBeams];
  __shared__ int n_found;
  __shared__ Ranked warp_best[kBestWarps], last;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int64_t g = blockIdx.x, r0 = g * a.beams;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) n_found = 0;
  for (int j = warp; j < a.beams; j += kBestWarps) {
    const int64_t r = r0 + j;
    const float score = a.scores[r];
    const bool ended = a.finished && a.finished[r];
    double log_s = 0.0;
    float m = -INFINITY;
    bool bad = false;
    if (!ended) {
      const float2* const st = z.stats + r * z.pieces;
      for (int i = lane; i < z.pieces; i += 32) {
        const float x = st[i].x;
        bad |= x != x;
        m = fmaxf(m, x);
      }
      m = warp_max(m);
      bad = __any_sync(0xffffffffu, bad);
      double s = 0.0;
      const float k = steps(a.tau);
      if (m > -INFINITY)
        for (int i = lane; i < z.pieces; i += 32) s += st[i].y * ex2_approx((st[i].x - m) * k);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      // log s = e log 2 + log f with f in [1, 2): only the small part in fp32
      int e;
      const float near = static_cast<float>(s), f = 2.f * frexpf(near, &e);
      const float rest = static_cast<float>(s - static_cast<double>(near)) / near;
      log_s = (e - 1) * 0.6931471805599453 + static_cast<double>(logf(f) + rest);
    }
    if (lane == 0) {
      const bool none = !ended && (bad || m == -INFINITY);
      if (a.lse) {
        const double lse = ended ? 0.0 : bad ? static_cast<double>(NAN)
                                             : m == -INFINITY ? static_cast<double>(m) : static_cast<double>(m) * inv + log_s;
        a.lse[r] = static_cast<float>(lse);
      }
      bias[j] = static_cast<double>(score) - log_s;
      rough[j] = static_cast<float>(bias[j]);
      tops[j] = m;
      kind[j] = none || !isfinite(score) ? kNone : ended ? kEnded : kLive;
    }
  }
  __syncthreads();
  const unsigned lists = static_cast<unsigned>(a.beams) * z.pieces;    // of `take` entries in falling order
  const unsigned more_places = kBestThreads / lists, more_lists = kBestThreads % lists;    // of a thread's next entry
  const int total = static_cast<int>(lists) * a.take;
  const float inv_f = static_cast<float>(inv);
  // an entry's score in fp32 and a bound of its error: a rounding of the difference, of
  // 1 / tau, of the product, of the beam's part and of the sums
  auto estimate = [&](int j, uint32_t order, float& err) {
    const float x = (from_order(order) - tops[j]) * inv_f, b = rough[j], f = x + b;
    err = 4.0e-7f * (fabsf(x) + fabsf(b)) + 1e-37f;   // 6.7 roundings; six are met
    return f;
  };
  // The first entry of every list, then the second of every list ...: the threads' first ones are the
  // largest, whose `take`-th sorts out nearly all of the others.  (List by list, a thread would
  // meet one place of every list where `take` divides the threads: 64 beams of 50,257 and 128 of
  // them left 6,400 entries, more than fit, and took 10.6 ms.)
  auto each = [&](auto&& f) {
    constexpr int kAhead = 8;        // entries in flight per thread
    const uint64_t* const entries = z.best + r0 * z.pieces * a.take;
    unsigned place = tid / lists, list = tid - place * lists;
    for (int i0 = tid; i0 < total; i0 += kAhead * kBestThreads) {
      uint64_t e[kAhead];
      unsigned of[kAhead];           // which list
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        e[q] = i0 + q * kBestThreads < total ? entries[list * a.take + place] : 0;
        of[q] = list;
        place += more_places;
        list += more_lists;
        if (list >= lists) {
          list -= lists;
          ++place;
        }
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (e[q] == 0) continue;
        const int j = static_cast<int>(of[q] / z.pieces);
        // an ended beam's entries were not written
        if (kind[j] == kLive) f(j, static_cast<uint32_t>(e[q] >> 32), static_cast<int>(~static_cast<uint32_t>(e[q])));
      }
    }
  };
  auto exact = [&](int j, uint32_t order, int v) {
    const double x = static_cast<double>(from_order(order)) - static_cast<double>(tops[j]);
    return Ranked{order_of(bias[j] + x * inv), entry_of(order, v), j};
  };
  auto end_of = [&](int j) { return Ranked{order_of(bias[j]), entry_of(0, a.eos), j}; };   // its one candidate
  float low = -INFINITY;
  each([&](int j, uint32_t order, int) {
    float err;
    const float f = estimate(j, order, err);
    low = fmaxf(low, f - err);       // NaN (an overflow) is passed over
  });
  // the take-th largest of the threads' largest lower bounds, bit by bit (0 where fewer
  // threads than that have one)
  const uint32_t key = low > -INFINITY ? order_of(low) : 0;
  uint32_t at_least = 0;
#pragma unroll 1
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t more = at_least | 1u << bit;
    const int n = __syncthreads_count(key >= more);
    if (n >= a.take) at_least = more;
    if (n == a.take) break;          // no tighter than this
  }
  low = at_least ? from_order(at_least) : -INFINITY;
  each([&](int j, uint32_t order, int v) {
    float err;
    const float f = estimate(j, order, err);
    if (f + err < low) return;       // not so where one is NaN
    const int n = atomicAdd(&n_found, 1);
    if (n < kRoom) found[n] = exact(j, order, v);
  });
  if (tid < a.beams && kind[tid] == kEnded) {
    const int n = atomicAdd(&n_found, 1);
    if (n < kRoom) found[n] = end_of(tid);
  }
  __syncthreads();
  auto put = [&](int n, const Ranked& x) {
    const int j = static_cast<int>(x.beam), v = static_cast<int>(~static_cast<uint32_t>(x.entry));
    const int64_t o = g * a.take + n;
    a.out_scores[o] = static_cast<float>(from_order(x.score));
    a.parents[o] = static_cast<int32_t>(r0 + j);
    a.tokens[o] = v;
    if (a.next_finished) a.next_finished[o] = kind[j] == kEnded || v == a.eos;
  };
  int n = n_found;
  if (n <= kRoom) {
    for (int i = tid; i < n; i += kBestThreads) {
      const Ranked me = found[i];
      int rank = 0, equals = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        const uint64_t s = found[j].score;
        rank += s > me.score;
        equals += s == me.score;
      }
      if (equals > 1)
        for (int j = 0; j < n; ++j) rank += found[j].score == me.score && first_of_equals(found[j], me);
      if (rank < a.take) put(rank, me);
    }
  } else {
    // more than fit (equal scores): one after the other, the first behind the last one put
    n = a.take;
    if (tid == 0) last = Ranked{~uint64_t{0}, 0, -1};
    for (int t = 0; t < a.take; ++t) {
      __syncthreads();
      const Ranked before = last;
      Ranked mine{0, 0, INT64_MAX};
      auto offer = [&](const Ranked& x) {
        if (ahead(before, x) && ahead(x, mine)) mine = x;
      };
      each([&](int j, uint32_t order, int v) { offer(exact(j, order, v)); });
      if (tid < a.beams && kind[tid] == kEnded)
        offer(end_of(tid));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const Ranked x{__shfl_xor_sync(0xffffffffu, mine.score, o), __shfl_xor_sync(0xffffffffu, mine.entry, o),
                       __shfl_xor_sync(0xffffffffu, mine.beam, o)};
        if (ahead(x, mine)) mine = x;
      }
      if (lane == 0) warp_best[warp] = mine;
      __syncthreads();
      if (tid == 0) {
        for (int w = 0; w < kBestWarps; ++w)
          if (ahead(warp_best[w], mine)) mine = warp_best[w];
        last = mine;
        put(t, mine);
      }
    }
  }
  for (int i = n + tid; i < a.take; i += kBestThreads) {
    const int64_t o = g * a.take + i;
    a.out_scores[o] = -INFINITY;
    a.parents[o] = -1;
    a.tokens[o] = -1;
    if (a.next_finished) a.next_finished[o] = 0;
  }
}

// ------------------------------------------------------------------ states
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;
constexpr int kMoveShared = 32768;    // bytes of a group's rows that a CTA of across_in_place_kernel holds

// Threads along the contiguous bytes (a power of two) and along `mid`.
struct Tile {
  int across;           // threads along inner
  int64_t parts;        // CTAs along inner
  int64_t mids;         // CTAs along mid
  int bytes;            // of a row per CTA (across_in_place_kernel)
};

// What a CTA moves.  All counts are below 2^31, as the number of CTAs is; 64-bit divisions
// would cost a thread more than its copy.
struct Place {
  int64_t part, m, r, o;
};
__device__ __forceinline__ Place place_of(const Tile& t, int64_t rows, int& x) {
  const unsigned parts = static_cast<unsigned>(t.parts), mids = static_cast<unsigned>(t.mids),
                 count = static_cast<unsigned>(rows), across = static_cast<unsigned>(t.across);
  unsigned b = blockIdx.x;
  Place p;
  p.part = b % parts;
  b /= parts;
  const unsigned mid = b % mids;
  b /= mids;
  p.r = b % count;
  p.o = b / count;
  x = static_cast<int>(threadIdx.x & (across - 1));       // a power of two
  p.m = static_cast<int64_t>(mid) * (kMoveThreads / across) + threadIdx.x / across;
  return p;
}

// kAligned: every row of both sides starts on a 16-byte boundary.  Otherwise 16-byte stores are
// counted from the first boundary of dst's row, and what they store lies across two blocks of
// src's; the bytes before, behind and beside the ends go one by one.
template <bool kAligned>
__global__ void __launch_bounds__(kMoveThreads) gather_kernel(BeamReorder a, Tile t) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  int x;
  const Place at = place_of(t, a.rows, x);
  const int from = a.parents[at.r];
  const bool none = from < 0 || from >= a.src_rows;
  if ((none && !a.clear) || at.m >= a.mid) return;
  const char* const src = a.src + at.o * a.src_outer + (none ? 0 : from * a.src_row) + at.m * a.src_mid;
  char* const dst = a.dst + at.o * a.dst_outer + at.r * a.dst_row + at.m * a.dst_mid;
  const int64_t head = kAligned ? 0 : min(static_cast<int64_t>(-reinterpret_cast<intptr_t>(dst) & 15), a.inner);
  const int64_t n = (a.inner - head) / 16, i0 = at.part * t.across * kMoveUnroll + x;
  uint4 q[kMoveUnroll];
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u) {
    const int64_t i = i0 + u * t.across;
    q[u] = make_uint4(0u, 0u, 0u, 0u);
    if (none || i >= n) continue;
    if (kAligned)
      q[u] = reinterpret_cast<const uint4*>(src)[i];
    else if (i > 0 && i + 2 <= n)
      q[u] = load_across(src + head + i * 16);
    else
      for (int e = 0; e < 16; ++e) reinterpret_cast<char*>(&q[u])[e] = src[head + i * 16 + e];
  }
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u)
    if (i0 + u * t.across < n) reinterpret_cast<uint4*>(dst + head)[i0 + u * t.across] = q[u];
  if (i0 == 0) {
    for (int64_t e = 0; e < head; ++e) dst[e] = none ? 0 : src[e];
    for (int64_t e = head + n * 16; e < a.inner; ++e) dst[e] = none ? 0 : src[e];
  }
}

// Group of `a.beams` rows: from[j] = the row that row j takes over, -1: it stays.
__device__ __forceinline__ bool find_moves(const BeamReorder& a, int64_t r0, int* from, int* moving) {
  if (threadIdx.x == 0) *moving = 0;
  __syncthreads();
  if (threadIdx.x < kMaxBeams) {
    int f = -1;
    if (threadIdx.x < a.beams) {
      const int64_t p = a.parents[r0 + threadIdx.x] - r0;
      if (p >= 0 && p < a.beams && p != threadIdx.x) f = static_cast<int>(p);
    }
    from[threadIdx.x] = f;
    if (f >= 0) *moving = 1;
  }
  __syncthreads();
  return *moving != 0;
}

// Bytes [at, end) of a group's rows, one after the other.
template <int BEAMS>
__device__ __noinline__ void move_bytes(char* at, char* end, int64_t stride, const int* from) {
  for (; at < end; ++at) {
    char c[BEAMS];
#pragma unroll
    for (int j = 0; j < BEAMS; ++j)
      if (from[j] >= 0) c[j] = at[from[j] * stride];
#pragma unroll
    for (int j = 0; j < BEAMS; ++j)
      if (from[j] >= 0) at[j * stride] = c[j];
  }
}

// Rows on 16-byte boundaries: BEAMS >= a.beams rows of a group, 16 bytes of each per thread.
template <int BEAMS>
__global__ void __launch_bounds__(kMoveThreads, BEAMS <= 4 ? 6 : BEAMS <= 8 ? 4 : 2) in_place_kernel(BeamReorder a, Tile t) {
  __shared__ int from[kMaxBeams], moving;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  int x;
  const Place at = place_of(t, a.rows / a.beams, x);
  if (!find_moves(a, at.r * a.beams, from, &moving) || at.m >= a.mid) return;
  char* const row = a.dst + at.o * a.dst_outer + at.r * a.beams * a.dst_row + at.m * a.dst_mid;
  const int64_t n = a.inner / 16, i = at.part * t.across + x;
  if (i == 0 && n * 16 < a.inner) move_bytes<BEAMS>(row + n * 16, row + a.inner, a.dst_row, from);
  if (i >= n) return;
  uint4 q[BEAMS];
#pragma unroll
  for (int j = 0; j < BEAMS; ++j)
    if (from[j] >= 0) q[j] = *reinterpret_cast<const uint4*>(row + i * 16 + from[j] * a.dst_row);
#pragma unroll
  for (int j = 0; j < BEAMS; ++j)
    if (from[j] >= 0) *reinterpret_cast<uint4*>(row + i * 16 + j * a.dst_row) = q[j];
}

// Any alignment, or more rows than registers hold: `t.bytes` of each row that moves go to shared
// memory, where a row keeps its source's place within 16 bytes, and from there to their
// place, 16 bytes at a time from the destination's first boundary on.
__global__ void __launch_bounds__(kMoveThreads) across_in_place_kernel(BeamReorder a, Tile t) {
  extern __shared__ __align__(16) char held[];
  __shared__ int from[kMaxBeams], moving;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  int x;
  const Place at = place_of(t, a.rows / a.beams, x);     // t.across is kMoveThreads
  if (!find_moves(a, at.r * a.beams, from, &moving)) return;
  char* const row = a.dst + at.o * a.dst_outer + at.r * a.beams * a.dst_row + at.m * a.dst_mid + at.part * t.bytes;
  const int bytes = static_cast<int>(min(static_cast<int64_t>(t.bytes), a.inner - at.part * t.bytes));
  const int room = t.bytes + 32, blocks = t.bytes / 16 + 2;
  for (int f = threadIdx.x; f < a.beams * blocks; f += kMoveThreads) {
    const int j = f / blocks, i = f % blocks;
    if (from[j] < 0) continue;
    const char* const src = row + from[j] * a.dst_row;
    const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15u);
    const int first = i * 16 - phase;       // of the row's bytes
    char* const to = held + j * room + i * 16;
    if (first >= 0 && first + 16 <= bytes)
      *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(src + first);
    else
      for (int e = max(0, -first); e < 16 && first + e < bytes; ++e) to[e] = src[first + e];
  }
  __syncthreads();
  for (int f = threadIdx.x; f < a.beams * blocks; f += kMoveThreads) {
    const int j = f / blocks, i = f % blocks;
    if (from[j] < 0) continue;
    char* const dst = row + j * a.dst_row;
    const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(row + from[j] * a.dst_row) & 15u);
    const int first = i * 16 - static_cast<int>(reinterpret_cast<uintptr_t>(dst) & 15u);
    const char* const src = held + j * room + phase + first;
    if (first >= 0 && first + 16 <= bytes)      // the second block read may lie behind the row's bytes, inside its room
      *reinterpret_cast<uint4*>(dst + first) = load_across(src);
    else
      for (int e = max(0, -first); e < 16 && first + e < bytes; ++e) dst[first + e] = src[e];
  }
}

bool aligned_rows(const BeamReorder& a) {
  const uint64_t bits = reinterpret_cast<uintptr_t>(a.src) | reinterpret_cast<uintptr_t>(a.dst) |
                        static_cast<uint64_t>(a.src_outer | a.dst_outer | a.src_row | a.dst_row | a.src_mid |
                                              a.dst_mid);
  return (bits & 15) == 0;
}

// The tile and the number of CTAs.
Tile tile_of(const BeamReorder& a, double& ctas) {
  const bool in_place = a.src == a.dst;
  Tile t{};
  if (in_place && (!aligned_rows(a) || a.beams > 16)) {
    t.across = kMoveThreads;
    t.bytes = kMoveShared / a.beams / 16 * 16 - 32;
    if (t.bytes > 4096) t.bytes = 4096;
    t.parts = (a.inner + t.bytes - 1) / t.bytes;
    t.mids = a.mid;
  } else {
    const int64_t n = (a.inner + 15) / 16, each = in_place ? 1 : kMoveUnroll;
    t.across = 1;
    while (t.across < kMoveThreads && t.across * each < n) t.across *= 2;
    t.parts = (n + t.across * each - 1) / (t.across * each);
    const int down = kMoveThreads / t.across;
    t.mids = (a.mid + down - 1) / down;
  }
  ctas = static_cast<double>(t.parts) * static_cast<double>(t.mids) * static_cast<double>(a.outer) *
         static_cast<double>(in_place ? a.rows / a.beams : a.rows);
  return t;
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

// Pieces of a row: several tiles each where rows alone nearly fill the GPU, one short tile
// each where they do not.  A row that starts off a 16-byte boundary spreads over up to one
// pack more.
template <typename T>
Pieces plan(int64_t R, int V, int& elements) {
  constexpr int VEC = kVec<T>;
  const int64_t packs = (static_cast<int64_t>(V) + 2 * VEC - 2) / VEC;
  auto tiles = [&](int elems) { return (packs * VEC + kThreads * elems - 1) / (static_cast<int64_t>(kThreads) * elems); };
  elements = R * tiles(kManyElements<T>) >= kManyTiles ? kManyElements<T> : kFewElements;
  int64_t pieces = tiles(elements);
  if (elements != kFewElements) {
    const int64_t most = R < kManyPieces ? kManyPieces / R : 1;
    pieces = pieces < most ? pieces : most;
  }
  Pieces z{};
  z.length = static_cast<int>((packs + pieces - 1) / pieces);
  z.pieces = static_cast<int>((packs + z.length - 1) / z.length);
  return z;
}

template <typename F>
auto by_type(int type, F&& f) {
  switch (type) {
    case kF32: return f(float{});
    case kBF16: return f(__nv_bfloat16{});
    default: return f(__half{});
  }
}

}  // namespace

size_t beam_workspace(int64_t R, int V, int take) {
  size_t most = 0;
  for (const int type : {kF32, kBF16}) {
    const size_t n = by_type(type, [&](auto t) {
      int elements;
      const size_t slots = static_cast<size_t>(R) * plan<decltype(t)>(R, V, elements).pieces;
      return round_up(slots * sizeof(float2)) + slots * sizeof(uint64_t) * take;
    });
    most = n > most ? n : most;
  }
  return most > 256 ? most : 256;
}

cudaError_t launch_beam_select(const BeamSelect& a, cudaStream_t s) {
  int elements = 0;
  Pieces z = by_type(a.type, [&](auto t) { return plan<decltype(t)>(a.R, a.V, elements); });
  const size_t slots = static_cast<size_t>(a.R) * z.pieces;      // below 2^31: see plan
  z.stats = static_cast<float2*>(a.workspace);
  z.best = reinterpret_cast<uint64_t*>(static_cast<char*>(a.workspace) + round_up(slots * sizeof(float2)));
  int groups = 8;      // of threads, a power of two and at least `take` of them
  while (groups < a.take) groups *= 2;
  cudaError_t e = traced_launch("beam_select_scan", s, [&] {
    return by_type(a.type, [&](auto t) {
      using T = decltype(t);
      if (elements == kFewElements)
        return launch_dependent(scan_kernel<T, kFewElements>, dim3(static_cast<unsigned>(slots)), kThreads,
                                kRingBytes<T, kFewElements>, 1, s, a, z, groups);
      static std::atomic<int> ready[64];
      constexpr size_t ring = kRingBytes<T, kManyElements<T>>;
      const cudaError_t r = allow_shared(ready, reinterpret_cast<const void*>(scan_kernel<T, kManyElements<T>>), ring);
      if (r != cudaSuccess) return r;
      return launch_dependent(scan_kernel<T, kManyElements<T>>, dim3(static_cast<unsigned>(slots)), kThreads, ring, 1, s, a,
                              z, groups);
    });
  });
  if (e != cudaSuccess) return e;
  return traced_launch("beam_select_best", s, [&] {
    return launch_dependent(best_kernel, dim3(static_cast<unsigned>(a.R / a.beams)), kBestThreads, 0, 1, s, a, z,
                            1.0 / static_cast<double>(a.tau));
  });
}

bool beam_reorder_fits(const BeamReorder& a) {
  double ctas = 0;
  tile_of(a, ctas);
  return ctas <= 2147483647.0;
}

cudaError_t launch_beam_reorder(const BeamReorder& a, cudaStream_t s) {
  double ctas = 0;
  const Tile t = tile_of(a, ctas);
  const dim3 grid(static_cast<unsigned>(ctas));
  return traced_launch("beam_reorder", s, [&] {
    const bool aligned = aligned_rows(a);
    if (a.src != a.dst)
      return launch_dependent(aligned ? gather_kernel<true> : gather_kernel<false>, grid, kMoveThreads, 0, 1, s, a, t);
    if (!aligned || a.beams > 16)
      return launch_dependent(across_in_place_kernel, grid, kMoveThreads, static_cast<size_t>(a.beams) * (t.bytes + 32), 1,
                              s, a, t);
    auto kern = a.beams <= 4 ? in_place_kernel<4> : a.beams <= 8 ? in_place_kernel<8> : in_place_kernel<16>;
    return launch_dependent(kern, grid, kMoveThreads, 0, 1, s, a, t);
  });
}

}  // namespace lmh
