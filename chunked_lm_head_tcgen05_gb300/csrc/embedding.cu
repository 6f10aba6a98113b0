// Rows of the vocabulary table by token id, scaled, and their gradient:
//   y_t = s W[id_t]          dW_v (+)= s sum_{t : id_t = v} dy_t
// HBM-bound both ways.
// Forward: one read of the rows (frequent ids come from the L2) and one write of
// y.  A warp takes part of a row, so that few tokens still fill the GPU.
// Backward: the tokens are sorted by id (sort_ids.cu), and a CTA sums the rows of
// kLong (or, for few tokens, kShort) consecutive sorted tokens for its columns, in
// fp32 registers, writing an id's sum when the id ends.  An id whose tokens cross
// from one such segment into the next leaves partial sums, which join_kernel adds
// in order: no atomics, same inputs, same bits.  A dense gradient also needs
// zeros in the rows of ids that do not occur: the SMs that do not sort write the first
// rows meanwhile, and CTAs of the summing launch the rest of them.
// Sums are rounded once, where d_weight is bf16.
#include "element.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace lmh {
namespace {

constexpr int kFwdThreads = 256;
constexpr int kFwdUnroll = 4;
constexpr int kSumThreads = 128;
constexpr int kLong = 32;       // sorted tokens per segment
constexpr int kShort = 8;       // of fewer than kFew tokens
constexpr int kFew = 8192;
constexpr int kFewIds = 1024;   // that one CTA sorts
constexpr size_t kSmallTable = size_t{256} << 20;
constexpr int kFillRows = 16;   // table rows per CTA that writes zeros
constexpr int kJoinThreads = 256;
constexpr int kJoinColumns = 128;
constexpr int kJoinSegments = 32;
constexpr int kJoinShort = 16;

int segment_of(int64_t n) { return n < kFew ? kShort : kLong; }

// ------------------------------------------------------------------ forward
// VEC elements of W become VEC of y.
template <typename W, typename Y, int VEC>
__device__ __forceinline__ Pack<Y, VEC> scaled(const Pack<W, VEC>& q, float scale) {
  Pack<Y, VEC> r;
  if constexpr (VEC == 1) {
    r.v[0] = from_f32<Y>(to_f32(q.v[0]) * scale);
  } else {
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const float2 x = pair_of(q, e);
      set_pair(r, e, make_float2(x.x * scale, x.y * scale));
    }
  }
  return r;
}

// Any alignment.  A warp handles `span` packs of one row: work item = (row, part of the row);
// bound by instructions (60,000 x 1,111 bf16: 65 us, 4.1 TB/s).
template <typename W, typename Y>
__global__ void __launch_bounds__(kFwdThreads) embed_kernel(EmbedFwd a, int parts, int span) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr int VEC = kVec<W>;
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kFwdThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = item / parts;
  const int part = static_cast<int>(item % parts);
  if (t >= a.N) return;
  int id = a.ids[t];
  if (id < 0) id += a.V;
  Y* const dst = static_cast<Y*>(a.y) + t * a.y_ld;
  // columns are counted in packs from the first 16-byte boundary of the result
  const int head = min(to_boundary(dst), a.H);
  const int packs = (a.H - head) / VEC;
  if (id < 0 || id >= a.V) {   // an id that the table does not have
    const Y bad = from_f32<Y>(NAN);
    for (int c = part * 32 + lane; c < a.H; c += parts * 32) dst[c] = bad;
    return;
  }
  const W* const src = static_cast<const W*>(a.weight) + id * a.w_ld;
  if (part == 0) {
    for (int c = lane; c < head; c += 32) dst[c] = from_f32<Y>(to_f32(src[c]) * a.scale);
  }
  if (part == parts - 1) {
    for (int c = head + packs * VEC + lane; c < a.H; c += 32)
      dst[c] = from_f32<Y>(to_f32(src[c]) * a.scale);
  }
  const int from = part * span, to = min(from + span, packs);
  const bool across = (reinterpret_cast<uintptr_t>(src + head) & 15u) != 0;
  for (int p0 = from; p0 < to; p0 += 32 * kFwdUnroll) {
    Pack<W, VEC> q[kFwdUnroll];
#pragma unroll
    for (int u = 0; u < kFwdUnroll; ++u) {
      const int p = p0 + u * 32 + lane;
      if (p >= to) continue;
      const W* const at = src + head + p * VEC;
      if (!across) {
        q[u] = *reinterpret_cast<const Pack<W, VEC>*>(at);
      } else if (p > 0 && p + 2 <= packs) {   // both blocks lie inside the row
        const uint4 w = load_across(at);
        q[u] = *reinterpret_cast<const Pack<W, VEC>*>(&w);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) q[u].v[e] = at[e];
      }
    }
#pragma unroll
    for (int u = 0; u < kFwdUnroll; ++u) {
      const int p = p0 + u * 32 + lane;
      if (p < to) *reinterpret_cast<Pack<Y, VEC>*>(dst + head + p * VEC) = scaled<W, Y>(q[u], a.scale);
    }
  }
}

// Rows of whole 16-byte packs on both sides: the packs of all rows as one list, a thread every
// kFwdThreads-th of a CTA's UNROLL * kFwdThreads, so that short rows fill it too (60,000 x 64
// fp16: 16 us with a warp per row, 6 so).  65,536 x 2,560 bf16: 85 us, 5.9 TB/s.
template <typename W, typename Y, int UNROLL>
__global__ void __launch_bounds__(kFwdThreads) embed_packs_kernel(EmbedFwd a, unsigned packs) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr int VEC = kVec<W>;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * UNROLL * kFwdThreads;
  const int64_t t0 = first / packs;
  const unsigned p0 = static_cast<unsigned>(first - t0 * packs) + threadIdx.x;
  Pack<W, VEC> q[UNROLL];
  Y* dst[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const unsigned f = p0 + u * kFwdThreads, down = f / packs, p = f - down * packs;
    const int64_t t = t0 + down;
    dst[u] = nullptr;
    if (t >= a.N) continue;
    int id = a.ids[t];
    if (id < 0) id += a.V;
    dst[u] = static_cast<Y*>(a.y) + t * a.y_ld + p * VEC;
    if (id >= 0 && id < a.V) {
      q[u] = *reinterpret_cast<const Pack<W, VEC>*>(static_cast<const W*>(a.weight) + id * a.w_ld + p * VEC);
    } else {      // an id that the table does not have
#pragma unroll
      for (int e = 0; e < VEC; ++e) q[u].v[e] = from_f32<W>(NAN);
    }
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u)
    if (dst[u]) *reinterpret_cast<Pack<Y, VEC>*>(dst[u]) = scaled<W, Y>(q[u], a.scale);
}

// ------------------------------------------------------------------ backward
struct Sorted {
  int* live;
  int32_t* keys;
  int32_t* pos;
  float* part;      // [segments][2][H]: sums that began before the segment, and that go on after it
  int segments;
  int filled;       // rows of d_weight that are zero already, a multiple of kFillRows
};

// Zeros in the rows [v0, v0 + kFillRows) of ids that do not occur; the rows before
// z.filled got theirs beside the sort.
template <typename O>
__device__ void fill_zeros(const EmbedBwd& a, const Sorted& z, int64_t v0) {
  __shared__ int absent[kFillRows];
  const int rows = static_cast<int>(min(static_cast<int64_t>(kFillRows), a.V - v0));
  const int live = *z.live;
  if (threadIdx.x < rows) {
    const int v = static_cast<int>(v0) + threadIdx.x;
    int lo = 0, hi = live;     // first place whose key is not below v
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (z.keys[mid] < v) lo = mid + 1; else hi = mid;
    }
    absent[threadIdx.x] = lo == live || z.keys[lo] != v;
  }
  __syncthreads();
  constexpr int VEC = kVec<O>;
  for (int r = 0; r < rows;) {
    if (!absent[r]) {
      ++r;
      continue;
    }
    int end = r + 1;       // rows next to each other are one stretch of memory
    while (end < rows && absent[end]) ++end;
    O* const dst = static_cast<O*>(a.d_weight) + (v0 + r) * a.H;
    const int64_t n = static_cast<int64_t>(end - r) * a.H;
    const int64_t head = min(static_cast<int64_t>(to_boundary(dst)), n), packs = (n - head) / VEC;
    if (threadIdx.x < head) dst[threadIdx.x] = from_f32<O>(0.f);
#pragma unroll 4
    for (int64_t p = threadIdx.x; p < packs; p += kSumThreads)
      *reinterpret_cast<uint4*>(dst + head + p * VEC) = make_uint4(0u, 0u, 0u, 0u);
    const int64_t c = head + packs * VEC + threadIdx.x;
    if (c < n) dst[c] = from_f32<O>(0.f);
    r = end;
  }
}

// sum * scale into (or onto) one row of the gradient.
template <typename O, int VEC>
__device__ __forceinline__ void put(O* dst, const float (&sum)[VEC], float scale, int accumulate) {
  if constexpr (VEC == 1) {
    *dst = from_f32<O>(accumulate ? to_f32(*dst) + sum[0] * scale : sum[0] * scale);
  } else {
    Pack<O, VEC>* const p = reinterpret_cast<Pack<O, VEC>*>(dst);
    Pack<O, VEC> q;
    if (accumulate) q = *p;
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      float2 x = make_float2(sum[2 * e] * scale, sum[2 * e + 1] * scale);
      if (accumulate) {
        const float2 old = pair_of(q, e);
        x = make_float2(old.x + x.x, old.y + x.y);
      }
      set_pair(q, e, x);
    }
    *p = q;
  }
}

// CTAs below segments * chunks: (segment, columns); those behind write zeros.  Bound by HBM:
// 65,536 x 2,560 bf16 into a bf16 gradient of 151,936 rows 141 us, 6.6 TB/s.
template <typename D, typename O, int VEC>
__global__ void __launch_bounds__(kSumThreads, VEC == 1 ? 12 : 8) sum_kernel(EmbedBwd a, Sorted z, int64_t first, int seg,
                                                          int chunks) {
  // rows in flight per thread: eight packs hold registers that more threads use better (170 us
  // where four take 149, 65,536 x 2,560 bf16)
  constexpr int kBatch = VEC == 1 ? 8 : 4;
  __shared__ int key[kLong], pos[kLong];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const unsigned summing = static_cast<unsigned>(z.segments) * chunks;
  if (blockIdx.x >= summing) {
    fill_zeros<O>(a, z, z.filled + static_cast<int64_t>(blockIdx.x - summing) * kFillRows);
    return;
  }
  const int sgm = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int live = *z.live, at = sgm * seg, n = min(seg, live - at);
  if (n <= 0) return;
  if (threadIdx.x < n) {
    key[threadIdx.x] = z.keys[at + threadIdx.x];
    pos[threadIdx.x] = z.pos[at + threadIdx.x];
  }
  __syncthreads();
  const int c = (chunk * kSumThreads + threadIdx.x) * VEC;
  if (c >= a.H) return;
  const bool from_before = at > 0 && z.keys[at - 1] == key[0];
  const bool goes_on = at + n < live && z.keys[at + n] == key[n - 1];
  float* const part = z.part + static_cast<int64_t>(sgm) * 2 * a.H + c;
  const D* const dy = static_cast<const D*>(a.dy) + first * a.dy_ld + c;
  O* const out = static_cast<O*>(a.d_weight) + c;
  float sum[VEC] = {};
  auto keep = [&](float* p) {
    Pack<float, VEC> q;
#pragma unroll
    for (int e = 0; e < VEC; ++e) q.v[e] = sum[e];
    *reinterpret_cast<Pack<float, VEC>*>(p) = q;
  };
  bool began = !from_before;    // the id at hand began in this segment
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    Pack<D, VEC> q[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (i0 + u < n)
        q[u] = *reinterpret_cast<const Pack<D, VEC>*>(dy + pos[i0 + u] * a.dy_ld);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u;
      if (i >= n) continue;
      if (i > 0 && key[i] != key[i - 1]) {
        if (began)
          put<O, VEC>(out + static_cast<int64_t>(key[i - 1]) * a.H, sum, a.scale, a.accumulate);
        else
          keep(part);
        began = true;
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum[e] += to_f32(q[u].v[e]);
    }
  }
  if (!began)
    keep(part);
  else if (goes_on)
    keep(part + a.H);
  else
    put<O, VEC>(out + static_cast<int64_t>(key[n - 1]) * a.H, sum, a.scale, a.accumulate);
}

// Ids that cross segments: the segment where such an id begins holds its first sum, the
// following ones the rest.  Grid (kJoinSegments segments, kJoinColumns columns).  A warp
// adds an id of up to kJoinShort segments more; longer ones take the whole CTA, its warps
// consecutive parts of the id's segments, whose sums are then added in order.
// One id after the other by the whole CTA, its end found by bisection, took 70 us for
// 65,536 tokens of 2,560 columns, most of them waiting for a few rows; this takes 13.
template <typename O>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(EmbedBwd a, Sorted z, int seg) {
  constexpr int kWarps = kJoinThreads / 32, kEach = kJoinColumns / 32;
  __shared__ uint32_t todo;
  __shared__ int rests[kJoinSegments];
  __shared__ float sums[kWarps][kJoinColumns];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int live = *z.live, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg0 = blockIdx.x * kJoinSegments;
  if (warp == 0) {
    const int64_t at = static_cast<int64_t>(seg0 + lane) * seg, next = at + seg;
    bool owns = false;
    if (next < live) {
      const int before = at > 0 ? z.keys[at - 1] : -1, first = z.keys[at], key = z.keys[next - 1], after = z.keys[next];
      owns = after == key && !(first == key && before == key);
    }
    const uint32_t b = __ballot_sync(0xffffffffu, owns);
    if (lane == 0) todo = b;
  }
  __syncthreads();
  if (todo == 0) return;
  const int last_segment = (live - 1) / seg, c0 = blockIdx.y * kJoinColumns + lane;
  auto partial = [&](int sgm, int which, float (&sum)[kEach]) {
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (c0 + 32 * e < a.H) sum[e] += z.part[(static_cast<int64_t>(sgm) * 2 + which) * a.H + c0 + 32 * e];
  };
  int turn = 0;
  for (uint32_t left = todo; left; left &= left - 1, ++turn) {
    if (turn % kWarps != warp) continue;
    const int bit = __ffs(static_cast<int>(left)) - 1, sgm = seg0 + bit;
    const int key = z.keys[(sgm + 1) * seg - 1];
    // segments behind this one that begin with the id
    int rest = 0;
    for (int from = sgm + 1;; from += 32) {
      const int s = from + lane;
      const bool same = s <= last_segment && z.keys[static_cast<int64_t>(s) * seg] == key;
      const uint32_t b = __ballot_sync(0xffffffffu, same);
      rest += b == 0xffffffffu ? 32 : __ffs(static_cast<int>(~b)) - 1;
      if (b != 0xffffffffu) break;
    }
    if (lane == 0) rests[bit] = rest;
    if (rest > kJoinShort) continue;
    float sum[kEach] = {};
    partial(sgm, 1, sum);
#pragma unroll 4
    for (int i = 1; i <= rest; ++i) partial(sgm + i, 0, sum);
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (c0 + 32 * e < a.H) {
        const float total[1] = {sum[e]};
        put<O, 1>(static_cast<O*>(a.d_weight) + static_cast<int64_t>(key) * a.H + c0 + 32 * e, total, a.scale,
                  a.accumulate);
      }
  }
  __syncthreads();
  for (uint32_t left = todo; left; left &= left - 1) {
    const int bit = __ffs(static_cast<int>(left)) - 1, sgm = seg0 + bit, rest = rests[bit];
    if (rest <= kJoinShort) continue;
    const int key = z.keys[(sgm + 1) * seg - 1];
    const int each = (rest + kWarps - 1) / kWarps;
    const int from = sgm + 1 + warp * each, to = min(from + each, sgm + rest + 1);
    float sum[kEach] = {};
    if (warp == 0) partial(sgm, 1, sum);
#pragma unroll 8
    for (int i = from; i < to; ++i) partial(i, 0, sum);
#pragma unroll
    for (int e = 0; e < kEach; ++e) sums[warp][lane + 32 * e] = sum[e];
    __syncthreads();
    const int c = blockIdx.y * kJoinColumns + threadIdx.x;
    if (threadIdx.x < kJoinColumns && c < a.H) {
      float total[1] = {0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) total[0] += sums[w][threadIdx.x];
      put<O, 1>(static_cast<O*>(a.d_weight) + static_cast<int64_t>(key) * a.H + c, total, a.scale, a.accumulate);
    }
    __syncthreads();
  }
}

template <typename F>
auto by_type(int type, F&& f) {
  switch (type) {
    case kF32: return f(float{});
    case kBF16: return f(__nv_bfloat16{});
    default: return f(__half{});
  }
}

bool whole_packs(const void* p, int64_t ld, int64_t width, size_t size, int vec) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && width % vec == 0;
}

template <typename D, typename O>
cudaError_t launch_sums(const EmbedBwd& a, const Sorted& z, int64_t first, int seg, bool fill, cudaStream_t s) {
  constexpr int VEC = kVec<D>;
  const bool wide = whole_packs(a.dy, a.dy_ld, a.H, sizeof(D), VEC) &&
                    reinterpret_cast<uintptr_t>(a.d_weight) % 16 == 0;
  const int per_cta = kSumThreads * (wide ? VEC : 1);
  const int chunks = (a.H + per_cta - 1) / per_cta;
  const int64_t grid = static_cast<int64_t>(z.segments) * chunks + (fill ? (a.V - z.filled + kFillRows - 1) / kFillRows : 0);
  auto kern = wide ? sum_kernel<D, O, VEC> : sum_kernel<D, O, 1>;
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), kSumThreads, 0, 1, s, a, z, first, seg, chunks);
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

// Bytes of zeros that the SMs beside the sort write meanwhile, at some 5 TB/s.  That is a
// little more than the sort's own time (12 us for 4,096 ids, 30 for 65,536; with these zeros
// 39), which costs nothing as the sums would wait for HBM as well: 65,536 x 2,560 bf16 take
// 207 us in all so, 208 with a third less, 219 without any beside the sort.
size_t sort_time_bytes(int n) { return n <= kFewIds ? 0 : (size_t{25} << 20) + static_cast<size_t>(n) * 2300; }

// Whether everything is cleared beside the sort, also the few rows that are written again: a
// table of this size by one CTA's worth of ids.  1,024 tokens, all beside | by the summing
// launch: 50,257 x 512 bf16 (51 MB) 22 | 32 us, 50,257 x 1,111 fp32 (223 MB) 51 | 56,
// 151,936 x 2,560 bf16 (778 MB) 133 | 129, fp32 254 | 233; 4,096 tokens of the last 362 | 239.
bool all_beside(int n, int V, size_t bytes) { return n <= kFewIds && n <= V / 32 && bytes <= kSmallTable; }

}  // namespace

// Count, sorted ids and positions, partial sums of the segments of one sort.
size_t embed_workspace(int64_t N, int H) {
  const int64_t n = N < kSortMost ? N : kSortMost;
  // a short list has more segments than a long one of somewhat greater length
  const int64_t segments = n < kFew ? (n + kShort - 1) / kShort : (n + kLong - 1) / kLong;
  const int64_t most = n < kFew ? segments : (segments > kFew / kShort ? segments : kFew / kShort);
  return 256 + 2 * round_up(4 * static_cast<size_t>(n)) + 8 * static_cast<size_t>(most) * static_cast<size_t>(H);
}

cudaError_t launch_embed_fwd(const EmbedFwd& a, cudaStream_t s) {
  auto run = [&](auto w, auto y) {
    using W = decltype(w);
    using Y = decltype(y);
    constexpr int VEC = kVec<W>;
    const int packs = (a.H + VEC - 1) / VEC;
    if (whole_packs(a.weight, a.w_ld, a.H, sizeof(W), VEC) && whole_packs(a.y, a.y_ld, a.H, sizeof(Y), VEC)) {
      const int64_t all = a.N * packs;
      const bool few = all < int64_t{304} * kFwdThreads * kFwdUnroll;
      const int64_t each = kFwdThreads * (few ? 1 : kFwdUnroll), ctas = (all + each - 1) / each;
      if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
      auto kern = few ? embed_packs_kernel<W, Y, 1> : embed_packs_kernel<W, Y, kFwdUnroll>;
      return launch_dependent(kern, dim3(static_cast<unsigned>(ctas)), kFwdThreads, 0, 1, s, a, static_cast<unsigned>(packs));
    }
    const int parts = (packs + 32 * kFwdUnroll - 1) / (32 * kFwdUnroll);
    const int span = ((packs + parts - 1) / parts + 31) / 32 * 32;
    const int64_t grid = (a.N * parts + kFwdThreads / 32 - 1) / (kFwdThreads / 32);
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(embed_kernel<W, Y>, dim3(static_cast<unsigned>(grid)), kFwdThreads, 0, 1, s, a, parts, span);
  };
  return by_type(a.type, [&](auto w) {
    using W = decltype(w);
    if (a.y_type == a.type) return run(w, w);
    if constexpr (sizeof(W) == 4) return run(w, __nv_bfloat16{});
    return run(w, float{});
  });
}

cudaError_t launch_embed_bwd(const EmbedBwd& call, cudaStream_t s) {
  EmbedBwd a = call;
  for (int64_t first = 0; first < call.N; first += kSortMost) {
    const int n = static_cast<int>(call.N - first < kSortMost ? call.N - first : kSortMost);
    const int seg = segment_of(n);
    char* p = static_cast<char*>(a.workspace);
    Sorted z;
    z.live = reinterpret_cast<int*>(p);
    z.keys = reinterpret_cast<int32_t*>(p + 256);
    z.pos = reinterpret_cast<int32_t*>(p + 256 + round_up(4 * static_cast<size_t>(n)));
    z.part = reinterpret_cast<float*>(p + 256 + 2 * round_up(4 * static_cast<size_t>(n)));
    z.segments = (n + seg - 1) / seg;
    // what the GPU writes while one cluster sorts
    const size_t row = (a.d_type == kF32 ? 4 : 2) * static_cast<size_t>(a.H);
    const bool beside = !a.accumulate && reinterpret_cast<uintptr_t>(a.d_weight) % 16 == 0;
    size_t rows = beside ? sort_time_bytes(n) / row / kFillRows * kFillRows : 0;
    if (beside && all_beside(n, a.V, row * static_cast<size_t>(a.V))) rows = a.V;
    if (rows > static_cast<size_t>(a.V)) rows = a.V / kFillRows * kFillRows;
    if (rows * row % 16) rows = rows / kFillRows * kFillRows;
    z.filled = static_cast<int>(rows);
    cudaError_t e = traced_launch("embedding_bwd_sort", s, [&] {
      return launch_sort_ids(a.ids + first, n, a.V, true, a.skip, z.keys, z.pos, z.live, s, a.d_weight, rows * row);
    });
    if (e != cudaSuccess) return e;
    e = traced_launch("embedding_bwd", s, [&] {
      return by_type(a.dy_type, [&](auto d) {
        using D = decltype(d);
        return a.d_type == kF32 ? launch_sums<D, float>(a, z, first, seg, !a.accumulate, s)
                                : launch_sums<D, __nv_bfloat16>(a, z, first, seg, !a.accumulate, s);
      });
    });
    if (e != cudaSuccess) return e;
    const dim3 grid((z.segments + kJoinSegments - 1) / kJoinSegments, (a.H + kJoinColumns - 1) / kJoinColumns);
    e = traced_launch("embedding_bwd_join", s, [&] {
      return a.d_type == kF32 ? launch_dependent(join_kernel<float>, grid, kJoinThreads, 0, 1, s, a, z, seg)
                              : launch_dependent(join_kernel<__nv_bfloat16>, grid, kJoinThreads, 0, 1, s, a, z, seg);
    });
    if (e != cudaSuccess) return e;
    a.accumulate = 1;   // what follows is added to the first part's sums
  }
  return cudaSuccess;
}

}  // namespace lmh
