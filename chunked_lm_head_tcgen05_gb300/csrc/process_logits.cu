// Penalties for repeated tokens, biases and grammar masks on logits, and the
// gradient through them.  For row r and id v, with c the occurrences of v in
// the row's outputs and `met` whether v occurs in its prompt or outputs:
//   x1 = met ? (x > 0 ? x / rho : x rho) : x
//   x2 = x1 - (f c + p [c > 0])
//   x3 = x2 + bias_v
//   out = allowed ? x3 : -inf
//   d x = allowed ? (met ? (x > 0 ? 1 / rho : rho) : 1) g : 0
// HBM-bound: one read and one write of the logits (or gradients).
// Forward, two kernels:
//  1. copy_kernel copies the rows, 16 bytes per access, with the mask applied; a
//     copy leaves every allowed element as it was, in its own type.  In place it
//     touches masked packs only, and without a mask it does not run.
//  2. rewrite_kernel, one CTA per row, finds the distinct ids of the row's
//     history and biases, counts them, and rewrites those elements from what the
//     copy left (in L2): in fp32 from the exact logit, rounded once.
// Backward, where only `met` matters, one kernel: grad_kernel, below.
// The distinct ids live in a bitmap over the vocabulary in shared memory.  Ranks
// (set bits before an id) number them without gaps, so counts take four bytes per
// distinct id and not per column, and ascending ranks are ascending columns.
// Integer counts do not depend on the order they are added in.
// One kernel that counted into a table over each CTA's column range before or
// after copying it took 127 to 225 us where these two take 50 (256 rows of
// 151,936 bf16, 5,100 tokens each): every range's CTA reads the row's whole
// history, and clearing and searching a table as large as the vocabulary costs
// more instructions than the copy.
#include "element.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace lmh {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kUnroll = 4;             // 16-byte accesses in flight per thread
constexpr int kMostColumns = 1 << 18;  // per CTA of rewrite_kernel: 32 KB of bitmap, 32 KB of ranks
constexpr int kBatch = 4;              // columns rewritten at a time: their loads first, then their stores
constexpr int kWindow = 4096;          // distinct ids handled at a time
constexpr int kGradThreads = 256;
constexpr int kGradMost = 65536;       // backward: bytes of gradients per CTA, most and
constexpr int kGradLeast = 16384;      // least (shorter rows aside)

// Bits [c, c + n) of a mask row, n <= 32; bits past the row's V are not read.
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* mask, int c, int n, int V) {
  const int w = c >> 5, sh = c & 31;
  uint32_t lo = mask[w];
  if (sh == 0) return lo;
  const uint32_t hi = (sh + n > 32 && ((w + 1) << 5) < V) ? mask[w + 1] : 0u;
  return __funnelshift_r(lo, hi, sh);
}

// A pack that is not read again: the L2 keeps what was written instead, which
// rewrite_kernel reads next.
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_once(const Pack<T, VEC>* p) {
  const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
  return *reinterpret_cast<const Pack<T, VEC>*>(&q);
}

// `on` = one bit per element of the pack: elements whose bit is clear become off.
template <typename T, int VEC>
__device__ __forceinline__ void keep_allowed(Pack<T, VEC>& q, uint32_t on, T off) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (!(on >> e & 1u)) q.v[e] = off;
  } else {
    // two elements per 32-bit word: a 0xffff mask for each bit, one select per word
    uint32_t* w = reinterpret_cast<uint32_t*>(&q);
    const uint32_t both = static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(&off)) * 0x10001u;
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const uint32_t m = (on >> (2 * e) & 1u) * 0xffffu | (on >> (2 * e + 1) & 1u) * 0xffff0000u;
      w[e] = (w[e] & m) | (both & ~m);
    }
  }
}

__device__ __forceinline__ const uint32_t* mask_of(const ProcessLogits& a, int64_t r) {
  if (!a.allowed) return nullptr;
  const int64_t m = a.allowed_rows ? a.allowed_rows[r] : r;
  return m >= 0 && m < a.M ? a.allowed + m * ((a.V + 31) / 32) : nullptr;
}

// Row r's history in the token buffer: prompt [p0, p1), outputs [p1, p2).
struct Span {
  int64_t p0, p1, p2;
};

__device__ __forceinline__ Span span_of(const ProcessLogits& a, int64_t r) {
  Span s{0, 0, 0};
  if (a.tokens) {
    s.p0 = min(max(a.spans[3 * r], int64_t{0}), a.n_tokens);
    s.p1 = min(max(a.spans[3 * r + 1], s.p0), a.n_tokens);
    s.p2 = min(max(a.spans[3 * r + 2], s.p1), a.n_tokens);
  }
  return s;
}

// each(id) for tokens[from, to) by a CTA of kCount threads, 16 bytes per load.
template <int kCount, class F>
__device__ __forceinline__ void each_token(const int32_t* tokens, int64_t from, int64_t to, F&& each) {
  const int64_t q0 = min(from + to_boundary(tokens + from), to), q1 = q0 + (to - q0) / 4 * 4;
  if (from + threadIdx.x < q0) each(tokens[from + threadIdx.x]);
  if (q1 + threadIdx.x < to) each(tokens[q1 + threadIdx.x]);
  const int4* const v4 = reinterpret_cast<const int4*>(tokens + q0);
  const int64_t packs = (q1 - q0) / 4;
#pragma unroll 2
  for (int64_t i = threadIdx.x; i < packs; i += kCount) {
    const int4 v = v4[i];
    each(v.x);
    each(v.y);
    each(v.z);
    each(v.w);
  }
}

// Grid (chunks of kUnroll * kCopyThreads packs, rows).
template <typename T>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(ProcessLogits a) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr int VEC = kVec<T>;
  constexpr uint32_t kAll = (1u << VEC) - 1u;
  const T off = from_f32<T>(-INFINITY);
  for (int64_t r = blockIdx.y; r < a.R; r += gridDim.y) {
    const uint32_t* const mask = mask_of(a, r);
    const T* const src = static_cast<const T*>(a.logits) + r * a.ld;
    T* const dst = static_cast<T*>(a.out) + r * a.out_ld;
    const bool in_place = src == dst;
    if (in_place && !mask) continue;
    auto allowed = [&](int c) { return !mask || (mask[c >> 5] >> (c & 31) & 1u); };
    if (!same_offset16(src, static_cast<const T*>(dst))) {
      constexpr int kChunk = kUnroll * kCopyThreads * VEC;
      const int64_t end = min(static_cast<int64_t>(blockIdx.x + 1) * kChunk, static_cast<int64_t>(a.V));
#pragma unroll 4
      for (int64_t c = static_cast<int64_t>(blockIdx.x) * kChunk + threadIdx.x; c < end; c += kCopyThreads)
        dst[c] = allowed(static_cast<int>(c)) ? src[c] : off;
      continue;
    }
    const int head = min(to_boundary(src), a.V), packs = (a.V - head) / VEC;
    const int tail = head + packs * VEC;
    if (blockIdx.x == 0) {   // what lies before the first and after the last pack
      const int i = threadIdx.x < head ? threadIdx.x : tail + static_cast<int>(threadIdx.x) - head;
      if (i < a.V && static_cast<int>(threadIdx.x) < 2 * VEC) dst[i] = allowed(i) ? src[i] : off;
    }
    const Pack<T, VEC>* const from = reinterpret_cast<const Pack<T, VEC>*>(src + head);
    Pack<T, VEC>* const to = reinterpret_cast<Pack<T, VEC>*>(dst + head);
    const int k0 = blockIdx.x * (kUnroll * kCopyThreads) + threadIdx.x;
    Pack<T, VEC> q[kUnroll];
    uint32_t on[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = k0 + u * kCopyThreads;
      on[u] = kAll;
      if (k >= packs) continue;
      if (mask) on[u] = mask_bits(mask, head + k * VEC, VEC, a.V) & kAll;
      if (on[u] && !(in_place && on[u] == kAll)) q[u] = load_once(from + k);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = k0 + u * kCopyThreads;
      if (k >= packs || (in_place && on[u] == kAll)) continue;
      if (mask) keep_allowed<T, VEC>(q[u], on[u], off);
      to[k] = q[u];
    }
  }
}

// Shared memory: bitmap [range / 32], rank of each word's first bit [range / 32],
// then per id of the window: column, 2 * outputs + met, and with biases 1 + the
// last entry's index.  Grid (column ranges, rows).  With after_copy the kernel
// follows copy_kernel, whose CTAs let it start once they know that what came
// before is complete; only the last step waits for the copy itself.
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    rewrite_kernel(ProcessLogits a, int range, int after_copy) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint32_t bitmap[];
  __shared__ int red[kWarps];
  if (!after_copy) pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* const rank = bitmap + range / 32;
  uint32_t* const column = rank + range / 32;
  uint32_t* const count = column + kWindow;
  uint32_t* const slot = count + kWindow;
  const int c0 = range * static_cast<int>(blockIdx.x), n = min(range, a.V - c0);
  const int map_words = (n + 31) / 32;
  for (int64_t r = blockIdx.y; r < a.R; r += gridDim.y) {
    const auto [p0, p1, p2] = span_of(a, r);
    int64_t b0 = 0, biases = 0;
    if (a.bias_offsets) {
      b0 = min(max(a.bias_offsets[r], int64_t{0}), a.n_bias);
      biases = min(max(a.bias_offsets[r + 1], b0), a.n_bias) - b0;
    }
    if (p2 == p0 && biases == 0) continue;
    const int32_t* const bias_ids = a.bias_ids + b0;
    // column of an id in this range; an id of another range, or none, gives >= n
    auto at = [&](int id) { return static_cast<uint32_t>(id) - static_cast<uint32_t>(c0); };

    // the distinct ids
    __syncthreads();   // the previous row's readers are done
    for (int i = threadIdx.x; i < (map_words + 3) / 4; i += kThreads)
      reinterpret_cast<uint4*>(bitmap)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    auto mark = [&](int id) {
      const uint32_t e = at(id);
      if (e < static_cast<uint32_t>(n)) atomicOr(&bitmap[e >> 5], 1u << (e & 31));
    };
    if (p2 > p0) each_token<kThreads>(a.tokens, p0, p2, mark);
    for (int64_t j = threadIdx.x; j < biases; j += kThreads) mark(bias_ids[j]);
    __syncthreads();
    // ranks: each thread sums a run of words, the runs are scanned once
    const int run = (map_words + kThreads - 1) / kThreads, w0 = threadIdx.x * run;
    int ones = 0;
    for (int i = w0; i < min(w0 + run, map_words); ++i) ones += __popc(bitmap[i]);
    int upto = ones;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) red[warp] = upto;
    __syncthreads();
    const int mine = lane < kWarps ? red[lane] : 0;
    const int distinct = __reduce_add_sync(0xffffffffu, mine);
    int before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0) + upto - ones;
    for (int i = w0; i < min(w0 + run, map_words); ++i) {
      rank[i] = before;
      before += __popc(bitmap[i]);
    }
    auto rank_of = [&](uint32_t e) {
      return rank[e >> 5] + __popc(bitmap[e >> 5] & ((1u << (e & 31)) - 1u));
    };

    const uint32_t* const mask = mask_of(a, r);
    const float rho = a.repetition ? a.repetition[r] : 1.f;
    const float fr = a.frequency ? a.frequency[r] : 0.f;
    const float pr = a.presence ? a.presence[r] : 0.f;
    T* const dst = static_cast<T*>(a.out) + r * a.out_ld;
    for (int first = 0; first < distinct; first += kWindow) {
      const uint32_t here = min(kWindow, distinct - first);
      if (first) __syncthreads();
      for (uint32_t i = threadIdx.x; i < here; i += kThreads) {
        count[i] = 0;
        if (biases) slot[i] = 0;
      }
      __syncthreads();   // also: the ranks are there
      // index of an id in the window; every occurrence notes the column
      auto place = [&](int id) -> uint32_t {
        const uint32_t e = at(id);
        if (e >= static_cast<uint32_t>(n)) return ~0u;
        const uint32_t k = rank_of(e) - first;
        if (k >= here) return ~0u;
        column[k] = e;
        return k;
      };
      if (p1 > p0)
        each_token<kThreads>(a.tokens, p0, p1, [&](int id) {
          const uint32_t k = place(id);
          if (k != ~0u) atomicOr(&count[k], 1u);
        });
      if (p2 > p1)
        each_token<kThreads>(a.tokens, p1, p2, [&](int id) {
          const uint32_t k = place(id);
          if (k != ~0u) atomicAdd(&count[k], 2u);
        });
      for (int64_t j = threadIdx.x; j < biases; j += kThreads) {   // the last entry counts
        const uint32_t k = place(bias_ids[j]);
        if (k != ~0u) atomicMax(&slot[k], static_cast<uint32_t>(j) + 1u);
      }
      __syncthreads();
      if (after_copy) pdl_wait_prerequisites();
      for (uint32_t k0 = threadIdx.x; k0 < here; k0 += kBatch * kThreads) {
        T v[kBatch];
        int c[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const uint32_t k = k0 + u * kThreads;
          c[u] = k < here ? static_cast<int>(column[k]) : -1;
          if (c[u] < 0) continue;
          v[u] = dst[c0 + c[u]];
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (c[u] < 0) continue;
          const uint32_t k = k0 + u * kThreads;
          const int at = c0 + c[u];
          if (mask && !(mask[at >> 5] >> (at & 31) & 1u)) continue;
          const uint32_t met = count[k];
          float y = to_f32(v[u]);
          if (met) {
            y = y > 0.f ? y / rho : y * rho;
            if (met > 1u) y -= fmaf(fr, static_cast<float>(met >> 1), pr);
          }
          if (biases && slot[k]) y += a.bias_values[b0 + slot[k] - 1];
          dst[at] = from_f32<T>(y);
        }
      }
    }
  }
  if (after_copy) pdl_wait_prerequisites();   // rows without history: still after the copy
}

// The gradient in one pass.  A bitmap of the CTA's columns says which were met; a pack
// with such a column loads its logits beside its gradients.  Every column range of a row
// scans the row's whole history (from L2 but for the first), which costs less than a
// second visit of scattered elements: copying first and rewriting the met ones then, as
// the forward does, took 59 us where this takes 51 (512 rows of 50,257 fp32, 2,300 tokens
// each), and 83 against 50 with 2,048 rows of 18,992 fp16.  Bound by instructions and the
// latency of bitmap, mask and gradient one after another, so by threads: eight CTAs per
// SM; two packs per thread do not gain.  1 / rho is rounded once and the product once.
template <typename T>
__global__ void __launch_bounds__(kGradThreads, 8) grad_kernel(ProcessLogits a, int range) {
  extern __shared__ uint32_t met[];   // bits of the range's columns, one word of zeros after them
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr int VEC = kVec<T>;
  constexpr uint32_t kAll = (1u << VEC) - 1u;
  const T zero = from_f32<T>(0.f);
  const int c0 = blockIdx.x * range, n = min(range, a.V - c0), words = (n + 31) / 32 + 1;
  for (int64_t r = blockIdx.y; r < a.R; r += gridDim.y) {
    const Span at = span_of(a, r);
    const bool touched = at.p2 > at.p0;
    const uint32_t* const mask = mask_of(a, r);
    const T* const src = static_cast<const T*>(a.grad) + r * a.grad_ld + c0;
    const T* const x = static_cast<const T*>(a.logits) + r * a.ld + c0;
    T* const dst = static_cast<T*>(a.out) + r * a.out_ld + c0;
    const bool in_place = src == dst;
    if (in_place && !mask && !touched) continue;
    __syncthreads();   // the previous row's readers are done
    for (int i = threadIdx.x; i < words; i += kGradThreads) met[i] = 0;
    __syncthreads();
    if (touched) {
      each_token<kGradThreads>(a.tokens, at.p0, at.p2, [&](int id) {
        const uint32_t e = static_cast<uint32_t>(id) - static_cast<uint32_t>(c0);
        if (e < static_cast<uint32_t>(n)) atomicOr(&met[e >> 5], 1u << (e & 31));
      });
      __syncthreads();
    }
    const float rho = a.repetition ? a.repetition[r] : 1.f, inv = 1.f / rho;
    auto one = [&](int c) {   // column c of the range
      const bool keep = !mask || (mask[(c0 + c) >> 5] >> ((c0 + c) & 31) & 1u);
      const bool was = met[c >> 5] >> (c & 31) & 1u;
      if (!keep)
        dst[c] = zero;
      else if (was)
        dst[c] = from_f32<T>(to_f32(src[c]) * (to_f32(x[c]) > 0.f ? inv : rho));
      else if (!in_place)
        dst[c] = src[c];
    };
    if (!same_offset16(src, static_cast<const T*>(dst))) {
      for (int c = threadIdx.x; c < n; c += kGradThreads) one(c);
      continue;
    }
    const int head = min(to_boundary(src), n), packs = (n - head) / VEC, tail = head + packs * VEC;
    const bool x_packs = same_offset16(src, x);
    if (threadIdx.x < 2 * VEC) {   // what lies before the first and after the last pack
      const int c = threadIdx.x < head ? threadIdx.x : tail + static_cast<int>(threadIdx.x) - head;
      if (c < n) one(c);
    }
    for (int k = threadIdx.x; k < packs; k += kGradThreads) {
      const int c = head + k * VEC;
      const uint32_t on = mask ? mask_bits(mask, c0 + c, VEC, a.V) & kAll : kAll;
      const uint32_t was = __funnelshift_r(met[c >> 5], met[(c >> 5) + 1], c & 31) & on;
      if (in_place && on == kAll && !was) continue;
      Pack<T, VEC> q, xq;
      if (on) q = *reinterpret_cast<const Pack<T, VEC>*>(src + c);
      if (was) {
        if (x_packs) xq = *reinterpret_cast<const Pack<T, VEC>*>(x + c);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (was >> e & 1u)
            q.v[e] = from_f32<T>(to_f32(q.v[e]) * (to_f32(x_packs ? xq.v[e] : x[c + e]) > 0.f ? inv : rho));
      }
      if (mask) keep_allowed<T, VEC>(q, on, zero);
      *reinterpret_cast<Pack<T, VEC>*>(dst + c) = q;
    }
  }
}

template <typename T, int kThreads>
cudaError_t rewrite(const ProcessLogits& a, unsigned rows, bool after_copy, cudaStream_t s) {
  static std::atomic<int> ready[64];
  auto* kern = rewrite_kernel<T, kThreads>;
  const cudaError_t e = allow_shared(ready, reinterpret_cast<const void*>(kern),
                                     2 * kMostColumns / 8 + 3 * 4 * kWindow);
  if (e != cudaSuccess) return e;
  const int64_t padded = (static_cast<int64_t>(a.V) + 127) / 128 * 128;   // whole 16-byte words of bitmap
  const int range = static_cast<int>(padded < kMostColumns ? padded : kMostColumns);
  const unsigned ranges = static_cast<unsigned>((padded + range - 1) / range);
  const size_t smem = 2 * static_cast<size_t>(range) / 8 + (a.bias_offsets ? 3 : 2) * 4 * kWindow;
  return launch_dependent(kern, dim3(ranges, rows), kThreads, smem, 1, s, a, range, after_copy ? 1 : 0);
}

template <typename T>
cudaError_t forward(const ProcessLogits& a, cudaStream_t s) {
  const unsigned rows = static_cast<unsigned>(a.R < 32768 ? a.R : 32768);
  const bool copy = a.logits != a.out || a.ld != a.out_ld || a.allowed;
  if (copy) {
    constexpr int kChunk = kUnroll * kCopyThreads * kVec<T>;
    const unsigned chunks = static_cast<unsigned>((static_cast<int64_t>(a.V) + kChunk - 1) / kChunk);
    const cudaError_t e = launch_dependent(copy_kernel<T>, dim3(chunks, rows),
                                           kCopyThreads, 0, 1, s, a);
    if (e != cudaSuccess) return e;
  }
  if (!a.tokens && !a.bias_offsets) return cudaSuccess;
  // More than two rounds of CTAs: four smaller ones per SM, whose barriers and latencies
  // overlap (2,048 rows of 18,992 fp16: 71 us against 83, 2,000 of 1,003 bf16: 30 against
  // 44); fewer rows keep large ones (256 rows of 151,936 bf16: 50 against 58, 512 of 50,257
  // fp32: 53 against 56).
  if (a.R > 4ll * sm_count()) return rewrite<T, 256>(a, rows, copy, s);
  return rewrite<T, 512>(a, rows, copy, s);
}

template <typename T>
cudaError_t backward(const ProcessLogits& a, cudaStream_t s) {
  // Ranges of about 64 KB, shorter while there are fewer than about four rounds of CTAs.
  const int64_t bytes = static_cast<int64_t>(a.V) * static_cast<int64_t>(sizeof(T));
  const int64_t least = (bytes + kGradMost - 1) / kGradMost, most = (bytes + kGradLeast - 1) / kGradLeast;
  int64_t ranges = (20ll * sm_count() + a.R - 1) / a.R;
  ranges = ranges < least ? least : ranges > most ? most : ranges;
  const int range = static_cast<int>(((a.V + ranges - 1) / ranges + 63) / 64 * 64);
  const unsigned rows = static_cast<unsigned>(a.R < 32768 ? a.R : 32768);
  return launch_dependent(grad_kernel<T>,
                          dim3(static_cast<unsigned>((static_cast<int64_t>(a.V) + range - 1) / range), rows),
                          kGradThreads, 4 * static_cast<size_t>(range / 32 + 1), 1, s, a, range);
}

template <typename T>
cudaError_t either(const ProcessLogits& a, cudaStream_t s) {
  return a.grad ? backward<T>(a, s) : forward<T>(a, s);
}

}  // namespace

cudaError_t launch_process_logits(const ProcessLogits& a, cudaStream_t s) {
  if (a.type == kF32) return either<float>(a, s);
  if (a.type == kBF16) return either<__nv_bfloat16>(a, s);
  return either<__half>(a, s);
}

}  // namespace lmh
