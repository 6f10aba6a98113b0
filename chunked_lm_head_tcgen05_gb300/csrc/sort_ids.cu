// Positions of a list of ids in ascending order of the ids, equal ids in the
// order of their positions: what the embedding's gradient sums by, and what
// groups rows by their adapter.  A stable radix sort in one launch of one
// cluster: the pairs (id, position) stay in the cluster's shared memory, a pass
// ranks them by one digit and writes each to its new place, in whichever CTA
// that is.  Up to 131,072 ids (8 CTAs x 16,384 pairs); digits of up to 9 bits, so
// a 151,936-id vocabulary takes two passes.
// Rank of a pair among those with its digit: pairs before it in its warp (votes
// over the warp's lanes, and the warp's own counts from earlier rounds), in
// earlier warps and in earlier CTAs; counts are sums of integers, so the order is
// the same in every run.
// Bound by latency and by the stores into other CTAs: two passes take 26 us for 60,000
// ids and 12 for 4,096 that come from HBM, one pass over 2,048 ids 6.
#include "operators.h"
#include "ptx.cuh"

namespace lmh {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDigits = 512;
constexpr int kCluster = 8;

struct SortArgs {
  const int32_t* ids;   // NULL: all 0
  int n;
  int bound;       // ids outside [0, bound) sort last, as `bound`
  int wrap;        // ids in [-bound, 0) mean id + bound
  int skip;        // an id (after wrapping) that counts as outside; -1: none
  int bits;        // of a digit
  int passes;
  int ctas;        // of the cluster
  int32_t* keys;   // [n] ascending
  int32_t* pos;    // [n]
  int* live;       // ids inside
  uint4* zeros;    // cleared by the clusters behind the first
  size_t n_zeros;  // 16-byte units
};

__device__ __forceinline__ uint64_t pair_of_key(uint32_t key, uint32_t pos) {
  return static_cast<uint64_t>(key) << 32 | pos;
}

template <int ITEMS>
__global__ void __launch_bounds__(kThreads) sort_kernel(SortArgs a) {
  extern __shared__ __align__(16) char smem[];
  uint64_t* const buf = reinterpret_cast<uint64_t*>(smem);                     // [kThreads * ITEMS]
  uint16_t* const cnt = reinterpret_cast<uint16_t*>(buf + kThreads * ITEMS);   // [kWarps][digits]
  int* const tot = reinterpret_cast<int*>(cnt + kWarps * kMaxDigits);          // [kCluster][digits]
  int* const base = tot + kCluster * kMaxDigits;                               // [digits]
  int* const part = base + kMaxDigits;                                         // [kWarps]
  int* const mine = part + kWarps;                                             // ids inside, this CTA
  constexpr int P = kThreads * ITEMS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x), ctas = a.ctas;   // the first cluster sorts
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= ctas) {
    const size_t stride = static_cast<size_t>(gridDim.x - ctas) * kThreads;
    for (size_t i = static_cast<size_t>(blockIdx.x - ctas) * kThreads + tid; i < a.n_zeros; i += stride)
      a.zeros[i] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int first = warp * 32 * ITEMS + lane;
  const int digits = 1 << a.bits;
  const uint32_t last = a.passes * a.bits >= 32 ? 0xffffffffu : (1u << (a.passes * a.bits)) - 1u;
  uint64_t pr[ITEMS];
  int inside = 0;
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int g = rank * P + first + j * 32;
    uint32_t key = last;               // places past the end sort behind everything
    if (g < a.n) {
      int id = a.ids ? a.ids[g] : 0;
      if (a.wrap && id < 0) id += a.bound;
      const bool in = id >= 0 && id < a.bound && id != a.skip;
      key = static_cast<uint32_t>(in ? id : a.bound);
      inside += in;
    }
    pr[j] = pair_of_key(key, static_cast<uint32_t>(g));
  }
  if (tid == 0) *mine = 0;
  cluster_sync();   // every CTA runs before one writes to its memory
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) inside += __shfl_xor_sync(0xffffffffu, inside, o);
  if (lane == 0 && inside) atomicAdd(mine, inside);

  uint16_t rnk[ITEMS];
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = 32 + pass * a.bits;
    const uint32_t mask = static_cast<uint32_t>(digits) - 1u;
    uint16_t* const own = cnt + warp * digits;
    for (int d = lane; d < digits; d += 32) own[d] = 0;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const uint32_t d = static_cast<uint32_t>(pr[j] >> shift) & mask;
      // lanes with the same digit, bit by bit: a match instruction over 32 different values
      // takes longer than nine votes
      uint32_t peers = 0xffffffffu;
      for (int b = 0; b < a.bits; ++b) {
        const bool on = d >> b & 1u;
        const uint32_t votes = __ballot_sync(0xffffffffu, on);
        peers &= on ? votes : ~votes;
      }
      const int before = own[d];
      rnk[j] = static_cast<uint16_t>(before + __popc(peers & ((1u << lane) - 1u)));
      __syncwarp();
      if (lane == __ffs(static_cast<int>(peers)) - 1)
        own[d] = static_cast<uint16_t>(before + __popc(peers));
      __syncwarp();
    }
    __syncthreads();
    if (tid < digits) {
      int c[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) c[w] = cnt[w * digits + tid];
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        cnt[w * digits + tid] = static_cast<uint16_t>(sum);
        sum += c[w];
      }
      // to every CTA: a store does not wait, a load from each of eight CTAs would
      const uint32_t at = smem_addr(tot + rank * kMaxDigits + tid);
      for (int c = 0; c < ctas; ++c)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_cta(at, c)), "r"(sum) : "memory");
    }
    cluster_sync();   // every CTA's totals, and every pair is in its thread's registers
    int before = 0, all = 0;
    if (tid < digits) {
#pragma unroll
      for (int c = 0; c < kCluster; ++c) {
        const int v = c < ctas ? tot[c * kMaxDigits + tid] : 0;
        before += c < rank ? v : 0;
        all += v;
      }
    }
    // exclusive sum over the digits
    int scan = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) part[warp] = scan;
    __syncthreads();
    int ahead = 0;
    for (int w = 0; w < warp && w * 32 < digits; ++w) ahead += part[w];
    if (tid < digits) base[tid] = ahead + scan - all + before;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const uint32_t d = static_cast<uint32_t>(pr[j] >> shift) & mask;
      const int to = base[d] + own[d] + rnk[j];
      const uint32_t at = map_to_cta(smem_addr(buf + (to & (P - 1))), static_cast<uint32_t>(to / P));
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(pr[j]) : "memory");
    }
    cluster_sync();   // every pair is in its new place, the totals are free again
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) pr[j] = buf[first + j * 32];
  }
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int g = rank * P + first + j * 32;
    if (g < a.n) {
      a.keys[g] = static_cast<int32_t>(pr[j] >> 32);
      a.pos[g] = static_cast<int32_t>(static_cast<uint32_t>(pr[j]));
    }
  }
  if (rank == 0 && tid == 0) {
    int sum = 0;
    for (int c = 0; c < ctas; ++c) {
      int v;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_cta(smem_addr(mine), c)) : "memory");
      sum += v;
    }
    *a.live = sum;
  }
  cluster_sync();   // no CTA leaves while its shared memory is read
}

template <int ITEMS>
cudaError_t launch(const SortArgs& a, int grid, cudaStream_t s) {
  static std::atomic<int> ready[64];
  constexpr size_t smem = size_t{8} * kThreads * ITEMS + 2 * kWarps * kMaxDigits + 4 * ((kCluster + 1) * kMaxDigits + kWarps + 1);
  const cudaError_t e = allow_shared(ready, reinterpret_cast<const void*>(sort_kernel<ITEMS>), smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(sort_kernel<ITEMS>, dim3(grid), kThreads, smem, a.ctas, s, a);
}

}  // namespace

cudaError_t launch_sort_ids(const int32_t* ids, int n, int bound, bool wrap, int skip, int32_t* keys,
                            int32_t* pos, int* live, cudaStream_t s, void* zeros, size_t zero_bytes) {
  if (n <= 0 || n > kSortMost) return cudaErrorInvalidValue;
  // keys run from 0 to `bound`
  int width = 1;
  while (width < 31 && (bound >> width) != 0) ++width;
  const int passes = (width + 8) / 9, ctas = n <= kThreads ? 1 : kCluster;
  const SortArgs a{ids, n, bound, wrap ? 1 : 0, skip, (width + passes - 1) / passes, passes, ctas, keys, pos, live,
                   static_cast<uint4*>(zeros), zero_bytes / 16};
  // one CTA per SM; the sorting cluster's are taken
  const int sms = zero_bytes ? sm_count() : 0;
  const int grid = sms > 2 * ctas ? sms / ctas * ctas : zero_bytes ? 2 * ctas : ctas;
  const int items = ctas == 1 ? 1 : (n + kCluster * kThreads - 1) / (kCluster * kThreads);
  if (items <= 1) return launch<1>(a, grid, s);
  if (items <= 2) return launch<2>(a, grid, s);
  if (items <= 4) return launch<4>(a, grid, s);
  if (items <= 8) return launch<8>(a, grid, s);
  return launch<16>(a, grid, s);
}

}  // namespace lmh
