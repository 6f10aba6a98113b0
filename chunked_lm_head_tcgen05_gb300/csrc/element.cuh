// Element types of the operators on caller-held tensors (fp32, bf16, fp16):
// conversion to and from the fp32 they are computed in, and 16-byte packs.
#pragma once

#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

namespace lmh {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
  return __float2half_rn(x);
}

// VEC elements moved by one 16-byte access or less (two for 8 fp32), aligned to it.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC > 16 ? 16 : sizeof(T) * VEC) Pack {
  T v[VEC];
};

// Elements of a 16-byte access.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

// Elements before the first 16-byte boundary at or after p (p is aligned to
// its element).
template <typename T>
__device__ __forceinline__ int to_boundary(const T* p) {
  return static_cast<int>(((16u - (static_cast<unsigned>(reinterpret_cast<uintptr_t>(p)) & 15u)) & 15u) /
                          sizeof(T));
}

template <typename T>
__device__ __forceinline__ bool same_offset16(const T* a, const T* b) {
  return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15u) == 0;
}

// Elements 2 i and 2 i + 1 of a pack.
template <int VEC>
__device__ __forceinline__ float2 pair_of(const Pack<float, VEC>& q, int i) {
  return make_float2(q.v[2 * i], q.v[2 * i + 1]);
}
template <int VEC>
__device__ __forceinline__ float2 pair_of(const Pack<__nv_bfloat16, VEC>& q, int i) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(&q)[i];   // bf16 is the upper half of fp32
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <int VEC>
__device__ __forceinline__ float2 pair_of(const Pack<__half, VEC>& q, int i) {
  return __half22float2(reinterpret_cast<const __half2*>(&q)[i]);
}

template <int VEC>
__device__ __forceinline__ void set_pair(Pack<float, VEC>& q, int i, float2 x) {
  q.v[2 * i] = x.x;
  q.v[2 * i + 1] = x.y;
}
template <int VEC>
__device__ __forceinline__ void set_pair(Pack<__nv_bfloat16, VEC>& q, int i, float2 x) {
  reinterpret_cast<__nv_bfloat162*>(&q)[i] = __floats2bfloat162_rn(x.x, x.y);
}
template <int VEC>
__device__ __forceinline__ void set_pair(Pack<__half, VEC>& q, int i, float2 x) {
  reinterpret_cast<__half2*>(&q)[i] = __floats2half2_rn(x.x, x.y);
}

// Asynchronous copy of 4, 8 or 16 bytes into shared memory; a thread that reads
// back only what it copied itself needs no barrier.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes)
                 : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Packs of VEC elements in flight, one column of slots per thread: slot s of
// thread i lies at unit (s kParts + part) threads + i, so that a warp's accesses
// are contiguous.
template <typename T, int VEC>
struct PackRing {
  static constexpr int kBytes = static_cast<int>(sizeof(T)) * VEC;
  static constexpr int kUnit = kBytes > 16 ? 16 : kBytes;
  static constexpr int kParts = kBytes / kUnit;
  static constexpr bool kAsync = kUnit >= 4;   // smaller units cannot be copied asynchronously
  char* mine;
  int stride;
  __device__ __forceinline__ PackRing(void* base, int threads, int thread)
      : mine(static_cast<char*>(base) + thread * kUnit), stride(threads * kUnit) {}
  __device__ __forceinline__ void fetch(int slot, const T* src) const {
#pragma unroll
    for (int q = 0; q < kParts; ++q)
      copy_async<kUnit>(static_cast<uint32_t>(__cvta_generic_to_shared(mine + (slot * kParts + q) * stride)),
                        reinterpret_cast<const char*>(src) + q * kUnit);
  }
  __device__ __forceinline__ void clear(int slot) const {
#pragma unroll
    for (int q = 0; q < kParts; ++q)
#pragma unroll
      for (int b = 0; b < kUnit; b += 4)
        *reinterpret_cast<uint32_t*>(mine + (slot * kParts + q) * stride + b) = 0;
  }
  __device__ __forceinline__ Pack<T, VEC> read(int slot) const {
    constexpr int N = VEC / kParts;
    Pack<T, VEC> out;
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
      const Pack<T, N> x = *reinterpret_cast<const Pack<T, N>*>(mine + (slot * kParts + q) * stride);
#pragma unroll
      for (int e = 0; e < N; ++e) out.v[q * N + e] = x.v[e];
    }
    return out;
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

}  // namespace lmh
