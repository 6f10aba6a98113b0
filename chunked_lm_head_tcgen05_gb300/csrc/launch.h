// Host-side pieces shared by the translation units that implement the C ABI:
// the launch counter / profile records, device facts, and a launcher with
// programmatic dependent launch and an optional cluster.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <utility>

namespace lmh {

// Event pair around one launch while profiling is on (both NULL otherwise).
struct LaunchTrace {
  cudaEvent_t start, stop;
};
LaunchTrace trace_start(cudaStream_t s);
void trace_stop(const char* name, cudaStream_t s, const LaunchTrace& t, bool launched) noexcept;

template <class F>
cudaError_t traced_launch(const char* name, cudaStream_t s, F&& f) {
  const LaunchTrace t = trace_start(s);
  const cudaError_t e = f();
  trace_stop(name, s, t, e == cudaSuccess);
  return e;
}

// SMs of the current device (0 if it cannot be read).
int sm_count();

// Allow `kern` that much dynamic shared memory, once per device: `ready` is the
// kernel's own (zeroed) table, so later launches make no configuration call.
inline cudaError_t allow_shared(std::atomic<int> (&ready)[64], const void* kern, size_t bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (ready[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess) ready[dev].store(1, std::memory_order_relaxed);
  return e;
}

// Launch that may start while its predecessor in the stream finishes; the
// kernel waits for the predecessor (griddepcontrol.wait) before it touches
// memory.  cluster > 1 groups that many consecutive CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), dim3 grid, int block, size_t smem,
                             int cluster, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  int n = 1;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

}  // namespace lmh
