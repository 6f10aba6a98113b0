// Instantiation of the tcgen05 GEMM for the distillation forward: the logits'
// online maximum and exponential sum, and the logits at each token's list of
// teacher ids (A = hidden rows, B = vocabulary rows, both K-major).
#include "tc_gemm.cuh"

namespace lmh {

cudaError_t launch_gemm_fwd_pick(const LaunchArgs& a, int grid, bool pair, cudaStream_t s) {
  return pair ? launch_tc_gemm<EPI_FWD_PICK, false, true>(a, grid, s)
              : launch_tc_gemm<EPI_FWD_PICK, false, false>(a, grid, s);
}

}  // namespace lmh
