// k_gemm_tc2_fused.cu -- the CTA-pair tensor-core GEMM with bias, activation
// and residual in its epilogue (gemm_pair_kernel.cuh, kFused).
#include "gemm_pair_kernel.cuh"

namespace dg {

cudaError_t launch_gemm_tc_pair_fused(const TcLaunch& L, const Params& prm, cudaStream_t s) {
    return L.fp16_in ? launch_pair_in<true, true>(L, prm, s) : launch_pair_in<false, true>(L, prm, s);
}

}  // namespace dg
