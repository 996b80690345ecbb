// k_gemm_tc_fused.cu -- the single-CTA tensor-core GEMM with bias, activation
// and residual in its epilogue (gemm_tc_kernel.cuh, kFused).
#include "gemm_tc_kernel.cuh"

namespace dg {

cudaError_t launch_gemm_tc_fused(const TcLaunch& L, const Params& prm, cudaStream_t s) {
    return L.fp16_in ? launch_in<true, true>(L, prm, s) : launch_in<false, true>(L, prm, s);
}

}  // namespace dg
