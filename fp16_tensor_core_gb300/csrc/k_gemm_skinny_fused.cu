// k_gemm_skinny_fused.cu -- the split-K tensor-core GEMM with bias, activation
// and residual in its epilogue (gemm_skinny_kernel.cuh, kFused).
#include "gemm_skinny_kernel.cuh"

namespace dg {

cudaError_t launch_gemm_skinny_fused(const TcLaunch& L, float* partials, uint32_t* counts, cudaStream_t s) {
    return L.fp16_in ? launch_in<true, true>(L, partials, counts, s) : launch_in<false, true>(L, partials, counts, s);
}

}  // namespace dg
