// k_epilogue.cu -- the fused product's epilogue alone: K = 0, an empty sum.
//   D[m, n] = out(act(bias[n]) + residual[m, n])
// One element a thread and step; no product of a model comes here.
#include <cuda_runtime.h>

#include <algorithm>

#include "activation.cuh"
#include "dg_internal.h"
#include "dg_ptx.cuh"

namespace dg {
namespace {

struct EmptySum {
    void* D;
    int64_t elements;
    int N, out_kind;
    const float* sd;
    uint32_t* amax_out;
    Epilogue epi;
};

__global__ void __launch_bounds__(256) epilogue_only_kernel(const EmptySum a) {
    pdl_wait();
    const ByScale by = a.out_kind == kOutE4M3 ? by_scale(*a.sd) : ByScale{1.0f, 1.0f};
    uint32_t top = 0u;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.elements;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        float y = activation(a.epi.act, a.epi.bias != nullptr ? a.epi.bias[i % a.N] : 0.0f);
        if (a.epi.residual != nullptr) {
            const uint32_t e = a.epi.residual[i];
            y += a.epi.residual_fp16 != 0 ? f16x2_to_f32x2(e).x : __uint_as_float(e << 16);
        }
        top = max(top, __float_as_uint(y) & 0x7FFFFFFFu);
        if (a.out_kind == kOutE4M3)
            static_cast<uint8_t*>(a.D)[i] = static_cast<uint8_t>(f32x2_to_e4m3x2(y * by.pre * by.inv, 0.0f) & 0xFFu);
        else if (a.out_kind == kOutFP16)
            static_cast<uint16_t*>(a.D)[i] = static_cast<uint16_t>(f32x2_to_f16x2(y, 0.0f) & 0xFFFFu);
        else
            static_cast<uint16_t*>(a.D)[i] = static_cast<uint16_t>(f32x2_to_bf16x2(y, 0.0f) & 0xFFFFu);
    }
    if (a.amax_out != nullptr) {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if ((threadIdx.x & 31) == 0 && top != 0u) atomicMax(a.amax_out, top);
    }
}

}  // namespace

cudaError_t launch_epilogue_only(const TcLaunch& L, cudaStream_t s) {
    EmptySum a{};
    a.D = L.D;
    a.elements = static_cast<int64_t>(L.M) * L.N;
    a.N = L.N;
    a.out_kind = L.out_kind;
    a.sd = L.sd;
    a.amax_out = L.amax_out;
    a.epi = *L.epi;
    const int64_t blocks = std::min<int64_t>((a.elements + 255) / 256, 4096);
    return launch_kernel(epilogue_only_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a);
}

}  // namespace dg
