// activation.cuh -- the activations of dg_activation and their derivatives in
// FP32, and division by a given scale: what the product's epilogue and the
// kernels on rows share.
//
// SiLU and the tanh form of GELU are x times a logistic function:
//   x / (1 + exp(-u)),  u = x  or  u = 2 sqrt(2 / pi) (x + 0.044715 x^3)
// ((1 + tanh(u / 2)) / 2 = 1 / (1 + exp(-u))), and GELU is x erfc(-x / sqrt 2) / 2.
// In these forms nothing cancels for negative x: the result keeps FP32's
// relative precision (the exponential's is 2^-22 times its argument's size).
#pragma once

#include <cstdint>

#include "dg.h"

namespace dg {

constexpr float kGeluSlope = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// 1 / (1 + exp(-u)); 0 where the exponential overflows.
__device__ __forceinline__ float logistic(float u) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-u)));
    return r;
}

// x^2 as the tanh form uses it: past 1000 the function has long been x or 0,
// and the bound keeps infinity times zero out.
__device__ __forceinline__ float gelu_square(float x) { return fminf(x * x, 1e6f); }

// The value.  `act` is the same for every thread of a launch.
__device__ __forceinline__ float activation(int act, float x) {
    switch (act) {
        case DG_ACT_RELU: return x < 0.0f ? 0.0f : x;   // NaN stays
        case DG_ACT_GELU: return 0.5f * x * erfcf(x * -0.70710678118654752f);
        case DG_ACT_GELU_TANH: return x * logistic(kGeluSlope * x * fmaf(kGeluCubic, gelu_square(x), 1.0f));
        case DG_ACT_SILU: return x * logistic(x);
        default: return x;
    }
}

struct ValueSlope {
    float value, slope;
};

// The value and the derivative.
__device__ __forceinline__ ValueSlope activation_slope(int act, float x) {
    switch (act) {
        case DG_ACT_RELU: return {x < 0.0f ? 0.0f : x, x > 0.0f ? 1.0f : x == x ? 0.0f : x};
        case DG_ACT_GELU: {
            const float phi = 0.5f * erfcf(x * -0.70710678118654752f);
            return {x * phi, fmaf(x * 0.3989422804014327f, __expf(-0.5f * x * x), phi)};
        }
        case DG_ACT_GELU_TANH: {
            const float x2 = gelu_square(x);
            const float g = logistic(kGeluSlope * x * fmaf(kGeluCubic, x2, 1.0f));
            const float du = kGeluSlope * fmaf(3.0f * kGeluCubic, x2, 1.0f);
            const float v = x * g;   // first: large -x times 0 is 0
            return {v, fmaf(v * (1.0f - g), du, g)};
        }
        case DG_ACT_SILU: {
            const float g = logistic(x);
            const float v = x * g;
            return {v, fmaf(v, 1.0f - g, g)};
        }
        default: return {x, 1.0f};
    }
}

// Division by a given scale as two multiplications: x / s = (x pre) inv.  pre
// is 1 but for scales whose reciprocal FP32 does not hold; with it the
// product overflows or vanishes only where the code saturates or is 0 anyway.
struct ByScale {
    float pre, inv;
};
__device__ __forceinline__ ByScale by_scale(float s) {
    const float m = fabsf(s);
    const float pre = m < 0x1p-120f ? 0x1p64f : m > 0x1p120f ? 0x1p-64f : 1.0f;
    return {pre, __frcp_rn(s * pre)};
}

}  // namespace dg
