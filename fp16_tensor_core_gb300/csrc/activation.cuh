// activation.cuh -- the activations of dg_activation and their derivatives in
// FP32, two elements at a time, and division by a given scale: what the
// product's epilogue and the kernels on rows share.
//
// SiLU and the tanh form of GELU are x times a logistic function:
//   x / (1 + exp(-u)),  u = x  or  u = 2 sqrt(2 / pi) (x + 0.044715 x^3)
// ((1 + tanh(u / 2)) / 2 = 1 / (1 + exp(-u))).  That function is the reciprocal
// of 2^-7 (1 + exp(-u)), times 2^-7: the reciprocal gives nothing below 2^-126,
// the product is a subnormal number down to 2^-133 (u from -92), of 16 bits at
// least, and x times it a normal one.  GELU is
//   max(x, 0) - |x| h(|x|),  h(a) = erfc(a / sqrt 2) / 2 = exp(-a^2 / 2) P(1 / (1 + 0.35 a))
// with P the polynomial of degree 7 that minimises the relative error over
// 0 <= a <= 14 (a Lawson fit of exp(a^2 / 2) erfc(a / sqrt 2) / 2: below 2^-20
// in FP32 arithmetic, 6.0e-7 of it with a rounded reciprocal and 8.8e-7 with
// one off by 2^-23).  In these forms nothing cancels for negative x: the other
// two keep FP32's relative precision, and all lose only by the exponential's
// argument (2^-23 of its size, or of 7).
//
// Pairs because FP32 additions, products and fused products of two elements
// are one instruction here: GELU takes 11 issue slots an element this way.
// Through the library's erfc, with branches, the 4096 x 11008 x 4096 E4M3
// product with GELU took 363 us instead of 127.
#pragma once

#include <cstdint>

#include "dg.h"

namespace dg {

// Two FP32 elements, the first in the low word.
using pair = unsigned long long;
__device__ __forceinline__ pair pair_of(float lo, float hi) {
    pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ pair pair_of(float both) { return pair_of(both, both); }
__device__ __forceinline__ float2 floats_of(pair v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ pair pair_mul(pair a, pair b) {
    pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ pair pair_add(pair a, pair b) {
    pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ pair pair_fma(pair a, pair b, pair c) {
    pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ pair pair_neg(pair a) { return a ^ 0x8000000080000000ull; }
// max(x, 0), NaN staying; and |x|, at most 2^20 (where h has long been 0: no
// infinity times zero).
__device__ __forceinline__ pair pair_relu(pair a) {
    float2 f = floats_of(a);
    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(f.x));
    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(f.y));
    return pair_of(f.x, f.y);
}
__device__ __forceinline__ pair pair_magnitude(pair a) {
    const float2 f = floats_of(a);
    return pair_of(fminf(fabsf(f.x), 0x1p20f), fminf(fabsf(f.y), 0x1p20f));
}
__device__ __forceinline__ pair pair_ex2(pair a) {
    float2 f = floats_of(a);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f.y));
    return pair_of(f.x, f.y);
}
__device__ __forceinline__ pair pair_rcp(pair a) {
    float2 f = floats_of(a);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(f.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(f.y));
    return pair_of(f.x, f.y);
}
// The largest of |a|, |b| and a magnitude that there is; NaN above all.
__device__ __forceinline__ float pair_top(pair v, float top) {
    const float2 f = floats_of(v);
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(f.x), "f"(f.y));
    return top;
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGeluSlope = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// 1 / (1 + exp(-u)), given -u log2(e) - 7; 0 where the exponential overflows.
constexpr float kLift = 7.0f;
__device__ __forceinline__ pair logistic(pair t) {
    return pair_mul(pair_rcp(pair_add(pair_ex2(t), pair_of(0x1p-7f))), pair_of(0x1p-7f));
}
__device__ __forceinline__ pair silu_logistic(pair x) {
    return logistic(pair_fma(x, pair_of(-kLog2E), pair_of(-kLift)));
}

// x^2 as the tanh form uses it: past 1000 the function has long been x or 0,
// and the bound keeps infinity times zero out.
__device__ __forceinline__ pair gelu_square(pair x) {
    const float2 f = floats_of(pair_mul(x, x));
    return pair_of(fminf(f.x, 1e6f), fminf(f.y, 1e6f));
}
__device__ __forceinline__ pair gelu_logistic(pair x, pair square) {
    const pair t = pair_fma(pair_of(-kLog2E * kGeluSlope * kGeluCubic), square, pair_of(-kLog2E * kGeluSlope));
    return logistic(pair_fma(x, t, pair_of(-kLift)));
}

// exp(-x^2 / 2), and h(|x|).
__device__ __forceinline__ pair gelu_bell(pair x) {
    return pair_ex2(pair_mul(pair_mul(x, x), pair_of(-0.5f * kLog2E)));
}
__device__ __forceinline__ pair gelu_tail(pair magnitude, pair bell) {
    const pair t = pair_rcp(pair_fma(magnitude, pair_of(0.35f), pair_of(1.0f)));
    pair p = pair_fma(t, pair_of(0.04894209f), pair_of(-0.20211793f));
    p = pair_fma(p, t, pair_of(0.24063873f));
    p = pair_fma(p, t, pair_of(-0.017021721f));
    p = pair_fma(p, t, pair_of(0.15596068f));
    p = pair_fma(p, t, pair_of(0.1333553f));
    p = pair_fma(p, t, pair_of(0.14027031f));
    p = pair_fma(p, t, pair_of(-2.7313865e-05f));
    return pair_mul(p, bell);
}

// The value.  `act` is the same for every thread of a launch.
__device__ __forceinline__ pair activation(int act, pair x) {
    switch (act) {
        case DG_ACT_RELU: return pair_relu(x);
        case DG_ACT_GELU: {
            const pair a = pair_magnitude(x);
            return pair_fma(pair_neg(a), gelu_tail(a, gelu_bell(x)), pair_relu(x));
        }
        case DG_ACT_GELU_TANH: return pair_mul(x, gelu_logistic(x, gelu_square(x)));
        case DG_ACT_SILU: return pair_mul(x, silu_logistic(x));
        default: return x;
    }
}
__device__ __forceinline__ float activation(int act, float x) { return floats_of(activation(act, pair_of(x))).x; }

struct ValueSlope {
    pair value, slope;
};

// The value and the derivative.
__device__ __forceinline__ ValueSlope activation_slope(int act, pair x) {
    switch (act) {
        case DG_ACT_RELU: {
            const float2 f = floats_of(x);
            return {pair_relu(x), pair_of(f.x > 0.0f ? 1.0f : f.x == f.x ? 0.0f : f.x,
                                                        f.y > 0.0f ? 1.0f : f.y == f.y ? 0.0f : f.y)};
        }
        case DG_ACT_GELU: {
            // Phi(x) = h(|x|) or 1 - h(|x|); the slope is Phi + x bell / sqrt(2 pi)
            const float2 f = floats_of(x);
            const pair a = pair_magnitude(x), bell = gelu_bell(x), tail = gelu_tail(a, bell);
            const float2 h = floats_of(tail);
            const pair phi = pair_of(f.x < 0.0f ? h.x : 1.0f - h.x, f.y < 0.0f ? h.y : 1.0f - h.y);
            return {pair_fma(pair_neg(a), tail, pair_relu(x)),
                    pair_fma(pair_mul(x, bell), pair_of(0.3989422804014327f), phi)};
        }
        case DG_ACT_GELU_TANH: {
            const pair square = gelu_square(x), g = gelu_logistic(x, square);
            const pair du = pair_fma(pair_of(3.0f * kGeluSlope * kGeluCubic), square, pair_of(kGeluSlope));
            const pair v = pair_mul(x, g);   // first: large -x times 0 is 0
            const pair rest = pair_fma(pair_neg(g), pair_of(1.0f), pair_of(1.0f));
            return {v, pair_fma(pair_mul(v, rest), du, g)};
        }
        case DG_ACT_SILU: {
            const pair g = silu_logistic(x), v = pair_mul(x, g);
            const pair rest = pair_fma(pair_neg(g), pair_of(1.0f), pair_of(1.0f));
            return {v, pair_fma(v, rest, g)};
        }
        default: return {x, pair_of(1.0f)};
    }
}

// Calls f with the activation as a compile-time constant: one branch for all
// that f does.
template <int kAct>
struct ActConstant {
    static constexpr int value = kAct;
};
template <typename F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
    switch (act) {
        case DG_ACT_RELU: f(ActConstant<DG_ACT_RELU>{}); break;
        case DG_ACT_GELU: f(ActConstant<DG_ACT_GELU>{}); break;
        case DG_ACT_GELU_TANH: f(ActConstant<DG_ACT_GELU_TANH>{}); break;
        case DG_ACT_SILU: f(ActConstant<DG_ACT_SILU>{}); break;
        default: f(ActConstant<DG_ACT_NONE>{}); break;
    }
}

// acc scale_a scale_b, where the scales' product may be no normal number of
// FP32 though the result is one: the larger scale first where their product
// is small, the smaller one where it is large.
__device__ __forceinline__ bool scale_in_range(float ab) {
    return fabsf(ab) >= 0x1p-126f && fabsf(ab) <= 3.4e38f;
}
__device__ __forceinline__ float scaled(float acc, float a, float b) {
    const float ab = a * b;
    if (scale_in_range(ab)) return acc * ab;
    const float small = fabsf(a) < fabsf(b) ? a : b, large = fabsf(a) < fabsf(b) ? b : a;
    return fabsf(ab) < 1.0f ? acc * large * small : acc * small * large;
}
// acc scale_a scale_b + bias of two elements.
__device__ __forceinline__ pair scale_and_bias(pair acc, pair a, float b, float bias) {
    const pair ab = pair_mul(a, pair_of(b));
    const float2 f = floats_of(ab);
    if (scale_in_range(f.x) && scale_in_range(f.y)) return pair_fma(acc, ab, pair_of(bias));
    const float2 x = floats_of(acc), s = floats_of(a);
    return pair_of(scaled(x.x, s.x, b) + bias, scaled(x.y, s.y, b) + bias);
}
// The same for many products: a scale as whole x rest, whole 2^-62, 1 or 2^64.
// The product of two rests is a normal number (of scales down to 2^-122), and
// acc times both wholes overflows only where the result does.
struct ScaleParts {
    float whole, rest;
};
__device__ __forceinline__ bool scale_is_rest(float s) { return fabsf(s) >= 0x1p-62f && fabsf(s) < 0x1p64f; }
__device__ __forceinline__ ScaleParts scale_parts(float s) {
    if (scale_is_rest(s)) return {1.0f, s};
    return fabsf(s) < 1.0f ? ScaleParts{0x1p-62f, s * 0x1p62f} : ScaleParts{0x1p64f, s * 0x1p-64f};
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
