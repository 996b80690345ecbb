// attn_common.cuh -- device helpers shared by the attention kernels.
#pragma once

#include <cstdint>

#include "dg_ptx.cuh"

namespace dg {

// Asynchronous copies global -> shared; `bytes` of them are read (the rest
// is zero).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                 :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four E4M3 codes (low byte first) -> two FP16 pairs, exactly.
__device__ __forceinline__ void codes_to_halves(uint32_t codes, uint32_t* lo, uint32_t* hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(*lo), "=r"(*hi) : "r"(codes));
}

__device__ __forceinline__ float4 scaled(float4 x, float w) {
    return make_float4(x.x * w, x.y * w, x.z * w, x.w * w);
}
__device__ __forceinline__ float4 plus_scaled(float4 x, float w, float4 y) {
    return make_float4(fmaf(w, y.x, x.x), fmaf(w, y.y, x.y), fmaf(w, y.z, x.z), fmaf(w, y.w, x.w));
}

// Largest magnitude of 8 BF16 values, as its bits.
__device__ __forceinline__ uint32_t top_abs_bf16(uint4 w) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
    return top;
}

// BF16 queries go to the MMA as FP16, which has more mantissa but less range:
// a row is divided by 2^-14 times the power of two at or below its largest
// magnitude (given as BF16 bits), so that its largest value lies in [2^14,
// 2^15) and FP16's whole range is below it: elements are exact down to 2^-32
// of the largest, and zero only below 2^-40.  (Rows below 2^-112 are divided
// by 2^-126: still exact.)
struct PowerOfTwo {
    float value, inverse;
};
__device__ __forceinline__ PowerOfTwo query_scale(uint32_t top_bf16) {
    const int e = min(max(static_cast<int>(top_bf16 >> 7), 15), 254);   // biased exponent
    return {__uint_as_float(static_cast<uint32_t>(e - 14) << 23), __uint_as_float(static_cast<uint32_t>(268 - e) << 23)};
}
__device__ __forceinline__ uint32_t bf16_to_half2(uint32_t v, float mul) {
    return f32x2_to_f16x2(__uint_as_float(v << 16) * mul, __uint_as_float(v & 0xFFFF0000u) * mul);
}
__device__ __forceinline__ uint4 bf16_to_half8(uint4 v, float mul) {
    return make_uint4(bf16_to_half2(v.x, mul), bf16_to_half2(v.y, mul), bf16_to_half2(v.z, mul),
                      bf16_to_half2(v.w, mul));
}

// Joins n states of one row (each m, l, 2 unused, D sums; `stride` floats
// apart) by one warp, in order, eight at a time with their loads in flight
// together: *m, *l the joined reference and sum, x the joined sums of this
// lane's dims 4 lane + 128 k.
template <int D>
__device__ __forceinline__ void join_states(const float* first, int64_t stride, int n, int lane,
                                            float* m, float* l, float4* x) {
    constexpr int kParts = D > 128 ? 2 : 1;
    const bool live = 4 * lane < D;
    float ref = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kParts; ++k) x[k] = make_float4(0, 0, 0, 0);
    for (int i0 = 0; i0 < n; i0 += 8) {
        float2 ml[8];
        float4 y[8][kParts];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ml[i] = make_float2(-INFINITY, 0.0f);
            if (i0 + i >= n) continue;
            const float* row = first + (i0 + i) * stride;
            ml[i] = *reinterpret_cast<const float2*>(row);
            if (live) {
#pragma unroll
                for (int k = 0; k < kParts; ++k)
                    y[i][k] = *reinterpret_cast<const float4*>(row + 4 + 4 * lane + 128 * k);
            }
        }
        float top = ref;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, ml[i].x);
        const float base = top == -INFINITY ? 0.0f : top;
        const float w0 = ex2(ref - base);
        ref = top;
        sum *= w0;
#pragma unroll
        for (int k = 0; k < kParts; ++k) x[k] = scaled(x[k], w0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i0 + i >= n) continue;
            const float w = ex2(ml[i].x - base);
            sum = fmaf(w, ml[i].y, sum);
#pragma unroll
            for (int k = 0; k < kParts; ++k) x[k] = plus_scaled(x[k], w, y[i][k]);
        }
    }
    *m = ref;
    *l = sum;
}

}  // namespace dg
