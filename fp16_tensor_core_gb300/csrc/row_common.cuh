// row_common.cuh -- pieces of the kernels that work on rows of BF16 or FP16
// elements (norm, activation and their gradients).
//
// A thread holds vectors of 8 elements (16 bytes): vector i of a thread is
// vector threadIdx.x + i * blockDim.x of the row, so that a warp's loads are
// whole lines.  Arithmetic is FP32; each output is rounded once.
#pragma once

#include <cstdint>

#include "activation.cuh"
#include "dg_internal.h"
#include "dg_ptx.cuh"

namespace dg {

constexpr int kRowThreads = 512;   // at most, a row

// Rows too wide for the vectors of one block are refused.
constexpr int kRowVectors = 8;     // at most, a thread
static_assert(kRowThreads * kRowVectors * 8 == kMaxRowElements, "widest row");

template <bool kFp16>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kFp16) {
            const float2 t = f16x2_to_f32x2(w[i]);
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return kFp16 ? f32x2_to_f16x2(lo, hi) : f32x2_to_bf16x2(lo, hi);
}

template <bool kFp16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2<kFp16>(f[0], f[1]), pack2<kFp16>(f[2], f[3]), pack2<kFp16>(f[4], f[5]),
                      pack2<kFp16>(f[6], f[7]));
}

// Eight values times `by` as E4M3 codes, saturating, NaN as 0x7F.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float by) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = static_cast<uint32_t>(f32x2_to_e4m3x2(f[4 * i] * by, f[4 * i + 1] * by)) |
               static_cast<uint32_t>(f32x2_to_e4m3x2(f[4 * i + 2] * by, f[4 * i + 3] * by)) << 16;
    return make_uint2(w[0], w[1]);
}

// Eight E4M3 codes times `by`.
__device__ __forceinline__ void decode8(uint2 q, float by, float (&f)[8]) {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)))));
        f[2 * i] = t.x * by;
        f[2 * i + 1] = t.y * by;
    }
}

// 16 bytes that no other block reads.  Not the read-only path: an output may
// be the input itself.
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 load_once8(const void* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// The largest magnitude of eight values, as ordered bits (NaN above all).
__device__ __forceinline__ uint32_t top8(const float (&f)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    return top;
}

// Reductions over a block that give every thread the result.  Two buffers,
// taken in turn: between two uses of one lies the barrier of the other, so
// that one barrier a reduction is enough.
struct RowReduce {
    float2 (*buffer)[kRowThreads / 32];   // [2], shared memory
    int turn = 0;

    __device__ __forceinline__ float2 sum2(float a, float b) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        const int warps = static_cast<int>(blockDim.x) >> 5;
        if (warps == 1) return make_float2(a, b);
        float2* buf = buffer[turn];
        turn ^= 1;
        const int lane = threadIdx.x & 31;
        if (lane == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 t = lane < warps ? buf[lane] : make_float2(0.0f, 0.0f);
        a = t.x;
        b = t.y;
#pragma unroll
        for (int o = kRowThreads / 64; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        return make_float2(__shfl_sync(0xFFFFFFFFu, a, 0), __shfl_sync(0xFFFFFFFFu, b, 0));
    }
    __device__ __forceinline__ float sum(float a) { return sum2(a, 0.0f).x; }

    // Two maxima of ordered bits.
    __device__ __forceinline__ uint2 max2(uint32_t a, uint32_t b) {
        a = __reduce_max_sync(0xFFFFFFFFu, a);
        b = __reduce_max_sync(0xFFFFFFFFu, b);
        const int warps = static_cast<int>(blockDim.x) >> 5;
        if (warps == 1) return make_uint2(a, b);
        uint2* buf = reinterpret_cast<uint2*>(buffer[turn]);
        turn ^= 1;
        const int lane = threadIdx.x & 31;
        if (lane == 0) buf[threadIdx.x >> 5] = make_uint2(a, b);
        __syncthreads();
        const uint2 t = lane < warps ? buf[lane] : make_uint2(0u, 0u);
        return make_uint2(__reduce_max_sync(0xFFFFFFFFu, t.x), __reduce_max_sync(0xFFFFFFFFu, t.y));
    }
    __device__ __forceinline__ uint32_t max1(uint32_t a) { return max2(a, 0u).x; }
};

// A row's scale: fl32(amax / 448), at least 2^-120 so that its reciprocal is
// finite (a row of zeros has a scale too); NaN and infinity stay.
__device__ __forceinline__ float row_scale(uint32_t top_bits) {
    const float s = __fdiv_rn(__uint_as_float(top_bits), 448.0f);
    return s < kRowMinScale ? kRowMinScale : s;
}

// Threads a row of `vectors` vectors gets when each thread holds `each`.
inline int row_threads(int vectors, int each) { return ((vectors + each - 1) / each + 31) / 32 * 32; }

// Sums of columns: out[c] = the sum over parts p of partials[p][c], in the
// order of p within eight runs, joined in order.  partials: [parts][cols].
cudaError_t launch_join_columns(const float* partials, int parts, int cols, float* out, cudaStream_t s);

}  // namespace dg
