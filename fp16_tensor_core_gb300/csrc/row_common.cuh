// row_common.cuh -- pieces of the kernels that work on rows of BF16 or FP16
// elements (norm, activation and their gradients).
//
// A thread holds vectors of 8 elements (16 bytes): vector i of thread t of a
// row's n is vector t + i n of the row, so that a warp's loads are whole
// lines.  Arithmetic is FP32, two elements an instruction; each output is
// rounded once.
#pragma once

#include <cstdint>

#include "activation.cuh"
#include "dg_internal.h"
#include "dg_ptx.cuh"

namespace dg {

constexpr int kRowThreads = 1024;   // at most, a row

// Eight elements as four pairs.
template <bool kFp16>
__device__ __forceinline__ void unpack8(uint4 v, pair (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kFp16) {
            const float2 t = f16x2_to_f32x2(w[i]);
            f[i] = pair_of(t.x, t.y);
        } else {
            f[i] = pair_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        }
    }
}

template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(pair v) {
    const float2 f = floats_of(v);
    return kFp16 ? f32x2_to_f16x2(f.x, f.y) : f32x2_to_bf16x2(f.x, f.y);
}

template <bool kFp16>
__device__ __forceinline__ uint4 pack8(const pair (&f)[4]) {
    return make_uint4(pack2<kFp16>(f[0]), pack2<kFp16>(f[1]), pack2<kFp16>(f[2]), pack2<kFp16>(f[3]));
}

// Eight values times `by` as E4M3 codes, saturating, NaN as 0x7F.
__device__ __forceinline__ uint2 codes8(const pair (&f)[4], float by) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = floats_of(pair_mul(f[2 * i], pair_of(by))), b = floats_of(pair_mul(f[2 * i + 1], pair_of(by)));
        w[i] = static_cast<uint32_t>(f32x2_to_e4m3x2(a.x, a.y)) | static_cast<uint32_t>(f32x2_to_e4m3x2(b.x, b.y)) << 16;
    }
    return make_uint2(w[0], w[1]);
}

// Eight E4M3 codes times `by`.
__device__ __forceinline__ void decode8(uint2 q, float by, pair (&f)[4]) {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)))));
        f[i] = pair_mul(pair_of(t.x, t.y), pair_of(by));
    }
}

// 16 (8) bytes that no other block reads, where `take`; else what was there.
// Predicated, without branches in a row's loop.
// Not the read-only path: an output may be the input itself.
__device__ __forceinline__ void load_if(bool take, const void* p, uint4& v) {
    asm volatile("{\n\t.reg .pred q;\n\t"
                 "setp.ne.u32 q, %5, 0;\n\t"
                 "@q ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w) : "l"(p), "r"(static_cast<uint32_t>(take)));
}
__device__ __forceinline__ void store_if(bool take, void* p, uint4 v) {
    asm volatile("{\n\t.reg .pred q;\n\t"
                 "setp.ne.u32 q, %5, 0;\n\t"
                 "@q st.global.v4.u32 [%0], {%1, %2, %3, %4};\n\t}"
                 :: "l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(static_cast<uint32_t>(take)));
}
__device__ __forceinline__ void store_if(bool take, void* p, uint2 v) {
    asm volatile("{\n\t.reg .pred q;\n\t"
                 "setp.ne.u32 q, %3, 0;\n\t"
                 "@q st.global.v2.u32 [%0], {%1, %2};\n\t}"
                 :: "l"(p), "r"(v.x), "r"(v.y), "r"(static_cast<uint32_t>(take)));
}
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v = make_uint4(0, 0, 0, 0);
    load_if(true, p, v);
    return v;
}
__device__ __forceinline__ uint2 load_once8(const void* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
// A pointer as it is known after pdl_wait: reads through it cannot come first.
__device__ __forceinline__ const uint16_t* behind_wait(const uint16_t* p) {
    asm volatile("" : "+l"(p) :: "memory");
    return p;
}
// A vector of the norm's weight (every block reads it for every row, from
// L1), or zeros.  The compiler may move it: past pdl_wait's call, `weight` is
// taken from behind_wait.
__device__ __forceinline__ uint4 weight_if(bool take, const uint16_t* weight, int at) {
    uint4 v = make_uint4(0, 0, 0, 0);
    asm("{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %5, 0;\n\t"
        "@q ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(weight + 8 * at), "r"(static_cast<uint32_t>(take)));
    return v;
}

// A row to come moves into L2 (one thread; 16-byte aligned, a multiple of 16
// bytes): no registers are held meanwhile.
__device__ __forceinline__ void prefetch_row(const void* p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(p), "r"(bytes) : "memory");
}

// The line at p is brought into L2 (any alignment; p inside the tensor).
__device__ __forceinline__ void prefetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" :: "l"(p)); }

// Forgets what has been formed from packed elements: they are unpacked again,
// where the compiler would keep (and spill) twice their registers.
__device__ __forceinline__ void forget(uint4& v) { asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)); }

// The largest magnitude of eight values and of one that there is.
__device__ __forceinline__ float top8(const pair (&f)[4], float top) {
#pragma unroll
    for (int i = 0; i < 4; ++i) top = pair_top(f[i], top);
    return top;
}

// The threads of a row: a block, or for narrow rows (kNarrow) a power of two
// of lanes, several rows to a warp.  Two kernels for the two: where a row is
// a block's, its addresses are uniform and its reductions have no loops.
template <bool kNarrow>
struct RowTeam {
    int size;     // threads a row
    int at;       // this thread's place in its row
    int row;      // the row's place among those of the block
    int rows;     // rows of a block
    __device__ __forceinline__ explicit RowTeam(int team_size) {
        if constexpr (kNarrow) {
            size = team_size;
            at = static_cast<int>(threadIdx.x) & (size - 1);
            row = static_cast<int>(threadIdx.x) / size;
            rows = static_cast<int>(blockDim.x) / size;
        } else {
            size = static_cast<int>(blockDim.x);
            at = static_cast<int>(threadIdx.x);
            row = 0;
            rows = 1;
        }
    }
};

// Reductions over a row's threads that give every one the result; all threads
// of the block take part.  Two buffers, taken in turn: between two uses of
// one lies the barrier of the other, so that one barrier a reduction is
// enough.
template <bool kNarrow>
struct RowReduce {
    float2 (*buffer)[kRowThreads / 32];   // [2], shared memory
    int size;                             // threads a row
    int turn = 0;

    __device__ __forceinline__ float sum(float a) {
        if constexpr (kNarrow) {
            for (int o = size >> 1; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            return a;
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            return tree(exchange(make_float2(a, 0.0f)).x);
        }
    }
    __device__ __forceinline__ float2 sum2(float a, float b) {
        if constexpr (kNarrow) {
            return make_float2(sum(a), sum(b));
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
                b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
            }
            const float2 t = exchange(make_float2(a, b));
            return make_float2(tree(t.x), tree(t.y));
        }
    }

    // Maxima of magnitudes (as ordered bits: NaN above all).
    __device__ __forceinline__ float max1(float a) {
        if constexpr (kNarrow) return narrow_max(a);
        const float2 t = exchange(make_float2(warp_max(a), 0.0f));
        return warp_max(t.x);
    }
    __device__ __forceinline__ float2 max2(float a, float b) {
        if constexpr (kNarrow) return make_float2(narrow_max(a), narrow_max(b));
        const float2 t = exchange(make_float2(warp_max(a), warp_max(b)));
        return make_float2(warp_max(t.x), warp_max(t.y));
    }

private:
    static __device__ __forceinline__ float warp_max(float a) {
        return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(a)));
    }
    __device__ __forceinline__ float narrow_max(float a) {
        uint32_t v = __float_as_uint(a);
        for (int o = size >> 1; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
        return __uint_as_float(v);
    }
    // The sum of what exchange gave.
    static __device__ __forceinline__ float tree(float a) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        return a;
    }
    // Every warp's value to every warp: lane i gets warp i's (or zero).
    __device__ __forceinline__ float2 exchange(float2 v) {
        float2* buf = buffer[turn];
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        const unsigned from = threadIdx.x & 31;
        return from < blockDim.x >> 5 ? buf[from] : make_float2(0.0f, 0.0f);
    }
};
static_assert(kRowThreads / 32 == 32, "exchange");

__device__ __forceinline__ float pair_sum(pair v) {
    const float2 f = floats_of(v);
    return f.x + f.y;
}

// Eight columns' sums, 16-byte aligned.
__device__ __forceinline__ void store_sums(float* dst, const pair (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = floats_of(f[2 * i]), b = floats_of(f[2 * i + 1]);
        reinterpret_cast<float4*>(dst)[i] = make_float4(a.x, a.y, b.x, b.y);
    }
}

// A tensor's scale: amax / 448, 1 for an all-zero one.
__device__ __forceinline__ float scale_of_amax(float a) { return a == 0.0f ? 1.0f : __fdiv_rn(a, 448.0f); }

// A row's scale: fl32(amax / 448), at least 2^-120 so that its reciprocal is
// finite (a row of zeros has a scale too); NaN and infinity stay.  The
// quotient as a product and its remainder's (Markstein, 1990), the rounded
// quotient for every mantissa: a remainder of a division by 7 is at least 1/14
// of a step from a tie.  Every thread of a row waits for it (through
// __fdiv_rn, 4000 x 8192 BF16 to codes took 21.4 us instead of 21.0).
__device__ __forceinline__ float row_scale(float top) {
    constexpr float kInv = 1.0f / 448.0f;
    const float q = top * kInv;
    const float s = top == __int_as_float(0x7F800000) ? top : fmaf(fmaf(-448.0f, q, top), kInv, q);
    return s < kRowMinScale ? kRowMinScale : s;
}

// What multiplies a row's values to give codes: the reciprocal of the scale
// that is written, rounded once (2^120 at most; 0 of an infinite scale).
__device__ __forceinline__ float row_factor(float scale) { return __frcp_rn(scale); }

// How rows are dealt out: `each` vectors a thread, `team` threads a row,
// blocks of `threads`, and as many of them as are resident at once.
struct RowPlan {
    int each, team, threads, blocks;
    bool narrow;
};
// Whether the kernels behind `limits` hold every row of up to kMaxRowElements
// (wider ones are refused before): row_plan takes the first that holds a row.
constexpr bool hold_widest_row(const int (&limits)[3]) {
    for (int k = 0; k < 3; ++k)
        if (limits[k] % 32 == 0 && limits[k] * (2 << k) * 8 >= kMaxRowElements) return true;
    return false;
}
// limits: a block's threads at most, per_sm: threads an SM holds at the
// kernel's registers, both by vectors a thread (2, 4, 8); 0 where there is no
// kernel of that many.
inline RowPlan row_plan(int64_t rows, int cols, int sm_count, const int (&limits)[3], const int (&per_sm)[3]) {
    const int vectors = cols >> 3;
    int k = 0;
    while (k < 2 && (vectors + (2 << k) - 1) / (2 << k) > limits[k]) ++k;
    RowPlan p{};
    p.each = 2 << k;
    const int need = (vectors + p.each - 1) / p.each;
    int64_t teams = rows;   // blocks that every row would fill
    if (need <= 16) {
        p.narrow = true;
        p.team = 1;
        while (p.team < need) p.team *= 2;
        p.threads = 128;
        teams = (rows + 128 / p.team - 1) / (128 / p.team);
    } else {
        p.team = p.threads = (need + 31) / 32 * 32;
    }
    const int64_t resident = static_cast<int64_t>(sm_count) * (per_sm[k] / p.threads > 0 ? per_sm[k] / p.threads : 1);
    p.blocks = static_cast<int>(teams < resident ? teams : resident);
    return p;
}

// Sums of columns: out[c] = the sum over parts p of partials[p][c], in an order
// that only their number and the columns' decides.  partials: [parts][cols].
cudaError_t launch_join_columns(const float* partials, int parts, int cols, float* out, cudaStream_t s);

}  // namespace dg
