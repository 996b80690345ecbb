// k_kvcache.cu -- what follows the QKV projection: rotary positions, and the
// E4M3 key/value cache written (rotation and quantisation in one pass) and
// read back.
//
// [FP8-guide] = "DeepGEMM实战：FP8矩阵乘法与JIT编译优化指南".  §3.2 and §4.3
// give the quantisation rule; here the tensor that shares a scale is one
// head of one token, so that a token can be added without touching the
// others.  All three operators are bound by HBM: each element is read and
// written once.
#include <cuda_runtime.h>

#include <algorithm>

#include "dg_internal.h"
#include "dg_ptx.cuh"

namespace dg {
namespace {

// 16 bytes read once (no L1 line kept).  Not the read-only path: dg_rope may
// run in place.
__device__ __forceinline__ uint4 ld_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

template <bool kFp16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (kFp16) {
        return f16x2_to_f32x2(w);
    } else {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
}
template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return kFp16 ? f32x2_to_f16x2(lo, hi) : f32x2_to_bf16x2(lo, hi);
}
template <bool kFp16>
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<kFp16>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <bool kFp16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2<kFp16>(x[0], x[1]), pack2<kFp16>(x[2], x[3]),
                      pack2<kFp16>(x[4], x[5]), pack2<kFp16>(x[6], x[7]));
}

// ------------------------------------------------------------ rotary table

// table[p][i] = magnitude * (cos, sin)(p * f_i).  Everything up to the final
// rounding is FP64: at p = 10^6 an FP32 angle would already be off by 0.06.
// One block column per frequency, so that each thread forms its frequency
// once and then walks over positions.
__global__ void __launch_bounds__(256)
rope_table_kernel(float2* __restrict__ table, int64_t positions, int half, dg_rope_scaling s) {
    pdl_wait();
    const int i = blockIdx.y;
    const double r = 2.0 * half;
    double base = s.base;
    if (s.scaling == DG_ROPE_NTK && half > 1) base *= pow(s.factor, r / (r - 2.0));
    double f = pow(base, -2.0 * i / r);
    if (s.scaling == DG_ROPE_LINEAR) f /= s.factor;
    if (s.scaling == DG_ROPE_BY_PARTS) {
        const double turns = s.original_positions * f / 6.283185307179586476925;
        const double keep = fmin(fmax((turns - s.slow_rotations) /
                                      (s.fast_rotations - s.slow_rotations), 0.0), 1.0);
        f = (1.0 - keep) * (f / s.factor) + keep * f;
    }
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t p = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; p < positions;
         p += stride) {
        double sn, cs;
        sincos(static_cast<double>(p) * f, &sn, &cs);
        table[p * half + i] = make_float2(static_cast<float>(s.magnitude * cs),
                                          static_cast<float>(s.magnitude * sn));
    }
}

// ------------------------------------------------------------------ rotary

struct RopeArgs {
    const uint16_t* x;
    uint16_t* out;
    int64_t x_ts, x_hs, o_ts, o_hs;   // token and head strides, elements
    int64_t tokens;
    int heads;
    int rot8;              // rotated dims / 8
    int items;             // work items per head
    int head_steps;        // heads are taken in this many interleaved sets (one per thread)
    int threads_per_token; // items * head_steps
    int tokens_per_block;
    const int32_t* positions;
    const float4* table;   // rows of rotary_dim floats: (cos, sin) per pair
    int64_t table_positions;
    float sign;            // -1 for the transposed rotation
    uint32_t* status;
};

// A thread owns one item (8 rotated pairs of the half layout, 4 of the
// interleaved one, or 8 dims that are copied) of one token for kHeads heads:
// its cosines and sines stay in registers across the heads, and both halves
// of a pair are in its hands, so each element is read and written once.
template <bool kFp16, bool kHalf, int kHeads>
__global__ void __launch_bounds__(256)
rope_kernel(const RopeArgs a) {
    const int local = static_cast<int>(threadIdx.x) / a.threads_per_token;
    const int rest = static_cast<int>(threadIdx.x) - local * a.threads_per_token;
    const int item = rest % a.items, h0 = rest / a.items;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block + local;
    pdl_wait();
    if (local >= a.tokens_per_block || t >= a.tokens) return;
    const int64_t pos = a.positions[t];
    if (pos < 0 || pos >= a.table_positions) {
        if (rest == 0) atomicOr(a.status, kStatusBadArgument);
        return;
    }
    const int pair_items = kHalf ? a.rot8 / 2 : a.rot8;
    const bool turn = item < pair_items;
    // first (and for the half layout second) 8 dims of the item
    const int d0 = kHalf && !turn ? 8 * (item - pair_items + a.rot8) : 8 * item;
    const int d1 = kHalf && turn ? d0 + 4 * a.rot8 : d0;
    const uint16_t* x = a.x + t * a.x_ts;
    uint16_t* out = a.out + t * a.o_ts;
    uint4 v0[kHeads], v1[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
        const int h = h0 + k * a.head_steps;
        if (h < a.heads) {
            v0[k] = ld_once(x + h * a.x_hs + d0);
            if (kHalf && turn) v1[k] = ld_once(x + h * a.x_hs + d1);
        }
    }
    constexpr int kPairs = kHalf ? 8 : 4;
    float c[kPairs], s[kPairs];
    if (turn) {
        const float4* row = a.table + (pos * (4 * a.rot8) + item * kPairs) / 2;
#pragma unroll
        for (int i = 0; i < kPairs / 2; ++i) {
            const float4 f = __ldg(row + i);
            c[2 * i] = f.x;
            s[2 * i] = a.sign * f.y;
            c[2 * i + 1] = f.z;
            s[2 * i + 1] = a.sign * f.w;
        }
    }
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
        const int h = h0 + k * a.head_steps;
        if (h >= a.heads) continue;
        if (turn) {
            float p[8];
            unpack8<kFp16>(v0[k], p);
            if constexpr (kHalf) {
                float q[8], y0[8], y1[8];
                unpack8<kFp16>(v1[k], q);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y0[i] = p[i] * c[i] - q[i] * s[i];
                    y1[i] = q[i] * c[i] + p[i] * s[i];
                }
                v0[k] = pack8<kFp16>(y0);
                *reinterpret_cast<uint4*>(out + h * a.o_hs + d1) = pack8<kFp16>(y1);
            } else {
                float y[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[2 * i] = p[2 * i] * c[i] - p[2 * i + 1] * s[i];
                    y[2 * i + 1] = p[2 * i + 1] * c[i] + p[2 * i] * s[i];
                }
                v0[k] = pack8<kFp16>(y);
            }
        }
        *reinterpret_cast<uint4*>(out + h * a.o_hs + d0) = v0[k];
    }
}

// ------------------------------------------------------------ cache writes

struct AppendArgs {
    const uint16_t* q;
    uint16_t* q_out;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_ts, q_hs, o_ts, o_hs, k_ts, k_hs, v_ts, v_hs;
    int q_heads;
    int dim;
    int rot;               // rotated dims (0: none)
    int interleaved;
    const int32_t* positions;
    const float* table;
    int64_t table_positions;
    const int32_t* slots;
    dg_kv_cache cache;
    int page_shift;
    int row_step;          // rows of a token between a lane group's rows
    uint32_t* status;
};

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// One row (one head of one token) per group of kLanes lanes, 8 dims a lane;
// a group takes kRows rows of its token.  A rotated lane also reads the 8
// dims that its own are paired with (the other lane's line, from L1).
template <bool kFp16, int kLanes, int kRows>
__global__ void __launch_bounds__(128)
kv_append_kernel(const AppendArgs a) {
    constexpr int kGroups = 128 / kLanes;
    const int l = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int64_t t = blockIdx.x;
    const int d = 8 * l;
    const bool live = d < a.dim;
    const bool turn = d < a.rot;
    const int half = a.rot / 2;
    const bool upper = !a.interleaved && d >= half;
    const int dp = !turn || a.interleaved ? d : upper ? d - half : d + half;
    const int kv_heads = a.cache.kv_heads;
    const int rows = a.q_heads + 2 * kv_heads;
    const int row0 = static_cast<int>(blockIdx.y) * (kGroups * kRows) + group;
    pdl_wait();
    const int slot = a.slots[t];
    const int64_t nslots = a.cache.pages << a.page_shift;
    const int64_t pos = a.rot > 0 ? a.positions[t] : 0;
    const bool bad = slot >= nslots || (a.rot > 0 && (pos < 0 || pos >= a.table_positions));
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, kStatusBadArgument);
        return;
    }

    uint4 own[kRows], pair[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const int r = row0 + j * kGroups;
        own[j] = pair[j] = make_uint4(0, 0, 0, 0);
        if (r < rows && live) {
            const uint16_t* src =
                r < a.q_heads ? a.q + t * a.q_ts + r * a.q_hs
                : r < a.q_heads + kv_heads ? a.k + t * a.k_ts + (r - a.q_heads) * a.k_hs
                                           : a.v + t * a.v_ts + (r - a.q_heads - kv_heads) * a.v_hs;
            own[j] = *reinterpret_cast<const uint4*>(src + d);
            if (turn && !a.interleaved && r < a.q_heads + kv_heads)
                pair[j] = *reinterpret_cast<const uint4*>(src + dp);
        }
    }
    __syncwarp();   // q may be rotated in place: a row is read before any of it is written
    // cosines and (signed) sines of this lane's dims
    float c[8], s[8];
    if (turn) {
        const float* row = a.table + pos * a.rot;
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(row + d + 4 * i));
                c[4 * i] = c[4 * i + 1] = f.x;
                s[4 * i] = -f.y;
                s[4 * i + 1] = f.y;
                c[4 * i + 2] = c[4 * i + 3] = f.z;
                s[4 * i + 2] = -f.w;
                s[4 * i + 3] = f.w;
            }
        } else {
            const int i0 = upper ? d - half : d;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(row + 2 * i0 + 4 * i));
                c[2 * i] = f.x;
                s[2 * i] = upper ? f.y : -f.y;
                c[2 * i + 1] = f.z;
                s[2 * i + 1] = upper ? f.w : -f.w;
            }
        }
    }
    const int page = slot >> a.page_shift, at = slot & ((1 << a.page_shift) - 1);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const int r = row0 + j * kGroups;
        const bool is_q = r < a.q_heads, is_k = !is_q && r < a.q_heads + kv_heads;
        float x[8];
        unpack8<kFp16>(own[j], x);
        if (turn && (is_q || is_k)) {
            float y[8], p[8];
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = x[i ^ 1];
            } else {
                unpack8<kFp16>(pair[j], p);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i] * c[i] + p[i] * s[i];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = y[i];
        }
        if (is_q) {
            if (live)
                *reinterpret_cast<uint4*>(a.q_out + t * a.o_ts + r * a.o_hs + d) = pack8<kFp16>(x);
        }
        // The rotated key goes to its scale and code in FP32, not through a
        // 16-bit rounding.
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, abs_bits(x[i]));
#pragma unroll
        for (int w = kLanes / 2; w > 0; w >>= 1)
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, w));
        if (is_q || r >= rows || slot < 0) continue;
        const int h = is_k ? r - a.q_heads : r - a.q_heads - kv_heads;
        const int64_t row = ((static_cast<int64_t>(page) * kv_heads + h) << a.page_shift) + at;
        const bool finite = top < 0x7F800000u;
        const float scale = finite ? fmaxf(__fdiv_rn(__uint_as_float(top), 448.0f), kKvMinScale)
                                   : __int_as_float(0x7FC00000);
        if (live) {
            uint32_t code[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                code[i] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale));
            const uint2 packed = finite ? make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16)
                                        : make_uint2(0, 0);
            uint8_t* codes = is_k ? a.cache.k : a.cache.v;
            *reinterpret_cast<uint2*>(codes + row * a.dim + d) = packed;
        }
        if (l == 0) (is_k ? a.cache.k_scale : a.cache.v_scale)[row] = scale;
    }
}

// ------------------------------------------------------------- cache reads

struct ReadArgs {
    dg_kv_cache cache;
    int page_shift;
    const int32_t* slots;
    int64_t tokens;
    uint16_t* k;
    uint16_t* v;
    int64_t k_ts, k_hs, v_ts, v_hs;
    int chunks;            // head_dim / 16
    int per_token;         // chunks * kv_heads * tensors
    int tokens_per_block;
    uint32_t* status;
};

// 16 codes of one row a thread and step: code x scale in FP32 (exact: 4 + 24
// bits need no more than one rounding), rounded once to the output type.
template <bool kFp16>
__global__ void __launch_bounds__(256)
kv_read_kernel(const ReadArgs a) {
    pdl_wait();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block;
    const int n = static_cast<int>(min(static_cast<int64_t>(a.tokens_per_block), a.tokens - t0)) *
                  a.per_token;
    const int64_t nslots = a.cache.pages << a.page_shift;
    const int kv_heads = a.cache.kv_heads;
    constexpr int kU = 4;
    for (int i0 = threadIdx.x; i0 < n; i0 += 256 * kU) {
        uint4 code[kU];
        float scale[kU];
        uint16_t* dst[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + 256 * u;
            dst[u] = nullptr;
            if (i >= n) continue;
            const int lt = i / a.per_token, in_token = i - lt * a.per_token;
            const int row = in_token / a.chunks, chunk = in_token - row * a.chunks;
            const bool is_v = a.k == nullptr || row >= kv_heads;
            const int h = row >= kv_heads ? row - kv_heads : row;
            const int64_t t = t0 + lt;
            const int slot = a.slots[t];
            dst[u] = (is_v ? a.v + t * a.v_ts + h * a.v_hs : a.k + t * a.k_ts + h * a.k_hs) + 16 * chunk;
            if (slot >= nslots) {
                atomicOr(a.status, kStatusBadArgument);
                dst[u] = nullptr;
            } else if (slot < 0) {
                code[u] = make_uint4(0, 0, 0, 0);
                scale[u] = 0.0f;
            } else {
                const int64_t page = slot >> a.page_shift;
                const int64_t r = ((page * kv_heads + h) << a.page_shift) +
                                  (slot & ((1 << a.page_shift) - 1));
                code[u] = ld_once((is_v ? a.cache.v : a.cache.k) + (r * a.chunks + chunk) * 16);
                scale[u] = __ldg((is_v ? a.cache.v_scale : a.cache.k_scale) + r);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (dst[u] == nullptr) continue;
            const uint32_t w[4] = {code[u].x, code[u].y, code[u].z, code[u].w};
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 lo = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i])));
                const float2 hi = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> 16)));
                o[2 * i] = pack2<kFp16>(lo.x * scale[u], lo.y * scale[u]);
                o[2 * i + 1] = pack2<kFp16>(hi.x * scale[u], hi.y * scale[u]);
            }
            uint4* p = reinterpret_cast<uint4*>(dst[u]);
            p[0] = make_uint4(o[0], o[1], o[2], o[3]);
            p[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

template <bool kFp16, bool kHalf>
cudaError_t rope_dispatch(const RopeArgs& a, int heads_per_thread, dim3 grid, cudaStream_t s) {
    return heads_per_thread == 4
               ? launch_kernel(rope_kernel<kFp16, kHalf, 4>, grid, dim3(256), 0, s, a)
               : launch_kernel(rope_kernel<kFp16, kHalf, 1>, grid, dim3(256), 0, s, a);
}

template <bool kFp16>
cudaError_t append_dispatch(const AppendArgs& a, int64_t tokens, int rows, bool few, cudaStream_t s) {
    const int lanes = a.dim <= 64 ? 8 : a.dim <= 128 ? 16 : 32;
    const int per_block = 128 / lanes * (few ? 1 : 4);
    const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>((rows + per_block - 1) / per_block));
    const dim3 block(128);
    if (few) {
        if (lanes == 8) return launch_kernel(kv_append_kernel<kFp16, 8, 1>, grid, block, 0, s, a);
        if (lanes == 16) return launch_kernel(kv_append_kernel<kFp16, 16, 1>, grid, block, 0, s, a);
        return launch_kernel(kv_append_kernel<kFp16, 32, 1>, grid, block, 0, s, a);
    }
    if (lanes == 8) return launch_kernel(kv_append_kernel<kFp16, 8, 4>, grid, block, 0, s, a);
    if (lanes == 16) return launch_kernel(kv_append_kernel<kFp16, 16, 4>, grid, block, 0, s, a);
    return launch_kernel(kv_append_kernel<kFp16, 32, 4>, grid, block, 0, s, a);
}

int shift_of(int page_size) {
    int k = 0;
    while ((1 << k) < page_size) ++k;
    return k;
}

}  // namespace

cudaError_t launch_rope_table(float* table, int64_t positions, int rotary_dim,
                              const dg_rope_scaling& sc, int sm_count, cudaStream_t s) {
    const int half = rotary_dim / 2;
    const int64_t need = (positions + 255) / 256;
    const unsigned x = static_cast<unsigned>(std::min<int64_t>(need, std::max(1, 16 * sm_count / half)));
    return launch_kernel(rope_table_kernel, dim3(x, static_cast<unsigned>(half)), dim3(256), 0, s,
                         reinterpret_cast<float2*>(table), positions, half, sc);
}

cudaError_t launch_rope(const dg_heads& x, const dg_heads& out, int64_t tokens, int heads,
                        int head_dim, const int32_t* positions, const dg_rotary& rot, bool inverse,
                        bool fp16, int sm_count, uint32_t* status, cudaStream_t s) {
    RopeArgs a;
    a.x = static_cast<const uint16_t*>(x.data);
    a.out = static_cast<uint16_t*>(out.data);
    a.x_ts = x.token_stride;
    a.x_hs = x.head_stride;
    a.o_ts = out.token_stride;
    a.o_hs = out.head_stride;
    a.tokens = tokens;
    a.rot8 = rot.rotary_dim / 8;
    a.heads = heads;
    const bool half = rot.layout == DG_ROPE_HALF;
    a.items = half ? head_dim / 8 - a.rot8 / 2 : head_dim / 8;
    // Four heads a thread once that still leaves every SM two blocks.
    int per_thread = 4;
    if (tokens * heads * a.items < static_cast<int64_t>(4) * 2 * sm_count * 256) per_thread = 1;
    a.head_steps = (heads + per_thread - 1) / per_thread;
    // A token has to fit one block: more heads a token than that are taken by further launches.
    const int most = 256 / a.items;
    const int64_t chunk_heads = static_cast<int64_t>(most) * per_thread;
    a.positions = positions;
    a.table = reinterpret_cast<const float4*>(rot.table);
    a.table_positions = rot.positions;
    a.sign = inverse ? -1.0f : 1.0f;
    a.status = status;
    for (int h = 0; h < heads; h += static_cast<int>(chunk_heads)) {
        RopeArgs b = a;
        b.x += h * a.x_hs;
        b.out += h * a.o_hs;
        b.heads = static_cast<int>(std::min<int64_t>(chunk_heads, heads - h));
        b.head_steps = (b.heads + per_thread - 1) / per_thread;
        b.threads_per_token = b.items * b.head_steps;
        b.tokens_per_block = 256 / b.threads_per_token;
        const dim3 grid(static_cast<unsigned>((tokens + b.tokens_per_block - 1) / b.tokens_per_block));
        cudaError_t e;
        if (fp16)
            e = half ? rope_dispatch<true, true>(b, per_thread, grid, s)
                     : rope_dispatch<true, false>(b, per_thread, grid, s);
        else
            e = half ? rope_dispatch<false, true>(b, per_thread, grid, s)
                     : rope_dispatch<false, false>(b, per_thread, grid, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_kv_append(const dg_heads* q, const dg_heads* q_out, int q_heads,
                             const dg_heads& k, const dg_heads& v, int64_t tokens,
                             const int32_t* positions, const dg_rotary* rot, const int32_t* slots,
                             const dg_kv_cache& cache, bool fp16, int sm_count, uint32_t* status,
                             cudaStream_t s) {
    AppendArgs a{};
    if (q != nullptr) {
        a.q = static_cast<const uint16_t*>(q->data);
        a.q_ts = q->token_stride;
        a.q_hs = q->head_stride;
        a.q_out = static_cast<uint16_t*>(q_out->data);
        a.o_ts = q_out->token_stride;
        a.o_hs = q_out->head_stride;
        a.q_heads = q_heads;
    }
    a.k = static_cast<const uint16_t*>(k.data);
    a.k_ts = k.token_stride;
    a.k_hs = k.head_stride;
    a.v = static_cast<const uint16_t*>(v.data);
    a.v_ts = v.token_stride;
    a.v_hs = v.head_stride;
    a.dim = cache.head_dim;
    if (rot != nullptr) {
        a.rot = rot->rotary_dim;
        a.interleaved = rot->layout == DG_ROPE_INTERLEAVED;
        a.table = rot->table;
        a.table_positions = rot->positions;
        a.positions = positions;
    }
    a.slots = slots;
    a.cache = cache;
    a.page_shift = shift_of(cache.page_size);
    a.status = status;
    const int rows = a.q_heads + 2 * cache.kv_heads;
    // One row a lane group while the call has too few rows to fill the SMs
    // (16 groups of 4 warps' worth each), four otherwise.
    const bool few = tokens * rows < static_cast<int64_t>(sm_count) * 512;
    return fp16 ? append_dispatch<true>(a, tokens, rows, few, s)
                : append_dispatch<false>(a, tokens, rows, few, s);
}

cudaError_t launch_kv_read(const dg_kv_cache& cache, const int32_t* slots, int64_t tokens,
                           const dg_heads* k, const dg_heads* v, bool fp16, int sm_count,
                           uint32_t* status, cudaStream_t s) {
    ReadArgs a{};
    a.cache = cache;
    a.page_shift = shift_of(cache.page_size);
    a.slots = slots;
    a.tokens = tokens;
    if (k != nullptr) {
        a.k = static_cast<uint16_t*>(k->data);
        a.k_ts = k->token_stride;
        a.k_hs = k->head_stride;
    }
    if (v != nullptr) {
        a.v = static_cast<uint16_t*>(v->data);
        a.v_ts = v->token_stride;
        a.v_hs = v->head_stride;
    }
    a.chunks = cache.head_dim / 16;
    a.per_token = a.chunks * cache.kv_heads * ((k != nullptr) + (v != nullptr));
    // About 1024 items (4 a thread) a block, fewer while that leaves SMs idle.
    int per_block = std::max(1, 1024 / a.per_token);
    while (per_block > 1 && tokens / per_block < 4 * sm_count) per_block /= 2;
    a.tokens_per_block = per_block;
    a.status = status;
    const dim3 grid(static_cast<unsigned>((tokens + per_block - 1) / per_block));
    return fp16 ? launch_kernel(kv_read_kernel<true>, grid, dim3(256), 0, s, a)
                : launch_kernel(kv_read_kernel<false>, grid, dim3(256), 0, s, a);
}

}  // namespace dg
