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
#include <climits>

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

__device__ __forceinline__ uint2 ld_once8(const void* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
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
// once and then walks over positions.  Bound by FP64 arithmetic, and in small
// tables by the one pow of a thread: 8192 positions of 64 pairs 140 us (by
// parts 163), 131072 of 64 601, 10^6 of 32 1900 (17 G entries/s; its bytes
// would take 38).  A program makes its table once.
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
    int head_steps;        // heads are taken in this many interleaved sets
    int sets;              // sets a block holds: all of them, or what fits it
    int head_blocks;       // blocks that share out a token's sets
    int threads_per_token; // items * sets
    int tokens_per_block;
    const int32_t* positions;   // null: nothing is rotated
    const float4* table;   // rows of rotary_dim floats: (cos, sin) per pair
    int64_t table_positions;
    float sign;            // -1 for the transposed rotation
    const int32_t* slots;  // beside a cache write: a token whose slot is past
    int64_t nslots;        // the cache is left alone; else null
    uint32_t* status;
};

// A thread owns one item (8 rotated pairs, or 16 dims that are copied) of one
// token for kHeads heads:
// its cosines and sines stay in registers across the heads, and both halves
// of a pair are in its hands, so each element is read and written once:
// 16385 tokens x 32 heads of 128, half of each turned, 42.5 us (6.4 TB/s, 0.95
// of a copy).
template <bool kFp16, bool kHalf, int kHeads>
__device__ __forceinline__ void rope_block(const RopeArgs& a, int token_block, int head_block) {
    const int local = static_cast<int>(threadIdx.x) / a.threads_per_token;
    const int rest = static_cast<int>(threadIdx.x) - local * a.threads_per_token;
    const int set = rest / a.items;
    const int item = rest - set * a.items, h0 = head_block * a.sets + set;
    const int64_t t = static_cast<int64_t>(token_block) * a.tokens_per_block + local;
    if (local >= a.tokens_per_block || t >= a.tokens || h0 >= a.head_steps) return;
    const int64_t pos = a.positions != nullptr ? a.positions[t] : 0;
    const int slot = a.slots != nullptr ? a.slots[t] : -1;
    const bool turn = item < a.rot8 / 2, apart = kHalf && turn;
    // first and second 8 dims of the item
    const int d0 = apart ? 8 * item : 16 * item;
    const int d1 = apart ? d0 + 4 * a.rot8 : d0 + 8;
    const uint16_t* x = a.x + t * a.x_ts;
    uint16_t* out = a.out + t * a.o_ts;
    uint4 v0[kHeads], v1[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
        const int h = h0 + k * a.head_steps;
        if (h < a.heads) {
            v0[k] = ld_once(x + h * a.x_hs + d0);
            v1[k] = ld_once(x + h * a.x_hs + d1);
        }
    }
    if (a.positions != nullptr && (pos < 0 || pos >= a.table_positions)) {
        if (rest == 0) atomicOr(a.status, kStatusBadArgument);
        return;
    }
    if (a.slots != nullptr && slot >= a.nslots) return;   // the cache's blocks report it
    float c[8], s[8];
    if (turn) {
        const float4* row = a.table + (pos * (4 * a.rot8) + item * 8) / 2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
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
            float p[8], q[8], y0[8], y1[8];
            unpack8<kFp16>(v0[k], p);
            unpack8<kFp16>(v1[k], q);
            if constexpr (kHalf) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y0[i] = p[i] * c[i] - q[i] * s[i];
                    y1[i] = q[i] * c[i] + p[i] * s[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y0[2 * i] = p[2 * i] * c[i] - p[2 * i + 1] * s[i];
                    y0[2 * i + 1] = p[2 * i + 1] * c[i] + p[2 * i] * s[i];
                    y1[2 * i] = q[2 * i] * c[4 + i] - q[2 * i + 1] * s[4 + i];
                    y1[2 * i + 1] = q[2 * i + 1] * c[4 + i] + q[2 * i] * s[4 + i];
                }
            }
            v0[k] = pack8<kFp16>(y0);
            v1[k] = pack8<kFp16>(y1);
        }
        *reinterpret_cast<uint4*>(out + h * a.o_hs + d0) = v0[k];
        *reinterpret_cast<uint4*>(out + h * a.o_hs + d1) = v1[k];
    }
}

template <bool kFp16, bool kHalf, int kHeads>
__global__ void __launch_bounds__(256)
rope_kernel(const RopeArgs a) {
    pdl_wait();
    rope_block<kFp16, kHalf, kHeads>(a, blockIdx.x, blockIdx.y);
}

// ------------------------------------------------------------ cache writes

struct AppendArgs {
    const uint16_t* k;
    const uint16_t* v;
    int64_t k_ts, k_hs, v_ts, v_hs;
    int64_t tokens;
    int dim;
    int rot;               // rotated dims (0: none)
    const int32_t* positions;
    const float* table;
    int64_t table_positions;
    const int32_t* slots;
    dg_kv_cache cache;
    int page_shift;
    int row_blocks;        // blocks that share out a token's rows
    int tokens_at_once;    // tokens whose rows one pass of a block holds
    uint32_t* status;
};

// max(|a|, |b|, |c|), NaN if any is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// (a, b) * m, both products in one instruction.
__device__ __forceinline__ void mul2(float a, float b, float m, float* x, float* y) {
    asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %4};\n\t"
        "mul.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "=f"(*x), "=f"(*y) : "f"(a), "f"(b), "f"(m));
}

__device__ __forceinline__ uint2 codes8(const float (&q)[8]) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = f32x2_to_e4m3x2(q[2 * i], q[2 * i + 1]);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Out of line: taken once in hundreds of rows.
__device__ __noinline__ uint2 divide8(float x0, float x1, float x2, float x3, float x4, float x5,
                                      float x6, float x7, float scale) {
    const float q[8] = {__fdiv_rn(x0, scale), __fdiv_rn(x1, scale), __fdiv_rn(x2, scale),
                        __fdiv_rn(x3, scale), __fdiv_rn(x4, scale), __fdiv_rn(x5, scale),
                        __fdiv_rn(x6, scale), __fdiv_rn(x7, scale)};
    return codes8(q);
}

// E4M3(fl32(x / scale)) of 8 elements, scale finite and at least 2^-60, |x|
// at most about 448 scale.  An IEEE division per element would cost more
// than the memory time of the whole row, so the quotient is enclosed: with
// r the approximate reciprocal (off by at most 2^-23 of it), x * r (1 -
// 2^-21) and x * r (1 + 2^-21) lie on either side of fl32(x / scale): the
// two products and the quotient itself round by at most 2^-24 each
// (quotients below 2^-100 have code 0 throughout).  Rounding to E4M3
// is monotone, so where both ends have one code that is the quotient's; the
// divisions are done for the few elements near the middle of two codes.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float scale) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale));
    const float below = r * (1.0f - 0x1p-21f), above = r * (1.0f + 0x1p-21f);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) mul2(x[i], x[i + 1], below, &q[i], &q[i + 1]);
    const uint2 lo = codes8(q);
#pragma unroll
    for (int i = 0; i < 8; i += 2) mul2(x[i], x[i + 1], above, &q[i], &q[i + 1]);
    const uint2 hi = codes8(q);
    if (lo.x == hi.x && lo.y == hi.y) return lo;
    return divide8(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], scale);
}

// A group of kLanes lanes owns one row (a key or value head) and walks over
// kTokens tokens, 16 dims a lane: row and dims are fixed, so a token costs
// little more than its loads, and what a row costs whatever its width (its
// place, maximum and scale) is spread over few lanes.  A rotated lane of the
// half layout owns 8 dims and the 8 they are paired with, so that nothing is
// read twice.
template <bool kFp16, bool kHalf, int kLanes, int kTokens>
__device__ __forceinline__ void append_block(const AppendArgs& a, int block) {
    constexpr int kGroups = 256 / kLanes;
    const int l = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int kv_heads = a.cache.kv_heads, rows = 2 * kv_heads;
    const int token_block = block / a.row_blocks;
    const int row_block = block - token_block * a.row_blocks;
    const int r = row_block * kGroups + (a.tokens_at_once > 1 ? group % rows : group);
    const int local = a.tokens_at_once > 1 ? group / rows : 0;
    const int64_t t0 = static_cast<int64_t>(token_block) * (a.tokens_at_once * kTokens) + local;
    const bool is_k = r < kv_heads;
    const bool live = 16 * l < a.dim && r < rows && local < a.tokens_at_once;
    const bool turn = live && is_k && 16 * l < a.rot;
    const bool apart = kHalf && turn;
    const int d = apart ? 8 * l : 16 * l;                    // this lane's first 8 dims
    const int d2 = apart ? a.rot / 2 + 8 * l : 16 * l + 8;   // and its others
    const int h = is_k ? r : r - kv_heads;
    const uint16_t* src = is_k ? a.k + h * a.k_hs : a.v + h * a.v_hs;
    const int64_t ts = is_k ? a.k_ts : a.v_ts;
    const int64_t nslots = a.cache.pages << a.page_shift;

    uint4 own[kTokens][2];
    int slot[kTokens];
    int64_t pos[kTokens];
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
        const int64_t t = t0 + j * a.tokens_at_once;
        own[j][0] = own[j][1] = make_uint4(0, 0, 0, 0);
        slot[j] = -1;
        pos[j] = 0;
        if (t < a.tokens) {
            slot[j] = a.slots[t];
            if (a.rot > 0) pos[j] = a.positions[t];
            if (live) {
                own[j][0] = *reinterpret_cast<const uint4*>(src + t * ts + d);
                own[j][1] = *reinterpret_cast<const uint4*>(src + t * ts + d2);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
        const bool bad = slot[j] >= nslots || pos[j] < 0 || (a.rot > 0 && pos[j] >= a.table_positions);
        if (bad && threadIdx.x % kLanes == 0) atomicOr(a.status, kStatusBadArgument);
        if (bad) slot[j] = -1;
        float x[2][8];
        unpack8<kFp16>(own[j][0], x[0]);
        unpack8<kFp16>(own[j][1], x[1]);
        if (turn && slot[j] >= 0) {
            const float* row = a.table + pos[j] * a.rot;
            if constexpr (kHalf) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float4 f = __ldg(reinterpret_cast<const float4*>(row + 2 * (d + i)));
                    const float p0 = x[0][i], q0 = x[1][i], p1 = x[0][i + 1], q1 = x[1][i + 1];
                    x[0][i] = p0 * f.x - q0 * f.y;
                    x[1][i] = q0 * f.x + p0 * f.y;
                    x[0][i + 1] = p1 * f.z - q1 * f.w;
                    x[1][i + 1] = q1 * f.z + p1 * f.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 f = __ldg(reinterpret_cast<const float4*>(row + d + i));
                    float* y = &x[i >> 3][i & 7];
                    const float y0 = y[0], y2 = y[2];
                    y[0] = y0 * f.x - y[1] * f.y;
                    y[1] = y[1] * f.x + y0 * f.y;
                    y[2] = y2 * f.z - y[3] * f.w;
                    y[3] = y[3] * f.z + y2 * f.w;
                }
            }
        }
        // The rotated key goes to its scale and code in FP32, not through a
        // 16-bit rounding.
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i += 2) top = max3_abs(top, x[i >> 3][i & 7], x[i >> 3][(i & 7) + 1]);
#pragma unroll
        for (int w = kLanes / 2; w > 0; w >>= 1) {
            const float other = __shfl_xor_sync(0xFFFFFFFFu, top, w);
            top = max3_abs(top, other, other);
        }
        if (!live || slot[j] < 0) continue;
        const int64_t page = slot[j] >> a.page_shift;
        const int64_t row = ((page * kv_heads + h) << a.page_shift) + (slot[j] & ((1 << a.page_shift) - 1));
        const bool finite = top <= 3.4028235e38f;   // false for NaN
        const float scale = finite ? fmaxf(__fdiv_rn(top, 448.0f), kKvMinScale) : __int_as_float(0x7FC00000);
        const uint2 lo = finite ? quantise8(x[0], scale) : make_uint2(0, 0);
        const uint2 hi = finite ? quantise8(x[1], scale) : make_uint2(0, 0);
        uint8_t* dst = (is_k ? a.cache.k : a.cache.v) + row * a.dim;
        if (apart) {
            *reinterpret_cast<uint2*>(dst + d) = lo;
            *reinterpret_cast<uint2*>(dst + d2) = hi;
        } else {
            *reinterpret_cast<uint4*>(dst + d) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
        if (l == 0) (is_k ? a.cache.k_scale : a.cache.v_scale)[row] = scale;
    }
}

constexpr int kAppendTokens = 2;   // of a lane group, in large calls

// Every kv_every-th block writes the cache (many instructions a load), the
// others turn the queries (bound by HBM): dealt out among one another they
// share the SMs.  16001 tokens of 32 + 8 + 8 heads of 128, half of each
// turned, interleaved: 60.5 us, 6.0 TB/s, 0.89 of a copy; whole heads in the
// half layout 61.9; 32 + 32 + 32 heads 146 in FP16 and 153 in BF16 (0.68 and
// 0.64): two thirds of those are cache rows, whose warps wait for their loads
// with 57% of the issue slots used and 28 warps an SM, so neither limit is
// reached.  With 8 dims a lane and 4 tokens in flight 72, 80 and 220.  Four
// blocks an SM, by the registers of the four query heads a thread holds; with
// two heads and six blocks 65 us.
template <bool kFp16, bool kHalf, int kLanes, bool kMany>
__global__ void __launch_bounds__(256, kMany ? 4 : 6)
kv_append_kernel(const AppendArgs a, const RopeArgs q, int kv_blocks, int kv_every) {
    pdl_wait();
    const int round = static_cast<int>(blockIdx.x) / kv_every;
    if (round < kv_blocks && static_cast<int>(blockIdx.x) - round * kv_every == kv_every - 1)
        append_block<kFp16, kHalf, kLanes, kMany ? kAppendTokens : 1>(a, round);
    else {
        const int b = static_cast<int>(blockIdx.x) - min(round, kv_blocks);
        const int token_block = q.head_blocks == 1 ? b : b / q.head_blocks;
        rope_block<kFp16, kHalf, kMany ? 4 : 1>(q, token_block, b - token_block * q.head_blocks);
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
    int chunks;            // head_dim / 8
    int items;             // chunks * kv_heads * tensors
    int item_blocks;       // blocks that share out a token's items
    int tokens_at_once;    // tokens whose items one pass of a block holds
    uint32_t* status;
};

// A thread owns 8 dims of one row (a warp's stores are whole lines) and walks
// over the tokens, kTokens at a time, the next ones' slots already on their
// way: code x scale in FP32, rounded once to the output type.  40001 tokens x
// 8 heads of 128, keys and values: 41.9 us (5.9 TB/s, 0.88 of a copy); two
// waves of blocks with half the walk 42.9, one pass a block 52.
template <bool kFp16, int kTokens>
__global__ void __launch_bounds__(256)
kv_read_kernel(const ReadArgs a) {
    const int lane_block = static_cast<int>(blockIdx.x) / a.item_blocks, steps = gridDim.x / a.item_blocks;
    const int item_block = static_cast<int>(blockIdx.x) - lane_block * a.item_blocks;
    const int local = a.tokens_at_once > 1 ? threadIdx.x / a.items : 0;
    const int item = item_block * 256 + static_cast<int>(threadIdx.x) - local * a.items;
    if (item >= a.items || local >= a.tokens_at_once) return;
    const int row = item / a.chunks, chunk = item - row * a.chunks;
    const int kv_heads = a.cache.kv_heads;
    const bool is_v = a.k == nullptr || row >= kv_heads;
    const int h = row >= kv_heads ? row - kv_heads : row;
    const uint8_t* codes = (is_v ? a.cache.v : a.cache.k) + 8 * chunk;
    const float* scales = is_v ? a.cache.v_scale : a.cache.k_scale;
    uint16_t* dst = (is_v ? a.v + h * a.v_hs : a.k + h * a.k_hs) + 8 * chunk;
    const int64_t ts = is_v ? a.v_ts : a.k_ts;
    const int64_t nslots = a.cache.pages << a.page_shift;
    const int in_page = (1 << a.page_shift) - 1;
    const int64_t step = static_cast<int64_t>(steps) * (a.tokens_at_once * kTokens);
    int64_t t = static_cast<int64_t>(lane_block) * (a.tokens_at_once * kTokens) + local;
    pdl_wait();
    int slot[kTokens];
    auto fetch = [&](int64_t from) {
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            const int64_t u = from + j * a.tokens_at_once;
            slot[j] = u < a.tokens ? a.slots[u] : -1;
        }
    };
    fetch(t);
    for (; t < a.tokens; t += step) {
        uint2 code[kTokens];
        float scale[kTokens];
        bool past[kTokens];
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            code[j] = make_uint2(0, 0);
            scale[j] = 0.0f;
            past[j] = slot[j] >= nslots;
            if (slot[j] >= 0 && !past[j]) {
                const int64_t r = ((static_cast<int64_t>(slot[j] >> a.page_shift) * kv_heads + h) << a.page_shift) +
                                  (slot[j] & in_page);
                code[j] = ld_once8(codes + r * (8 * a.chunks));
                scale[j] = __ldg(scales + r);
            }
        }
        fetch(t + step);
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            const int64_t u = t + j * a.tokens_at_once;
            if (u >= a.tokens) continue;
            if (past[j]) {
                if (chunk == 0) atomicOr(a.status, kStatusBadArgument);
                continue;
            }
            const uint32_t w[2] = {code[j].x, code[j].y};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 lo = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i])));
                const float2 hi = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> 16)));
                o[2 * i] = pack2<kFp16>(lo.x * scale[j], lo.y * scale[j]);
                o[2 * i + 1] = pack2<kFp16>(hi.x * scale[j], hi.y * scale[j]);
            }
            *reinterpret_cast<uint4*>(dst + u * ts) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

template <bool kFp16, bool kHalf>
cudaError_t rope_dispatch(const RopeArgs& a, int heads_per_thread, dim3 grid, cudaStream_t s) {
    return heads_per_thread == 4
               ? launch_kernel(rope_kernel<kFp16, kHalf, 4>, grid, dim3(256), 0, s, a)
               : launch_kernel(rope_kernel<kFp16, kHalf, 1>, grid, dim3(256), 0, s, a);
}

template <bool kFp16, bool kHalf, bool kMany>
cudaError_t append_dispatch(const AppendArgs& a, const RopeArgs& q, int64_t q_blocks, int64_t kv_blocks,
                            cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(q_blocks + kv_blocks)), block(256);
    const int kv = static_cast<int>(kv_blocks), every = static_cast<int>((q_blocks + kv_blocks) / kv_blocks);
    if (a.dim <= 64) return launch_kernel(kv_append_kernel<kFp16, kHalf, 4, kMany>, grid, block, 0, s, a, q, kv, every);
    if (a.dim <= 128) return launch_kernel(kv_append_kernel<kFp16, kHalf, 8, kMany>, grid, block, 0, s, a, q, kv, every);
    return launch_kernel(kv_append_kernel<kFp16, kHalf, 16, kMany>, grid, block, 0, s, a, q, kv, every);
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

namespace {

// The arguments of a rotation but for the split over blocks.
RopeArgs rope_args(const dg_heads& x, const dg_heads& out, int64_t tokens, int heads, int head_dim,
                   const int32_t* positions, const dg_rotary* rot, bool inverse, uint32_t* status) {
    RopeArgs a{};
    a.x = static_cast<const uint16_t*>(x.data);
    a.out = static_cast<uint16_t*>(out.data);
    a.x_ts = x.token_stride;
    a.x_hs = x.head_stride;
    a.o_ts = out.token_stride;
    a.o_hs = out.head_stride;
    a.tokens = tokens;
    a.heads = heads;
    if (rot != nullptr) {
        a.rot8 = rot->rotary_dim / 8;
        a.positions = positions;
        a.table = reinterpret_cast<const float4*>(rot->table);
        a.table_positions = rot->positions;
    }
    const bool half = rot == nullptr || rot->layout == DG_ROPE_HALF;
    a.items = head_dim / 16;
    a.sign = inverse ? -1.0f : 1.0f;
    a.status = status;
    return a;
}

// Splits a rotation over blocks with `per_thread` heads a thread; returns
// their number.
int64_t rope_split(RopeArgs* a, int per_thread) {
    a->head_steps = (a->heads + per_thread - 1) / per_thread;
    a->sets = std::min(a->head_steps, 256 / a->items);
    a->head_blocks = (a->head_steps + a->sets - 1) / a->sets;
    a->threads_per_token = a->items * a->sets;
    a->tokens_per_block = 256 / a->threads_per_token;
    return (a->tokens + a->tokens_per_block - 1) / a->tokens_per_block * a->head_blocks;
}

}  // namespace

cudaError_t launch_rope(const dg_heads& x, const dg_heads& out, int64_t tokens, int heads,
                        int head_dim, const int32_t* positions, const dg_rotary& rot, bool inverse,
                        bool fp16, int sm_count, uint32_t* status, cudaStream_t s) {
    RopeArgs a = rope_args(x, out, tokens, heads, head_dim, positions, &rot, inverse, status);
    const bool half = rot.layout == DG_ROPE_HALF;
    // Four heads a thread once that still leaves every SM two blocks.
    const int per_thread = tokens * heads * a.items < static_cast<int64_t>(4) * 2 * sm_count * 256 ? 1 : 4;
    const int64_t blocks = rope_split(&a, per_thread) / a.head_blocks;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(a.head_blocks));
    if (fp16)
        return half ? rope_dispatch<true, true>(a, per_thread, grid, s)
                    : rope_dispatch<true, false>(a, per_thread, grid, s);
    return half ? rope_dispatch<false, true>(a, per_thread, grid, s)
                : rope_dispatch<false, false>(a, per_thread, grid, s);
}

cudaError_t launch_kv_append(const dg_heads* q, const dg_heads* q_out, int q_heads,
                             const dg_heads& k, const dg_heads& v, int64_t tokens,
                             const int32_t* positions, const dg_rotary* rot, const int32_t* slots,
                             const dg_kv_cache& cache, bool fp16, int sm_count, uint32_t* status,
                             cudaStream_t s) {
    AppendArgs a{};
    a.k = static_cast<const uint16_t*>(k.data);
    a.k_ts = k.token_stride;
    a.k_hs = k.head_stride;
    a.v = static_cast<const uint16_t*>(v.data);
    a.v_ts = v.token_stride;
    a.v_hs = v.head_stride;
    a.tokens = tokens;
    a.dim = cache.head_dim;
    if (rot != nullptr) {
        a.rot = rot->rotary_dim;
        a.table = rot->table;
        a.table_positions = rot->positions;
        a.positions = positions;
    }
    a.slots = slots;
    a.cache = cache;
    a.page_shift = shift_of(cache.page_size);
    a.status = status;
    const bool half = rot == nullptr || rot->layout == DG_ROPE_HALF;
    const int lanes = a.dim <= 64 ? 4 : a.dim <= 128 ? 8 : 16;
    const int groups = 256 / lanes, rows = 2 * cache.kv_heads;
    a.row_blocks = (rows + groups - 1) / groups;
    a.tokens_at_once = a.row_blocks == 1 ? groups / rows : 1;
    // Two tokens a lane group (and four query heads a thread) once that still
    // leaves every SM four blocks of cache rows.
    const int64_t passes = (tokens + a.tokens_at_once - 1) / a.tokens_at_once;
    const bool few = passes * a.row_blocks < static_cast<int64_t>(4) * 2 * sm_count;
    const int per_block = a.tokens_at_once * (few ? 1 : kAppendTokens);
    const int64_t kv_blocks = (tokens + per_block - 1) / per_block * a.row_blocks;
    RopeArgs qa{};
    int64_t q_blocks = 0;
    if (q != nullptr) {
        qa = rope_args(*q, *q_out, tokens, q_heads, cache.head_dim, positions, rot, false, status);
        qa.slots = slots;
        qa.nslots = cache.pages * cache.page_size;
        q_blocks = rope_split(&qa, few ? 1 : 4);
    }
    if (q_blocks + kv_blocks > INT_MAX) return cudaErrorInvalidValue;
    if (fp16) {
        if (half)
            return few ? append_dispatch<true, true, false>(a, qa, q_blocks, kv_blocks, s)
                       : append_dispatch<true, true, true>(a, qa, q_blocks, kv_blocks, s);
        return few ? append_dispatch<true, false, false>(a, qa, q_blocks, kv_blocks, s)
                   : append_dispatch<true, false, true>(a, qa, q_blocks, kv_blocks, s);
    }
    if (half)
        return few ? append_dispatch<false, true, false>(a, qa, q_blocks, kv_blocks, s)
                   : append_dispatch<false, true, true>(a, qa, q_blocks, kv_blocks, s);
    return few ? append_dispatch<false, false, false>(a, qa, q_blocks, kv_blocks, s)
               : append_dispatch<false, false, true>(a, qa, q_blocks, kv_blocks, s);
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
    a.chunks = cache.head_dim / 8;
    a.items = a.chunks * cache.kv_heads * ((k != nullptr) + (v != nullptr));
    a.item_blocks = (a.items + 255) / 256;
    a.tokens_at_once = a.item_blocks == 1 ? 256 / a.items : 1;
    a.status = status;
    // Four tokens a thread and step once that still leaves every SM its
    // resident blocks (4), which then stay and walk over the tokens.
    const int64_t passes = (tokens + a.tokens_at_once - 1) / a.tokens_at_once;
    const int64_t resident = static_cast<int64_t>(4) * sm_count;
    const bool few = passes * a.item_blocks < 4 * resident;
    const int64_t want = (passes + (few ? 1 : 4) - 1) / (few ? 1 : 4);
    const int64_t walk = few ? want : std::max<int64_t>(1, std::min(want, resident / a.item_blocks));
    if (walk * a.item_blocks > INT_MAX) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(walk * a.item_blocks));
    if (fp16)
        return few ? launch_kernel(kv_read_kernel<true, 1>, grid, dim3(256), 0, s, a)
                   : launch_kernel(kv_read_kernel<true, 4>, grid, dim3(256), 0, s, a);
    return few ? launch_kernel(kv_read_kernel<false, 1>, grid, dim3(256), 0, s, a)
               : launch_kernel(kv_read_kernel<false, 4>, grid, dim3(256), 0, s, a);
}

}  // namespace dg
