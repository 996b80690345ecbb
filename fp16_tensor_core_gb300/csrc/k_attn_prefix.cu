// k_attn_prefix.cu -- attention of many query rows over a prefix that a
// whole batch shares, on tcgen05.
//
// The formulas are those of k_attn_decode.cu.  Where dozens of rows share a
// key head the work is no longer reading the cache but its 4 flop per cached
// element and row, so 128 rows at a time meet 128 tokens on the tensor cores:
//   S = Q Kc^T   (FP16 operands from shared memory, FP32 in tensor memory)
//   W = exp(scale sk S + ln sv - m), to FP16, back into tensor memory
//   O += W Vc    (W from tensor memory, Vc from shared memory)
// A CTA holds one 128-row tile of one key head and walks over its share of
// the prefix.  Roles: four warps take the codes from the cache and write them
// as FP16 (exact) into swizzled shared memory, keys and values in two stages
// each; one thread issues the MMAs; four warps turn scores into weights.  S
// has two buffers (a tile's weights take the place of its scores), so the
// next tile's scores are formed while this one's weights are.
//
// A warp of the softmax reads its 32 rows in the MMA fragment shape (a thread
// holds 2 of 8 columns of 4 rows) instead of a row per thread: the per-token
// factors it needs are then a quarter, and packed pairs of columns feed the
// two-wide FP32 instructions.  The reference m of a row follows its maximum
// only when that has grown by 2^8: O is rescaled rarely, weights stay below
// 2^8, where FP16 has the same 11 bits.
//
// V is stored token-major, as in the cache: the second product takes it as an
// operand whose N side is contiguous (bit 16 of the instruction descriptor).
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_common.cuh"
#include "dg_internal.h"
#include "dg_ptx.cuh"

namespace dg {
namespace {

constexpr int kTileTokens = 128;
constexpr int kTileRows = 128;
constexpr int kThreads = 384;   // warpgroups: softmax, converters, MMA (one thread of it)
constexpr float kGrowth = 8.0f; // log2 of how far weights may pass 1

__device__ __forceinline__ void tmem_load_frag16(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, "
        "%33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, "
        "%49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, "
        "[%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]),
          "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
          "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
          "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]),
          "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]),
          "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_load_frag8(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
        "[%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_store_frag8(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
          "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
          "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
          "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
          "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_store_pairs16(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
          "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
          "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
          "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
          "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem], FP16 operands.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of an operand whose M or N side is contiguous (64 elements of
// 16 bits a 128-byte row, one row per k, 128-byte swizzle): 64-element
// columns `column_bytes` apart (leading offset), groups of 8 k 1024 apart.
__device__ __forceinline__ uint64_t sdesc_mn_major_sw128(uint32_t smem_byte_addr, uint32_t column_bytes) {
    uint64_t d = sdesc_k_major_sw128(smem_byte_addr);
    d &= ~(static_cast<uint64_t>(0x3FFF) << 16);
    return d | static_cast<uint64_t>(column_bytes >> 4) << 16;
}

// Two FP32 lanes at once.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack(f32x2 v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

struct PrefixArgs {
    const uint16_t* q;
    int64_t q_ts, q_hs;
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    int64_t pages;
    int kv_heads, page_shift;
    const int32_t* page_list;
    int len;               // tokens of the prefix
    int rows;              // query rows per key head
    int group, q_heads;
    int row_tiles, splits;
    float scale_log2;
    float* slots;          // splits > 1: states of each CTA's 128 rows
    float* states;         // per (token, query head)
    uint32_t* status;
    uint64_t timeout_ns;
};

template <int D>
struct PrefixShape {
    static constexpr int kHalves = D / 64;                       // 64-dim columns of an operand
    static constexpr int kColumnBytes = kTileTokens * 128;       // 16 KB
    static constexpr int kOperandBytes = kHalves * kColumnBytes; // Q, or one stage of K or V
    static constexpr int kState = D + 4;
    static constexpr int kOCol = 256;                            // tensor memory: S0, S1, O
    static constexpr int kKAt = kOperandBytes;
    static constexpr int kVAt = kKAt + 2 * kOperandBytes;
    static constexpr int kFactorsAt = kVAt + 2 * kOperandBytes;  // [2][3][128] per-token factors
    static constexpr int kRowsAt = kFactorsAt + 2 * 3 * 128 * 4; // [2][128] cache rows
    static constexpr int kQScaleAt = kRowsAt + 2 * 128 * 8;
    static constexpr int kBarsAt = kQScaleAt + 128 * 4;
    static constexpr int kSmem = kBarsAt + 256 + 1024;           // and alignment
};

// 16 codes of a token's row as two 16-byte chunks of FP16 in the swizzled
// operand; lanes of the upper half store their second chunk first, which
// keeps a quarter warp's stores in different banks.
template <int D>
__device__ __forceinline__ void store_chunk16(uint8_t* operand, int token, int chunk, uint4 codes) {
    uint32_t h[8];
    codes_to_halves(codes.x, &h[0], &h[1]);
    codes_to_halves(codes.y, &h[2], &h[3]);
    codes_to_halves(codes.z, &h[4], &h[5]);
    codes_to_halves(codes.w, &h[6], &h[7]);
    const int c0 = 2 * chunk;
    uint8_t* row = operand + (c0 >> 3) * PrefixShape<D>::kColumnBytes + token * 128;
    const uint32_t a0 = smem_addr(row + (((c0 & 7) ^ (token & 7)) * 16));
    const uint32_t a1 = smem_addr(row + ((((c0 & 7) + 1) ^ (token & 7)) * 16));
    if (D == 128 && chunk >= 4) {
        st_shared_v4(a1, h[4], h[5], h[6], h[7]);
        st_shared_v4(a0, h[0], h[1], h[2], h[3]);
    } else {
        st_shared_v4(a0, h[0], h[1], h[2], h[3]);
        st_shared_v4(a1, h[4], h[5], h[6], h[7]);
    }
}

template <int D, bool kFp16>
__global__ void __launch_bounds__(kThreads, 1) attn_prefix_kernel(const PrefixArgs a) {
    using S = PrefixShape<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sq = smem;
    float* factors = reinterpret_cast<float*>(smem + S::kFactorsAt);
    int64_t* cache_rows = reinterpret_cast<int64_t*>(smem + S::kRowsAt);
    float* qscale = reinterpret_cast<float*>(smem + S::kQScaleAt);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBarsAt);
    uint64_t* q_full = bars;          // 128 arrivals
    uint64_t* k_full = bars + 1;      // [2], 128
    uint64_t* v_full = bars + 3;      // [2], 128
    uint64_t* s_full = bars + 5;      // [2], commit
    uint64_t* w_full = bars + 7;      // [2], 128: weights in place, scores and factors read
    uint64_t* o_done = bars + 9;      // [2], commit
    uint64_t* drain = bars + 11;      // commit
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 12);
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 128);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&k_full[b], 128);
            mbar_init(&v_full[b], 128);
            mbar_init(&s_full[b], 1);
            mbar_init(&w_full[b], 128);
            mbar_init(&o_done[b], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc<512>(tmem_slot);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl ctl{abort_flag, a.status, a.timeout_ns};

    // this CTA: row tile, share of the prefix, key head
    const int rt = static_cast<int>(blockIdx.x) % a.row_tiles;
    const int share = static_cast<int>(blockIdx.x) / a.row_tiles;
    const int split = share % a.splits, head = share / a.splits;
    const int all_tiles = (a.len + kTileTokens - 1) / kTileTokens;
    const int tile0 = static_cast<int>(static_cast<int64_t>(all_tiles) * split / a.splits);
    const int tiles = static_cast<int>(static_cast<int64_t>(all_tiles) * (split + 1) / a.splits) - tile0;
    pdl_wait();

    // Registers: 168 a thread at launch; the softmax warps hold 128 scores
    // each and take 72 more of the MMA warpgroup's (240 + 168 + 96 = 3 * 168).
    if (warp < 4) {
        // -------------------------------------------------- queries, softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
        const int g = lane >> 2, c = lane & 3;
        {   // thread i takes row i of the tile, scaled by a power of two (BF16)
            const int i = threadIdx.x, r = rt * kTileRows + i;
            uint4 w[D / 8];
            float factor = a.scale_log2;
            if (r < a.rows) {
                const int token = r / a.group;
                const uint16_t* src = a.q + static_cast<int64_t>(token) * a.q_ts +
                                      static_cast<int64_t>(head * a.group + r - token * a.group) * a.q_hs;
#pragma unroll
                for (int k = 0; k < D / 8; ++k) w[k] = reinterpret_cast<const uint4*>(src)[k];
            } else {
#pragma unroll
                for (int k = 0; k < D / 8; ++k) w[k] = make_uint4(0, 0, 0, 0);
            }
            float mul = 1.0f;
            if constexpr (!kFp16) {
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < D / 8; ++k) top = max(top, top_abs_bf16(w[k]));
                const PowerOfTwo p = power_below(top);
                mul = p.inverse;
                factor *= p.value;
            }
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                if constexpr (!kFp16) w[k] = bf16_to_half8(w[k], mul);
                st_shared_v4(smem_addr(sq + (k >> 3) * S::kColumnBytes + i * 128 + (((k & 7) ^ (i & 7)) * 16)),
                             w[k].x, w[k].y, w[k].z, w[k].w);
            }
            qscale[i] = factor;
            fence_proxy_async_smem();
            mbar_arrive(q_full);
            named_bar_sync(1, 128);
        }
        // row 16 h + 8 i + g of the warp's 32: index 2 h + i
        float m[4], qs[4];
        f32x2 l[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            m[x] = -INFINITY;
            l[x] = 0ull;
            qs[x] = qscale[32 * warp + 16 * (x >> 1) + 8 * (x & 1) + g];
        }
        const uint32_t quad = tmem + (static_cast<uint32_t>(32 * warp) << 16);
        bool ok = true;
        for (int j = 0; j < tiles; ++j) {
            const int b = j & 1;
            const uint32_t parity = (j >> 1) & 1;
            // the keys' barrier also hands over the per-token factors
            ok = wait_bounded(&k_full[b], parity, ctl) && wait_bounded(&s_full[b], parity, ctl);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after_sync();
            uint32_t s[2][64];
            tmem_load_frag16(quad + 128 * b, s[0]);
            tmem_load_frag16(quad + (16u << 16) + 128 * b, s[1]);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 64; ++k) asm volatile("" : "+r"(s[h][k]));
            const float* f = factors + b * 3 * 128 + 2 * c;
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                const f32x2 sk = *reinterpret_cast<const f32x2*>(f + 8 * n);
                const f32x2 lg = *reinterpret_cast<const f32x2*>(f + 128 + 8 * n);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t* p = &s[x >> 1][4 * n + 2 * (x & 1)];
                    const f32x2 y = fma2(mul2(pack(__uint_as_float(p[0]), __uint_as_float(p[1])), sk),
                                         pack(qs[x], qs[x]), lg);
                    const float2 v = unpack(y);
                    top[x] = fmaxf(top[x], fmaxf(v.x, v.y));
                    p[0] = __float_as_uint(v.x);
                    p[1] = __float_as_uint(v.y);
                }
            }
            bool grew = false;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], 1));
                top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], 2));
                grew |= top[x] > m[x] + kGrowth;
            }
            if (__any_sync(0xFFFFFFFFu, grew)) {
                float by[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const bool move = top[x] > m[x] + kGrowth;
                    by[x] = move ? ex2(m[x] - top[x]) : 1.0f;
                    if (move) m[x] = top[x];
                    l[x] = mul2(l[x], pack(by[x], by[x]));
                }
                if (j > 0) {
                    // O as the previous tile left it
                    ok = wait_bounded(&o_done[b ^ 1], ((j - 1) >> 1) & 1, ctl);
                    if (!__all_sync(0xFFFFFFFFu, ok)) break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll 1
                        for (int part = 0; part < D / 64; ++part) {
                            uint32_t o[32];
                            const uint32_t at = quad + (static_cast<uint32_t>(16 * h) << 16) + S::kOCol + 64 * part;
                            tmem_load_frag8(at, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                asm volatile("" : "+r"(o[k]));
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * by[2 * h + ((k >> 1) & 1)]);
                            }
                            tmem_store_frag8(at, o);
                        }
                    }
                    tmem_wait_st();
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[32];
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                    const f32x2 rs = *reinterpret_cast<const f32x2*>(f + 256 + 8 * n);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int x = 2 * h + i;
                        const float base = m[x] == -INFINITY ? 0.0f : -m[x];
                        const uint32_t* p = &s[h][4 * n + 2 * i];
                        const float2 y = unpack(add2(pack(__uint_as_float(p[0]), __uint_as_float(p[1])),
                                                     pack(base, base)));
                        const float e0 = ex2(y.x), e1 = ex2(y.y);
                        l[x] = fma2(pack(e0, e1), rs, l[x]);
                        w[2 * n + i] = f32x2_to_f16x2(e0, e1);
                    }
                }
                tmem_store_pairs16(quad + (static_cast<uint32_t>(16 * h) << 16) + 128 * b, w);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            mbar_arrive(&w_full[b]);
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok) ok = __all_sync(0xFFFFFFFFu, wait_bounded(&o_done[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1, ctl));
        if (ok) {
            tc_fence_after_sync();
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                float* dst[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int x = 2 * h + i;
                    const float2 part = unpack(l[x]);
                    float sum = part.x + part.y;
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                    const int in_tile = 32 * warp + 16 * h + 8 * i + g, r = rt * kTileRows + in_tile;
                    dst[i] = nullptr;
                    if (r >= a.rows) continue;
                    if (a.splits > 1) {
                        dst[i] = a.slots + (static_cast<int64_t>(blockIdx.x) * kTileRows + in_tile) * S::kState;
                    } else {
                        const int token = r / a.group;
                        const int64_t row = static_cast<int64_t>(token) * a.q_heads + head * a.group + r - token * a.group;
                        dst[i] = a.states + row * S::kState;
                    }
                    if (c == 0) *reinterpret_cast<float2*>(dst[i]) = make_float2(m[x], sum);
                }
#pragma unroll 1
                for (int part = 0; part < D / 64; ++part) {
                    uint32_t o[32];
                    tmem_load_frag8(quad + (static_cast<uint32_t>(16 * h) << 16) + S::kOCol + 64 * part, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k) asm volatile("" : "+r"(o[k]));
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (dst[i] != nullptr)
                                *reinterpret_cast<float2*>(dst[i] + 4 + 64 * part + 8 * n + 2 * c) =
                                    make_float2(__uint_as_float(o[4 * n + 2 * i]),
                                                __uint_as_float(o[4 * n + 2 * i + 1]));
                }
            }
        }
    } else if (warp < 8) {
        // -------------------------------------------------- codes to operands
        const int i = static_cast<int>(threadIdx.x) - 128;
        constexpr int kPerRow = D / 16, kPasses = kPerRow;   // 128 / kPerRow tokens a pass
        const int chunk = i % kPerRow, token_in = i / kPerRow;
        constexpr int kStep = 128 / kPerRow;
        const int in_page = (1 << a.page_shift) - 1;
        // cache row of token i of tile j (-1: none), from its page
        auto find_row = [&](int j) -> int64_t {
            const int t = (tile0 + j) * kTileTokens + i;
            if (j >= tiles || t >= a.len) return -1;
            const int p = a.page_list[t >> a.page_shift];
            if (p < 0 || p >= a.pages) {
                atomicOr(a.status, kStatusBadArgument);
                return -1;
            }
            return ((static_cast<int64_t>(p) * a.kv_heads + head) << a.page_shift) + (t & in_page);
        };
        auto load = [&](const uint8_t* codes, const int64_t* rows, uint4 (&x)[kPasses]) {
#pragma unroll
            for (int s = 0; s < kPasses; ++s) {
                const int64_t r = rows[token_in + s * kStep];
                x[s] = make_uint4(0, 0, 0, 0);
                if (r >= 0) x[s] = __ldg(reinterpret_cast<const uint4*>(codes + r * D + chunk * 16));
            }
        };
        auto load_scales = [&](int64_t r, float* sk, float* sv) {
            *sk = 0.0f;
            *sv = -1.0f;   // no token
            if (r >= 0) {
                *sk = __ldg(a.k_scale + r);
                *sv = __ldg(a.v_scale + r);
            }
        };
        uint4 kc[kPasses], vc[kPasses];
        float sk, sv;
        int64_t mine = find_row(0);
        cache_rows[i] = mine;
        load_scales(mine, &sk, &sv);
        int64_t next = find_row(1);
        cache_rows[128 + i] = next;
        named_bar_sync(2, 128);
        load(a.k, cache_rows, kc);
        load(a.v, cache_rows, vc);
        named_bar_sync(2, 128);   // before rows are replaced
        bool ok = true;
        for (int j = 0; j < tiles && ok; ++j) {
            const int b = j & 1;
            const int64_t after = find_row(j + 2);   // its page is on its way meanwhile
            // scores and factors of tile j - 2 are read
            if (j >= 2) ok = __all_sync(0xFFFFFFFFu, wait_bounded(&w_full[b], ((j - 2) >> 1) & 1, ctl));
            const int64_t* rows_next = cache_rows + (b ^ 1) * 128;
            if (ok) {
                uint8_t* keys = smem + S::kKAt + b * S::kOperandBytes;
#pragma unroll
                for (int s = 0; s < kPasses; ++s) store_chunk16<D>(keys, token_in + s * kStep, chunk, kc[s]);
                float* f = factors + b * 3 * 128;
                const bool none = sv == -1.0f;
                const float safe = sv < 0x1p-100f ? 0x1p-100f : sv;
                f[i] = sk;
                f[128 + i] = none ? -INFINITY : __log2f(safe);
                f[256 + i] = none ? 0.0f : rcp(safe);
                fence_proxy_async_smem();
                mbar_arrive(&k_full[b]);
                if (j + 1 < tiles) {
                    load(a.k, rows_next, kc);
                    load_scales(next, &sk, &sv);
                }
                // the values of tile j - 2 are read
                if (j >= 2) ok = __all_sync(0xFFFFFFFFu, wait_bounded(&o_done[b], ((j - 2) >> 1) & 1, ctl));
            }
            if (ok) {
                uint8_t* values = smem + S::kVAt + b * S::kOperandBytes;
#pragma unroll
                for (int s = 0; s < kPasses; ++s) store_chunk16<D>(values, token_in + s * kStep, chunk, vc[s]);
                fence_proxy_async_smem();
                mbar_arrive(&v_full[b]);
                if (j + 1 < tiles) load(a.v, rows_next, vc);
            }
            // rows of tile j (whose loads were issued an iteration ago) make
            // room for those of tile j + 2; after a wait that ran out the
            // four warps leave together
            next = after;
            cache_rows[b * 128 + i] = after;
            ok = named_bar_and(2, 128, ok);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == 8 && lane == 0) {
            // -------------------------------------------------- MMA issue
            constexpr uint32_t kScoreDesc = idesc_f32acc(kTileRows, kTileTokens, 0, 0);
            constexpr uint32_t kValueDesc = idesc_f32acc(kTileRows, D, 0, 0) | (1u << 16);
            auto scores = [&](int j) {
                const uint32_t k0 = smem_addr(smem + S::kKAt + (j & 1) * S::kOperandBytes), q0 = smem_addr(sq);
#pragma unroll
                for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        mma_f16(tmem + 128 * (j & 1), sdesc_k_major_sw128(q0 + h * S::kColumnBytes + 32 * x),
                                sdesc_k_major_sw128(k0 + h * S::kColumnBytes + 32 * x), kScoreDesc,
                                h > 0 || x > 0);
                mma_commit(&s_full[j & 1]);
            };
            bool ok = wait_bounded(q_full, 0, ctl) && wait_bounded(&k_full[0], 0, ctl);
            bool issued = false;
            if (ok) {
                tc_fence_after_sync();
                issued = true;
                scores(0);
            }
            for (int j = 0; j < tiles && ok; ++j) {
                const int b = j & 1;
                if (j + 1 < tiles) {
                    // the buffer of tile j + 1's scores holds the weights of tile j - 1
                    ok = wait_bounded(&k_full[b ^ 1], ((j + 1) >> 1) & 1, ctl) &&
                         (j == 0 || wait_bounded(&o_done[b ^ 1], ((j - 1) >> 1) & 1, ctl));
                    if (!ok) break;
                    tc_fence_after_sync();
                    scores(j + 1);
                }
                ok = wait_bounded(&v_full[b], (j >> 1) & 1, ctl) && wait_bounded(&w_full[b], (j >> 1) & 1, ctl);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t v0 = smem_addr(smem + S::kVAt + b * S::kOperandBytes);
#pragma unroll
                for (int x = 0; x < kTileTokens / 16; ++x)
                    mma_f16_ts(tmem + S::kOCol, tmem + 128 * b + 8 * x,
                               sdesc_mn_major_sw128(v0 + x * 2048, S::kColumnBytes), kValueDesc, j > 0 || x > 0);
                mma_commit(&o_done[b]);
            }
            if (issued) {
                // Tensor memory is freed below: wait for every MMA issued.
                mma_commit(drain);
                wait_bounded(drain, 0, ctl, false);
            }
        }
    }
    tc_fence_before_sync();
    cta_sync_diverged();
    tc_fence_after_sync();
    if (warp == 8) {
        __syncwarp();
        tmem_dealloc<512>(tmem);
    }
}

// The states of a row's shares of the prefix, joined in token order: one warp
// a row.
template <int D>
__global__ void __launch_bounds__(128) attn_prefix_join_kernel(const PrefixArgs a) {
    constexpr int kState = D + 4;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int r = static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5), head = blockIdx.y;
    if (r >= a.rows) return;
    const int rt = r / kTileRows;
    const int64_t stride = static_cast<int64_t>(a.row_tiles) * kTileRows * kState;   // from split to split
    const float* first = a.slots + ((static_cast<int64_t>(head) * a.splits * a.row_tiles + rt) * kTileRows +
                                    (r - rt * kTileRows)) * kState;
    float m = -INFINITY, l = 0.0f;
    float4 x = make_float4(0, 0, 0, 0);
    join_states<D>(first, stride, a.splits, lane, &m, &l, &x);
    const int token = r / a.group;
    float* dst = a.states + (static_cast<int64_t>(token) * a.q_heads + head * a.group + r - token * a.group) * kState;
    if (lane == 0) *reinterpret_cast<float2*>(dst) = make_float2(m, l);
    if (4 * lane < D) *reinterpret_cast<float4*>(dst + 4 + 4 * lane) = x;
}

template <int D, bool kFp16>
cudaError_t run_prefix(const PrefixArgs& a, cudaStream_t s) {
    const cudaError_t set = cudaFuncSetAttribute(
        attn_prefix_kernel<D, kFp16>, cudaFuncAttributeMaxDynamicSharedMemorySize, PrefixShape<D>::kSmem);
    if (set != cudaSuccess) return set;
    const unsigned blocks = static_cast<unsigned>(a.kv_heads) * a.splits * a.row_tiles;
    const cudaError_t e = launch_kernel(attn_prefix_kernel<D, kFp16>, dim3(blocks), dim3(kThreads),
                                        PrefixShape<D>::kSmem, s, a);
    if (e != cudaSuccess || a.splits == 1) return e;
    return launch_kernel(attn_prefix_join_kernel<D>, dim3((a.rows + 3) / 4, a.kv_heads), dim3(128), 0, s, a);
}

}  // namespace

// Shares a key head's prefix is cut into: the CTAs fill one wave at most.
int attn_prefix_splits(int rows, int kv_heads, int64_t prefix_len, int sm_count) {
    const int64_t units = static_cast<int64_t>(kv_heads) * ((rows + kTileRows - 1) / kTileRows);
    const int64_t tiles = (prefix_len + kTileTokens - 1) / kTileTokens;
    return static_cast<int>(std::max<int64_t>(1, std::min(tiles, sm_count / units)));
}

int64_t attn_prefix_slot_floats(int sm_count, int head_dim) {
    return static_cast<int64_t>(sm_count) * kTileRows * (head_dim + 4);
}

cudaError_t launch_attn_prefix(const AttnLaunch& L, float* slots, float* states, cudaStream_t s) {
    PrefixArgs a{};
    a.q = static_cast<const uint16_t*>(L.q->data);
    a.q_ts = L.q->token_stride;
    a.q_hs = L.q->head_stride;
    a.k = L.cache->k;
    a.v = L.cache->v;
    a.k_scale = L.cache->k_scale;
    a.v_scale = L.cache->v_scale;
    a.pages = L.cache->pages;
    a.kv_heads = L.cache->kv_heads;
    while ((1 << a.page_shift) < L.cache->page_size) ++a.page_shift;
    a.page_list = L.prefix_pages;
    a.len = static_cast<int>(L.prefix_len);
    a.group = L.q_heads / a.kv_heads;
    a.q_heads = L.q_heads;
    a.rows = L.batch * L.q_len * a.group;
    a.row_tiles = (a.rows + kTileRows - 1) / kTileRows;
    a.splits = attn_prefix_splits(a.rows, a.kv_heads, L.prefix_len, L.sm_count);
    a.scale_log2 = static_cast<float>(L.scale * 1.4426950408889634074);
    a.slots = slots;
    a.states = states;
    a.status = L.status;
    a.timeout_ns = wait_timeout_ns();
    if (L.cache->head_dim == 64)
        return L.fp16 ? run_prefix<64, true>(a, s) : run_prefix<64, false>(a, s);
    return L.fp16 ? run_prefix<128, true>(a, s) : run_prefix<128, false>(a, s);
}

}  // namespace dg
