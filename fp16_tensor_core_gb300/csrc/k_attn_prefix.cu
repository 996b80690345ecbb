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
// the prefix.  Roles: four warps each take the codes of the keys and of the
// values from the cache and write them as FP16 (exact) into swizzled shared
// memory, in two stages; one thread issues the MMAs; two groups of four warps
// turn scores into weights.  Tiles of even and odd number are two streams with a group, a
// stage, S and O of their own (a tile's weights take the place of its
// scores), joined at the end: while one stream's weights are formed the
// tensor cores work for the other.  One stream alone left them idle: its
// softmax is a chain of latencies (4300 cycles a tile against 1024 of MMA).
//
// A warp of the softmax reads its rows in the MMA fragment shape (a thread
// holds 2 of 8 columns of 4 rows) instead of a row per thread: the per-token
// factors it needs are then a quarter, and packed pairs of columns feed the
// two-wide FP32 instructions.  The reference m of a row lies 2^7 below its
// maximum when it is set, and follows only when that has grown by 2^8: O is
// rescaled rarely, weights stay below 2^15, and what FP16's subnormals lose is
// at most 2^-32 of the row's largest contribution a token.
//
// Measured: 384 rows x 12000 tokens x 8 heads of 128 in 38 us, 0.26 of the
// tensor rate.  A pair of tiles takes 6600 cycles against 2048 of MMA; what
// shared memory has to pass for a tile (operands written and read, factors)
// is half of its bandwidth, and each stream waits 1900 of its cycles for the
// products between its softmax passes.  Twice the softmax warps, or codes on
// their way through shared memory, were slower.
//
// V is stored token-major, as in the cache: the second product takes it as an
// operand whose N side is contiguous (bit 16 of the instruction descriptor).
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_common.cuh"
#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "prefix_barriers.h"

namespace dg {
namespace {

constexpr int kTileTokens = 128;
constexpr int kTileRows = kPrefixTileRows;
constexpr int kThreads = 640;   // warpgroups: softmax of even and of odd tiles, keys, values, MMA
// log2 of a row's largest weight: when the reference moves, and what it may
// grow to before it moves again (FP16 ends at 2^16).
constexpr float kLow = 7.0f, kHigh = 15.0f;
// Registers a thread of the softmax, the conversion and the MMA warps.  Their
// sum has to be there at the launch (an increase waits for what others give
// back, and for ever for what nobody has): run_prefix() looks.
constexpr int kSoftmaxRegs = 144, kConvertRegs = 72, kMmaRegs = 40;

__device__ __forceinline__ void tmem_load_frag4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_store_frag4(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
          "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
          "r"(r[14]), "r"(r[15])
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

// wait_bounded for waits that are on the critical path and often short: the
// clock (a read of about a microsecond) is first looked at after 64 tries.
__device__ __forceinline__ bool wait_soon(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return wait_bounded(bar, parity, ctl);
}
__device__ __forceinline__ bool wait_soon(uint64_t* bars, prefix::Phase p, const WaitCtl& ctl) {
    return wait_soon(bars + p.barrier, p.parity, ctl);
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
    static constexpr int kOCol = 256;                            // tensor memory: S0, S1, O0, O1
    static_assert(kOCol + 2 * D <= 512, "tensor memory");
    static constexpr int kKAt = kOperandBytes;
    static constexpr int kVAt = kKAt + 2 * kOperandBytes;
    static constexpr int kFactorsAt = kVAt + 2 * kOperandBytes;  // [slots][3][128] per-token factors
    static constexpr int kRowsAt = kFactorsAt + prefix::kFactorSlots * 3 * 128 * 4;   // [2][2][128] cache rows
    static constexpr int kQScaleAt = kRowsAt + 2 * 2 * 128 * 8;
    static constexpr int kBarsAt = kQScaleAt + 128 * 4;
    static_assert(prefix::kBarriers * 8 + 8 <= 256, "barriers, tensor memory's address, abort flag");
    static constexpr int kSmem = kBarsAt + 256 + 1024;           // and alignment
};

// What BF16 queries are scaled up by (query_scale) leaves a score with the
// key's scale, which is applied first, so that their product stays in FP32.
template <bool kFp16>
constexpr float kKeyFactor = kFp16 ? 1.0f : 0x1p-14f;

// The keys' (or values') four warps: codes from the cache to swizzled FP16.
template <int D, bool kFp16, bool kValues>
__device__ __forceinline__ void convert_role(const PrefixArgs& a, uint8_t* smem, uint64_t* bars,
                                             const WaitCtl& ctl, int tile0, int tiles, int head) {
    using S = PrefixShape<D>;
    constexpr uint32_t kBarrier = kValues ? 4 : 2;
    // A stage is free when the product that reads it is done.  The factors
    // are read later, but are four deep: the scores of tile j come after the
    // weights of tile j - 2.
    float* factors = reinterpret_cast<float*>(smem + S::kFactorsAt);
    int64_t* cache_rows = reinterpret_cast<int64_t*>(smem + S::kRowsAt) + (kValues ? 2 * 128 : 0);
    uint8_t* operand = smem + (kValues ? S::kVAt : S::kKAt);
    const int i = static_cast<int>(threadIdx.x) & 127;
    // 16 bytes a thread and pass: 32 tokens x 64 dims.  Four chunks of two
    // tokens a quarter warp keep its stores (chunks 2c, then 2c + 1, of FP16)
    // in different banks.
    constexpr int kHalves = S::kHalves, kPasses = 4 * kHalves;   // pass s: tokens 32 (s / kHalves) ..
    const int token0 = i >> 2, swz = token0 & 7;
    const uint32_t dst0 = smem_addr(operand) + token0 * 128 + ((2 * (i & 3)) ^ swz) * 16;
    const uint32_t dst1 = smem_addr(operand) + token0 * 128 + ((2 * (i & 3) + 1) ^ swz) * 16;
    const int in_page = (1 << a.page_shift) - 1;
    // Order of the factors: a softmax thread's columns 2c and 2c + 1 of two
    // groups of 8 lie side by side, one load of 16 bytes.
    const int factor_at = (i & ~15) + ((i >> 1) & 3) * 4 + ((i >> 3) & 1) * 2 + (i & 1);
    const uint8_t* codes = (kValues ? a.v : a.k) + (i & 3) * 16;
    // Page of token i of tile j (kNoToken past the end); its cache row is
    // formed later, so that nothing waits for the load.
    constexpr int kNoToken = -0x7FFFFFFF;
    auto find_page = [&](int j) {
        const int t = (tile0 + j) * kTileTokens + i;
        return j < tiles && t < a.len ? a.page_list[t >> a.page_shift] : kNoToken;
    };
    auto row_of = [&](int p, int j) -> int64_t {   // -1: none
        if (p < 0 || p >= a.pages) {
            if (p != kNoToken) atomicOr(a.status, kStatusBadArgument);
            return -1;
        }
        const int t = (tile0 + j) * kTileTokens + i;
        return ((static_cast<int64_t>(p) * a.kv_heads + head) << a.page_shift) + (t & in_page);
    };
    // The next tile's codes wait in registers: through shared memory they
    // would take its bandwidth, which is what the CTA runs short of.
    uint4 x[kPasses];
    auto fetch = [&](int j) {
        const int64_t* rows = cache_rows + (j & 1) * 128;
#pragma unroll
        for (int s = 0; s < kPasses; ++s) {
            const int64_t r = rows[token0 + 32 * (s / kHalves)];
            x[s] = make_uint4(0, 0, 0, 0);
            if (r >= 0) x[s] = __ldg(reinterpret_cast<const uint4*>(codes + r * D + 64 * (s % kHalves)));
        }
    };
    auto load_scales = [&](int64_t r, float* sk, float* sv) {
        *sk = 0.0f;
        *sv = -1.0f;   // no token
        if (!kValues && r >= 0) {
            *sk = __ldg(a.k_scale + r);
            *sv = __ldg(a.v_scale + r);
        }
    };
    float sk, sv;
    int64_t row1;   // this thread's token of the next tile
    {
        const int p0 = find_page(0), p1 = find_page(1);
        const int64_t row0 = row_of(p0, 0);
        row1 = row_of(p1, 1);
        cache_rows[i] = row0;
        cache_rows[128 + i] = row1;
        load_scales(row0, &sk, &sv);
    }
    named_bar_sync(kBarrier, 128);
    fetch(0);
    named_bar_sync(kBarrier, 128);   // before rows are replaced
    bool ok = true;
    for (int j = 0; j < tiles && ok; ++j) {
        const int b = j & 1;
        const int page2 = find_page(j + 2);   // on its way meanwhile
        if (j >= 2)
            ok = __all_sync(0xFFFFFFFFu, wait_soon(bars, kValues ? prefix::output(j - 2) : prefix::scores(j - 2), ctl));
        if (ok) {
#pragma unroll
            for (int s = 0; s < kPasses; ++s) {
                const uint32_t at = b * S::kOperandBytes + (s % kHalves) * S::kColumnBytes + (s / kHalves) * (32 * 128);
                uint32_t h[8];
                codes_to_halves(x[s].x, &h[0], &h[1]);
                codes_to_halves(x[s].y, &h[2], &h[3]);
                codes_to_halves(x[s].z, &h[4], &h[5]);
                codes_to_halves(x[s].w, &h[6], &h[7]);
                st_shared_v4(dst0 + at, h[0], h[1], h[2], h[3]);
                st_shared_v4(dst1 + at, h[4], h[5], h[6], h[7]);
            }
            if constexpr (!kValues) {
                float* f = factors + prefix::factor_slot(j) * 3 * 128 + factor_at;
                const float safe = sv < 0x1p-100f ? 0x1p-100f : sv;
                f[0] = sk * kKeyFactor<kFp16>;
                f[128] = sv == -1.0f ? -INFINITY : __log2f(safe);
                f[256] = sv == -1.0f ? 0.0f : rcp(safe);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if ((i & 31) == 0) {
                mbar_arrive(bars + (kValues ? prefix::values(j) : prefix::keys(j)).barrier);
                if (!kValues) mbar_arrive(bars + prefix::factors(j).barrier);
            }
            if (j + 1 < tiles) {
                fetch(j + 1);
                load_scales(row1, &sk, &sv);
            }
        }
        // rows of tile j (whose loads were issued an iteration ago) make room
        // for those of tile j + 2; after a wait that ran out the four warps
        // leave together
        row1 = row_of(page2, j + 2);
        cache_rows[b * 128 + i] = row1;
        ok = named_bar_and(kBarrier, 128, ok);
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
    float* qscale = reinterpret_cast<float*>(smem + S::kQScaleAt);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBarsAt);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + prefix::kBarriers);
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        // arrivals: a thread, four warps, or a commit of the MMA thread
        mbar_init(bars + prefix::kQueries, 128);
        for (int b = 0; b < 2; ++b) {
            mbar_init(bars + prefix::kKeys + b, 4);
            mbar_init(bars + prefix::kValues + b, 4);
            mbar_init(bars + prefix::kScores + b, 1);
            mbar_init(bars + prefix::kWeights + b, 4);
            mbar_init(bars + prefix::kOutput + b, 1);
        }
        for (int f = 0; f < prefix::kFactorSlots; ++f) mbar_init(bars + prefix::kFactors + f, 4);
        mbar_init(bars + prefix::kDrain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 16) {
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
    // With several shares the own tokens' kernels ran before: they waited for
    // all that this one reads, which may begin while they end.
    if (a.splits == 1) pdl_wait();

    // The softmax warps take the registers that the others leave.
    if (warp < 8) {
        // -------------------------------------------------- queries, softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftmaxRegs));
        const int b = warp >> 2;   // stream
        const int g = lane >> 2, c = lane & 3;
        if (b == 0) {   // thread i takes row i of the tile, scaled by a power of two (BF16)
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
                const PowerOfTwo p = query_scale(top);
                mul = p.inverse;
                factor *= p.value / kKeyFactor<kFp16>;
            }
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                if constexpr (!kFp16) w[k] = bf16_to_half8(w[k], mul);
                st_shared_v4(smem_addr(sq + (k >> 3) * S::kColumnBytes + i * 128 + (((k & 7) ^ (i & 7)) * 16)),
                             w[k].x, w[k].y, w[k].z, w[k].w);
            }
            qscale[i] = factor;
            fence_proxy_async_smem();
            mbar_arrive(bars + prefix::kQueries);
        }
        named_bar_sync(1, 256);   // before the factors are read
        const int quarter = warp & 3;
        // row 16 h + 8 i + g of the warp's 32: index 2 h + i
        float m[4], qs[4];
        f32x2 l[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            m[x] = -INFINITY;
            l[x] = 0ull;
            qs[x] = qscale[32 * quarter + 16 * (x >> 1) + 8 * (x & 1) + g];
        }
        const uint32_t quad = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        const uint32_t o_col = S::kOCol + D * b;
        bool ok = true;
        for (int j = b; j < tiles; j += 2) {
            ok = *ctl.abort_flag == 0 && wait_soon(bars, prefix::factors(j), ctl) &&
                 wait_soon(bars, prefix::scores(j), ctl);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after_sync();
            const float* f = factors + prefix::factor_slot(j) * 3 * 128 + 4 * c;
            // 16 rows at a time, in one pass against the reference as it
            // stands; only where a row's maximum has outgrown it (the first
            // tiles) the reference moves and the pass is made again.
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t half = quad + (static_cast<uint32_t>(16 * h) << 16);
                const int x0 = 2 * h;
                uint32_t w[32];
                f32x2 part[2];
                float top[2];
#pragma unroll 1
                for (int again = 0; again < 2; ++again) {
                    const float base0 = m[x0] == -INFINITY ? 0.0f : -m[x0];
                    const float base1 = m[x0 + 1] == -INFINITY ? 0.0f : -m[x0 + 1];
                    const f32x2 base[2] = {pack(base0, base0), pack(base1, base1)};
                    const f32x2 q2[2] = {pack(qs[x0], qs[x0]), pack(qs[x0 + 1], qs[x0 + 1])};
                    part[0] = part[1] = 0ull;
                    top[0] = top[1] = -INFINITY;
                    uint32_t s[2][16];
                    ulonglong2 sk2, lg2, rs2;   // factors of two groups of 8 columns
                    tmem_load_frag4(half + 128 * b, s[0]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t(&v)[16] = s[k & 1];
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(v[e]));
                        if (k < 3) tmem_load_frag4(half + 128 * b + 32 * (k + 1), s[(k + 1) & 1]);
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            if ((n & 1) == 0) {
                                const int at = 32 * k + 8 * n;
                                sk2 = *reinterpret_cast<const ulonglong2*>(f + at);
                                lg2 = *reinterpret_cast<const ulonglong2*>(f + 128 + at);
                                rs2 = *reinterpret_cast<const ulonglong2*>(f + 256 + at);
                            }
                            const f32x2 sk = n & 1 ? sk2.y : sk2.x, lg = n & 1 ? lg2.y : lg2.x,
                                        rs = n & 1 ? rs2.y : rs2.x;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const f32x2 sc = pack(__uint_as_float(v[4 * n + 2 * i]),
                                                      __uint_as_float(v[4 * n + 2 * i + 1]));
                                const float2 y = unpack(fma2(mul2(sc, sk), q2[i], add2(lg, base[i])));
                                top[i] = fmaxf(top[i], fmaxf(y.x, y.y));
                                const float e0 = ex2(y.x), e1 = ex2(y.y);
                                part[i] = fma2(pack(e0, e1), rs, part[i]);
                                w[8 * k + 2 * n + i] = f32x2_to_f16x2(e0, e1);
                            }
                        }
                    }
                    bool grew = false;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
                        top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
                        // relative to the reference, or to 0 while there is none
                        grew |= m[x0 + i] == -INFINITY ? top[i] > -INFINITY : top[i] > kHigh;
                    }
                    if (!__any_sync(0xFFFFFFFFu, grew) || again == 1) break;
                    float by[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float& ref = m[x0 + i];
                        const bool none = ref == -INFINITY;
                        const bool move = none ? top[i] > -INFINITY : top[i] > kHigh;
                        by[i] = !move ? 1.0f : none ? 0.0f : ex2(kLow - top[i]);
                        if (move) ref = none ? top[i] - kLow : ref + (top[i] - kLow);
                        l[x0 + i] = mul2(l[x0 + i], pack(by[i], by[i]));
                    }
                    // O as the stream's previous tile left it; a wait that
                    // runs out ends the loop below
                    if (j >= 2 && __all_sync(0xFFFFFFFFu, wait_soon(bars, prefix::output(j - 2), ctl))) {
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int p = 0; p < D / 32; ++p) {
                            uint32_t o[16];
                            tmem_load_frag4(half + o_col + 32 * p, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                asm volatile("" : "+r"(o[k]));
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * by[(k >> 1) & 1]);
                            }
                            tmem_store_frag4(half + o_col + 32 * p, o);
                        }
                    }
                }
                l[x0] = add2(l[x0], part[0]);
                l[x0 + 1] = add2(l[x0 + 1], part[1]);
                tmem_store_pairs16(half + 128 * b, w);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + prefix::weights(j).barrier);
        }
        // ---- both streams' results, joined by the first group
        if (ok && tiles > b) {
            const int last = tiles - 1 - ((tiles - 1 - b) & 1);
            ok = wait_soon(bars, prefix::output(last), ctl);
        }
        // Every MMA is done: the operands' memory is free.  (And the kernel
        // before this one: whoever waits for this one waits for both.)
        pdl_wait();
        ok = named_bar_and(3, 256, ok);
        tc_fence_after_sync();
        float* other = reinterpret_cast<float*>(smem + S::kKAt);   // the second stream's states
        float sums[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float2 part = unpack(l[x]);
            sums[x] = part.x + part.y;
            sums[x] += __shfl_xor_sync(0xFFFFFFFFu, sums[x], 1);
            sums[x] += __shfl_xor_sync(0xFFFFFFFFu, sums[x], 2);
        }
        const bool second = tiles > 1;   // the second stream has a tile
        if (ok && b == 1 && second) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float* row[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    row[i] = other + (32 * quarter + 16 * h + 8 * i + g) * S::kState;
                    if (c == 0) *reinterpret_cast<float2*>(row[i]) = make_float2(m[2 * h + i], sums[2 * h + i]);
                }
#pragma unroll 1
                for (int part = 0; part < D / 32; ++part) {
                    uint32_t o[16];
                    tmem_load_frag4(quad + (static_cast<uint32_t>(16 * h) << 16) + o_col + 32 * part, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) asm volatile("" : "+r"(o[k]));
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            *reinterpret_cast<uint2*>(row[i] + 4 + 32 * part + 8 * n + 2 * c) =
                                make_uint2(o[4 * n + 2 * i], o[4 * n + 2 * i + 1]);
                }
            }
        }
        ok = named_bar_and(3, 256, ok);
        if (ok && b == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float* dst[2];
                const float* row[2];
                float w0[2], w1[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int x = 2 * h + i;
                    const int in_tile = 32 * quarter + 16 * h + 8 * i + g, r = rt * kTileRows + in_tile;
                    row[i] = other + in_tile * S::kState;
                    const float2 ml = second ? *reinterpret_cast<const float2*>(row[i]) : make_float2(-INFINITY, 0.0f);
                    const float top = fmaxf(m[x], ml.x), base = top == -INFINITY ? 0.0f : top;
                    w0[i] = ex2(m[x] - base);
                    w1[i] = ex2(ml.x - base);
                    dst[i] = nullptr;
                    if (r >= a.rows) continue;
                    if (a.splits > 1) {
                        dst[i] = a.slots + (static_cast<int64_t>(blockIdx.x) * kTileRows + in_tile) * S::kState;
                    } else {
                        const int token = r / a.group;
                        const int64_t at = static_cast<int64_t>(token) * a.q_heads + head * a.group + r - token * a.group;
                        dst[i] = a.states + at * S::kState;
                    }
                    if (c == 0)
                        *reinterpret_cast<float2*>(dst[i]) =
                            make_float2(top, w0[i] * sums[x] + (second ? w1[i] * ml.y : 0.0f));
                }
                __syncwarp();   // the rows past the end skipped ahead
#pragma unroll 1
                for (int part = 0; part < D / 32; ++part) {
                    uint32_t o[16];
                    tmem_load_frag4(quad + (static_cast<uint32_t>(16 * h) << 16) + o_col + 32 * part, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) asm volatile("" : "+r"(o[k]));
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (dst[i] == nullptr) continue;
                            const int d = 4 + 32 * part + 8 * n + 2 * c;
                            float2 y = make_float2(__uint_as_float(o[4 * n + 2 * i]) * w0[i],
                                                   __uint_as_float(o[4 * n + 2 * i + 1]) * w0[i]);
                            if (second) {
                                const float2 z = *reinterpret_cast<const float2*>(row[i] + d);
                                y.x = fmaf(w1[i], z.x, y.x);
                                y.y = fmaf(w1[i], z.y, y.y);
                            }
                            *reinterpret_cast<float2*>(dst[i] + d) = y;
                        }
                    __syncwarp();
                }
            }
        }
    } else if (warp < 16) {
        // ---------------------------- codes to operands: keys, then values' warps
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kConvertRegs));
        if (warp < 12)
            convert_role<D, kFp16, false>(a, smem, bars, ctl, tile0, tiles, head);
        else
            convert_role<D, kFp16, true>(a, smem, bars, ctl, tile0, tiles, head);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kMmaRegs));
        if (warp == 16 && lane == 0) {
            // -------------------------------------------------- MMA issue
            constexpr uint32_t kScoreDesc = idesc_f32acc(kTileRows, kTileTokens, 0, 0);
            constexpr uint32_t kValueDesc = idesc_f32acc(kTileRows, D, 0, 0) | (1u << 16);
            // Descriptors are formed once: a step along k is an addition to
            // the start address (in 16-byte units).  Formed at each MMA they
            // kept this thread, and with it the tensor cores, at 90 cycles
            // an MMA.
            const uint64_t q_desc = sdesc_k_major_sw128(smem_addr(sq));
            const uint64_t k_desc = sdesc_k_major_sw128(smem_addr(smem + S::kKAt));
            const uint64_t v_desc = sdesc_mn_major_sw128(smem_addr(smem + S::kVAt), S::kColumnBytes);
            constexpr uint64_t kStage = S::kOperandBytes >> 4, kColumn = S::kColumnBytes >> 4;
            auto scores = [&](int j) {
                const uint64_t kd = k_desc + (j & 1) * kStage;
                const uint32_t d = tmem + 128 * (j & 1);
#pragma unroll
                for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        mma_f16(d, q_desc + h * kColumn + 2 * x, kd + h * kColumn + 2 * x, kScoreDesc, h > 0 || x > 0);
                mma_commit(bars + prefix::scores(j).barrier);
            };
            bool ok = wait_soon(bars + prefix::kQueries, 0, ctl);
            bool issued = false;
            for (int j = 0; j < 2 && j < tiles && ok; ++j) {
                ok = wait_soon(bars, prefix::keys(j), ctl);
                if (!ok) break;
                tc_fence_after_sync();
                issued = true;
                scores(j);
            }
            for (int j = 0; j < tiles && ok; ++j) {
                const int b = j & 1;
                ok = wait_soon(bars, prefix::values(j), ctl) && wait_soon(bars, prefix::weights(j), ctl);
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t vd = v_desc + b * kStage;
#pragma unroll
                for (int x = 0; x < kTileTokens / 16; ++x)
                    mma_f16_ts(tmem + S::kOCol + D * b, tmem + 128 * b + 8 * x, vd + x * (2048 >> 4), kValueDesc,
                               j > 1 || x > 0);
                mma_commit(bars + prefix::output(j).barrier);
                if (j + 2 < tiles) {
                    // they take the place of the weights just read
                    ok = wait_soon(bars, prefix::keys(j + 2), ctl) && wait_soon(bars, prefix::output(j), ctl);
                    if (!ok) break;
                    tc_fence_after_sync();
                    scores(j + 2);
                }
            }
            if (issued) {
                // Tensor memory is freed below: wait for every MMA issued.
                mma_commit(bars + prefix::kDrain);
                wait_bounded(bars + prefix::kDrain, 0, ctl, false);
            }
        }
    }
    tc_fence_before_sync();
    cta_sync_diverged();
    tc_fence_after_sync();
    if (warp == 16) {
        __syncwarp();
        tmem_dealloc<512>(tmem);
    }
}

template <int D, bool kFp16>
cudaError_t run_prefix(const PrefixArgs& a, cudaStream_t s) {
    const cudaError_t set = allow_smem(attn_prefix_kernel<D, kFp16>, PrefixShape<D>::kSmem);
    if (set != cudaSuccess) return set;
    static const cudaError_t registers = [] {
        cudaFuncAttributes f{};
        const cudaError_t e = cudaFuncGetAttributes(&f, attn_prefix_kernel<D, kFp16>);
        if (e != cudaSuccess) return e;
        return kThreads / 128 * f.numRegs >= 2 * kSoftmaxRegs + 2 * kConvertRegs + kMmaRegs
                   ? cudaSuccess
                   : cudaErrorInvalidConfiguration;
    }();
    if (registers != cudaSuccess) return registers;
    const unsigned blocks = static_cast<unsigned>(a.kv_heads) * a.splits * a.row_tiles;
    return launch_kernel(attn_prefix_kernel<D, kFp16>, dim3(blocks), dim3(kThreads), PrefixShape<D>::kSmem, s, a);
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
