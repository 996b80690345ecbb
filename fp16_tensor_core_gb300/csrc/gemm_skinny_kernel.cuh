// gemm_skinny_kernel.cuh -- the split-K tensor-core kernel that
// k_gemm_skinny.cu describes, as a template: k_gemm_skinny.cu holds the plain
// form, k_gemm_skinny_fused.cu the one with a fused epilogue (kFused: row and
// column scales, bias, activation, residual in place of one scale).
#pragma once

#include <mutex>

#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "gemm_common.cuh"

namespace dg {
namespace {

constexpr int kRows = kSkinnyTileRows;            // MMA M: rows of B per tile
constexpr int kWBytes = kRows * kBKBytes;         // 16 KB of B per K block
constexpr int kBarBytes = 512;
constexpr uint32_t kEpiBar = 1;                   // named barrier of the epilogue warps
constexpr uint32_t kEpiThreads = 128;
// Hand-off to warps 0-3 for a CTA's last tile: valid, tile, accumulator,
// first and last CTA of the tile, the first CTA's slot, staged.
constexpr int kHelpInts = 7;

// K blocks in flight per CTA for MMA N = nc (the rows of A, padded): as many
// as fit in 227 KB of shared memory, rounded down to an even number.
constexpr int ring_kblocks(int nc) {
    const int r = (kSmemLimit - 1024 - kBarBytes) / (kWBytes + nc * kBKBytes);
    const int even = r & ~1;
    return even > 12 ? 12 : even;
}

// Configuration for MMA N = NC (16, 32, 64 or 128 rows of A) with KPS
// consecutive K blocks per stage, loaded together so that each row of B is
// requested KPS x 128 contiguous bytes at a time.
template <int NC, int KPS>
struct SkCfg {
    static constexpr int kXBytes = NC * kBKBytes;           // A rows per K block
    static constexpr int kKBBytes = kWBytes + kXBytes;
    static constexpr int kRing = ring_kblocks(NC);
    static constexpr int kStages = kRing / KPS;
    static constexpr int kStageW = KPS * kWBytes;
    static constexpr int kStageX = KPS * kXBytes;
    static constexpr int kSmemBytes = 1024 + kRing * kKBBytes + kBarBytes;
    static constexpr int kScalesOff = kRing * kKBBytes + kBarBytes;   // fused: the rows' scales of A (rests [NC], wholes [NC])
    static constexpr int kResidualOff = kScalesOff + NC * 8;          // and the tile's residual [NC][128]
    static constexpr int kFusedSmemBytes = kSmemBytes + NC * 8 + NC * kRows * 2;
    static constexpr uint32_t kTmemCols = pow2_at_least(2 * NC);   // two accumulators
    static constexpr uint32_t kIdesc = idesc_f32acc(kRows, NC, 0, 0);
    static_assert(NC % 16 == 0 && NC >= 16 && NC <= kSplitkMaxCols, "MMA N");
    static_assert(kRing % KPS == 0 && kStages <= 12, "ring");
    static_assert(kFusedSmemBytes <= kSmemLimit, "shared memory");
    static_assert(kXBytes % 1024 == 0, "1024-byte aligned A blocks (128-byte swizzle atoms)");
    // barriers: full/empty per stage, 2 + 2 accumulator, drain, fix-up,
    // helpers; then the TMEM address, the abort flag, the last-arrival flag
    // and the helpers' hand-off block
    static_assert((2 * kStages + 7) * 8 + 3 * 4 + kHelpInts * 4 <= kBarBytes, "barrier block");
};

struct SkParams {
    void* D;
    int M, N, K;
    const float* sa;
    const float* sb;
    const float* sd;
    int out_kind;
    uint32_t* status;
    uint64_t timeout_ns;
    int skip_first_load;
    uint32_t* amax_out;
    float* partials;       // [2 * gridDim.x][NC / 4][128] float4: column quads
    uint32_t* counts;      // [tiles]
    int tiles;             // ceil(N / tile_rows)
    int tile_rows;         // rows of B per tile: 128, or a row range (<= 128)
    int kblocks;           // ceil(K / BK)
    int prefetch_kblocks;  // B boxes of its range a CTA moves into L2 up front
    Epilogue epi;          // of the fused kernels only
};

// CTA i's range of units is [range_start(i), range_start(i + 1)).
__device__ __forceinline__ int64_t range_start(int i, int G, int64_t units) {
    return static_cast<int64_t>(i) * units / G;
}

// The CTA whose range holds unit u.
__device__ __forceinline__ int cta_of_unit(int64_t u, int G, int64_t units) {
    return static_cast<int>(((u + 1) * G - 1) / units);
}

// Workspace slots: a CTA has at most two partial segments, its first (slot
// 2c) and its last (2c + 1).  In a split tile t, every CTA after the first
// one (c_first) starts its range inside t, so its segment there is its first
// (slot 2c); c_first's segment is its first only if its range starts exactly
// at the tile.

// Scale, convert and store rows c0 .. c0 + jn - 1 of A's side (m) at column
// n: one branch on the output type, then one strided store per row.
__device__ __forceinline__ void store_chunk16(const SkParams& p, int c0, int n, int jn,
                                              const float (&v)[16], float alpha) {
    const int64_t ld = p.N;
    const int64_t off = static_cast<int64_t>(c0) * ld + n;
    if (p.out_kind == kOutE4M3) {
        uint8_t* d = static_cast<uint8_t*>(p.D) + off;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j < jn) d[j * ld] = static_cast<uint8_t>(f32x2_to_e4m3x2(v[j] * alpha, 0.0f) & 0xFFu);
    } else if (p.out_kind == kOutFP16) {
        uint16_t* d = static_cast<uint16_t*>(p.D) + off;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j < jn) d[j * ld] = static_cast<uint16_t>(f32x2_to_f16x2(v[j] * alpha, 0.0f) & 0xFFFFu);
    } else {
        uint16_t* d = static_cast<uint16_t*>(p.D) + off;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j < jn) d[j * ld] = static_cast<uint16_t>(f32x2_to_bf16x2(v[j] * alpha, 0.0f) & 0xFFFFu);
    }
}

// The fused epilogue of column n of D (a row of B): its scale of B and bias,
// loaded while the tile's main loop runs.
struct FusedColumn {
    float sb = 1.0f, bias = 0.0f;
};
__device__ __forceinline__ FusedColumn fused_column(const SkParams& p, bool live, int n) {
    FusedColumn c;
    if (live && p.sb != nullptr) c.sb = ld_float(p.sb + static_cast<int64_t>(n) * p.epi.sb_step);
    if (live && p.epi.bias != nullptr) c.bias = ld_float(p.epi.bias + n);
    return c;
}

// The residual of tile t into shared memory while the tile's main loop runs:
// asynchronous copies of 16 bytes of a row, of 4 where N is only even, or
// elements one by one.  (Never the read-only path: D
// may be the residual.)  Read at the end instead, 16 rows at a time, behind
// the weight stream of the next launch, it took 6 us of a 64 x 4096 x 11008
// product's 21.
__device__ __forceinline__ void stage_residual(const SkParams& p, uint16_t* tile, int t, int r) {
    if ((p.N & 7) == 0 && (p.tile_rows & 7) == 0) {
        for (int i = r; i < p.M * (kRows / 8); i += 128) {
            const int m = i >> 4, at = 8 * (i & 15), n = t * p.tile_rows + at;
            if (at < p.tile_rows && n < p.N)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                             :: "r"(smem_addr(tile + m * kRows + at)),
                                "l"(p.epi.residual + static_cast<int64_t>(m) * p.N + n)
                             : "memory");
        }
        return;
    }
    if ((p.N & 1) == 0 && (p.tile_rows & 1) == 0) {
        for (int i = r; i < p.M * (kRows / 2); i += 128) {
            const int m = i >> 6, at = 2 * (i & 63), n = t * p.tile_rows + at;
            if (at < p.tile_rows && n < p.N)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                             :: "r"(smem_addr(tile + m * kRows + at)),
                                "l"(p.epi.residual + static_cast<int64_t>(m) * p.N + n)
                             : "memory");
        }
        return;
    }
    const int n = t * p.tile_rows + r;
    if (r >= p.tile_rows || n >= p.N) return;
#pragma unroll 1
    for (int m0 = 0; m0 < p.M; m0 += 16) {
        uint32_t e[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (m0 + i < p.M)
                asm volatile("ld.global.u16 %0, [%1];"
                             : "=r"(e[i]) : "l"(p.epi.residual + static_cast<int64_t>(m0 + i) * p.N + n));
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (m0 + i < p.M) tile[(m0 + i) * kRows + r] = static_cast<uint16_t>(e[i]);
    }
}

// act(scale_a[m] scale_b[n] acc + bias[n]) + residual[m, n] for rows c0 ..
// c0 + jn - 1 (sa: the rows' scales, rests and then wholes, residual: row c0 of
// this thread's column, both in shared memory); returns the largest magnitude
// (ordered bits).  Two products more a pair for the wholes: a branch around
// them took 0.3 to 0.7 us more of 64 x 4096 x 11008's 16.9.
template <int NC>
__device__ __forceinline__ uint32_t fuse16(const SkParams& p, int c0, int jn, const FusedColumn& col,
                                           ByScale out, const float* sa, const uint16_t* residual,
                                           float (&f)[16]) {
    pair v[8];
    const ScaleParts column = scale_parts(col.sb);
    const float* wholes = sa + NC;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ulonglong2 s = reinterpret_cast<const ulonglong2*>(sa + c0)[i];
        const ulonglong2 w = reinterpret_cast<const ulonglong2*>(wholes + c0)[i];
        const pair x = pair_mul(pair_mul(pair_of(f[4 * i], f[4 * i + 1]), w.x), pair_of(column.whole));
        const pair y = pair_mul(pair_mul(pair_of(f[4 * i + 2], f[4 * i + 3]), w.y), pair_of(column.whole));
        v[2 * i] = pair_fma(x, pair_mul(s.x, pair_of(column.rest)), pair_of(col.bias));
        v[2 * i + 1] = pair_fma(y, pair_mul(s.y, pair_of(column.rest)), pair_of(col.bias));
    }
    with_activation(p.epi.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = activation(act.value, v[i]);
    });
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (p.epi.residual != nullptr) {
            const uint32_t w = residual[2 * i * kRows] | static_cast<uint32_t>(residual[(2 * i + 1) * kRows]) << 16;
            const float2 x = p.epi.residual_fp16 != 0
                                 ? f16x2_to_f32x2(w)
                                 : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
            v[i] = pair_add(v[i], pair_of(x.x, x.y));
        }
        const float2 y = floats_of(v[i]);
        if (2 * i + 1 < jn)
            top = pair_top(v[i], top);
        else if (2 * i < jn)
            top = pair_top(pair_of(y.x), top);
        f[2 * i] = y.x * out.pre * out.inv;
        f[2 * i + 1] = y.y * out.pre * out.inv;
    }
    return __float_as_uint(top);
}

// Adds up, scales and stores the 16-column chunks c0 = c0_begin,
// c0_begin + c0_step, ... (c0 < NC, c0 < M) of a finished tile for the
// calling thread's row r (its tensor-memory lane): the segments c_first ..
// c_last in that order, the own one (CTA me) from tensor memory, the others
// from the staged copies in shared memory or from their workspace slots.
// `first` holds chunk 0 when the CTA published its own partial.
template <int NC, bool kFused>
__device__ __forceinline__ void finish_chunks(const SkParams& p, uint8_t* smem, uint32_t tacc,
                                              int r, int n, int c0_begin, int c0_step, int me,
                                              int c_first, int c_last, int first_slot,
                                              bool staged, int quads, const float (&first)[16],
                                              float alpha, uint32_t& amax_bits,
                                              const FusedColumn& column, ByScale out, const float* sa,
                                              const uint16_t* residual_tile) {
    const int others = c_last - c_first;
    const bool live = r < p.tile_rows && n < p.N;
#pragma unroll 1
    for (int c0 = c0_begin; c0 < NC && c0 < p.M; c0 += c0_step) {
        float v[16];
        if (c_last > c_first && c0 == 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = first[j];
        } else {
            uint32_t raw[16];
            __syncwarp();
            tmem_load_16cols(tacc + static_cast<uint32_t>(c0), raw);
            tmem_load_wait(raw);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(raw[j]);
        }
        if (staged) {
            // Segments in order c_first .. c_last from the staged
            // copies, the own one written into its position first
            // (this thread reads back only what it wrote itself).
            float4* stage = reinterpret_cast<float4*>(smem) + (c0 >> 2) * kRows + r;
            const int seg_stride = quads * kRows;   // float4s per position
            float4* own = stage + (me - c_first) * seg_stride;
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (c0 + 4 * g < p.M)
                    own[g * kRows] = make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2],
                                                 v[4 * g + 3]);
            float4 sum[4];
#pragma unroll
            for (int g = 0; g < 4; ++g)
                sum[g] = c0 + 4 * g < p.M ? stage[g * kRows]
                                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
            for (int i = 1; i <= others; ++i) {
                const float4* w = stage + i * seg_stride;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (c0 + 4 * g < p.M) {
                        const float4 x = w[g * kRows];
                        sum[g].x += x.x;
                        sum[g].y += x.y;
                        sum[g].z += x.z;
                        sum[g].w += x.w;
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                v[4 * g] = sum[g].x;
                v[4 * g + 1] = sum[g].y;
                v[4 * g + 2] = sum[g].z;
                v[4 * g + 3] = sum[g].w;
            }
        } else if (c_last > c_first) {
            // Sum the segments in order c_first .. c_last, the own
            // one from tensor memory, the others from their slots.
            // The slots of four segments are requested together
            // and then added in order, so the order (and the
            // result) is fixed while four loads are in flight.
            float sum[16];
#pragma unroll 1
            for (int cb = c_first; cb <= c_last; cb += 4) {
                float4 x[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = cb + i;
                    const int slot = c == c_first ? first_slot : 2 * c;
                    const float4* w = reinterpret_cast<const float4*>(p.partials) +
                                      static_cast<int64_t>(slot) * (NC / 4) * kRows;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        x[i][g] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (c <= c_last && c != me && c0 + 4 * g < p.M)
                            x[i][g] = __ldcg(w + ((c0 >> 2) + g) * kRows + r);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = cb + i;
                    if (c > c_last) break;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float y[4] = {x[i][g].x, x[i][g].y, x[i][g].z, x[i][g].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = 4 * g + e;
                            const float val = c == me ? v[j] : y[e];
                            sum[j] = c == c_first ? val : sum[j] + val;
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = sum[j];
        }
        if (live) {
            const int jn = min(16, p.M - c0);   // rows of A in this chunk
            if constexpr (kFused) {
                amax_bits = max(amax_bits, fuse16<NC>(p, c0, jn, column, out, sa, residual_tile + c0 * kRows + r, v));
                store_chunk16(p, c0, n, jn, v, 1.0f);
                continue;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j < jn) amax_bits = max(amax_bits, __float_as_uint(v[j]) & 0x7FFFFFFFu);
            store_chunk16(p, c0, n, jn, v, alpha);
        }
    }
}

template <bool kFp16In, int KPS, int NC, bool kFused>
__global__ void __launch_bounds__(kThreads, 1)
gemm_skinny_kernel(const __grid_constant__ CUtensorMap tmap_w,
                   const __grid_constant__ CUtensorMap tmap_x, const SkParams p) {
    constexpr int kBK = kFp16In ? 64 : 128;   // K elements per K block
    using C = SkCfg<NC, KPS>;
    constexpr int kStages = C::kStages;
    constexpr int kRingKBlocks = C::kRing;
    constexpr int kKBBytes = C::kKBBytes;
    constexpr int kXBytes = C::kXBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sW = smem;                          // B rows (MMA operand A)
    uint8_t* sX = smem + kStages * C::kStageW;   // A rows (MMA operand B)
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRingKBlocks * kKBBytes);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;   // [2]
    uint64_t* acc_empty = acc_full + 2;     // [2]
    uint64_t* drain = acc_empty + 2;        // [1]
    uint64_t* fix_bar = drain + 1;          // [1] partial tiles staged for the fix-up
    uint64_t* help_bar = fix_bar + 1;       // [1] last tile handed to warps 0-3
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(help_bar + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
    volatile int* last_flag = abort_flag + 1;
    volatile int* help = last_flag + 1;     // [kHelpInts]

    float* row_scales = reinterpret_cast<float*>(smem + C::kScalesOff);   // [NC], fused
    uint16_t* residual_tile = reinterpret_cast<uint16_t*>(smem + C::kResidualOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 4);
        }
        mbar_init(drain, 1);
        mbar_init(fix_bar, 1);
        mbar_init(help_bar, 1);
        *abort_flag = 0;
        *last_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmap_w);
        tma_prefetch_desc(&tmap_x);
    }
    if (warp == 2) {
        tmem_alloc<C::kTmemCols>(tmem_slot);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;

    const WaitCtl ctl{abort_flag, p.status, p.timeout_ns};
    const int G = gridDim.x;
    const int KB = p.kblocks;
    const int64_t units = static_cast<int64_t>(p.tiles) * KB;
    const int64_t u_begin = range_start(blockIdx.x, G, units);
    const int64_t n_units = range_start(blockIdx.x + 1, G, units) - u_begin;
    const int t_begin = static_cast<int>(u_begin / KB);
    const int kb_begin = static_cast<int>(u_begin - static_cast<int64_t>(t_begin) * KB);

    if (warp == 0 && lane == 0) {
        // Warm L2 with the start of this CTA's range of B while the preceding
        // kernel finishes (a prefetch only moves lines into L2).
        int t = t_begin, kb = kb_begin;
        for (int i = 0; i < p.prefetch_kblocks && i < n_units; ++i) {
            tma_prefetch_l2_2d(&tmap_w, kb * kBK, t * p.tile_rows);
            if (++kb == KB) { kb = 0; ++t; }
        }
    }
    pdl_wait();   // the prologue above overlaps the preceding kernel's tail
    // The next kernel may now take over each SM as soon as this grid's CTA
    // on it exits; it waits for the whole grid before touching memory.
    pdl_launch_dependents();

    // Every role walks the same segments: tile t from K block kb0 to kb_end.
    if (warp == 0 && lane == 0) {
        // ------------------------------------------------ TMA producer
        int stage = 0;
        uint32_t phase = 0;
        uint32_t issued_mask = 0;
        uint32_t issued_phase = 0;
        bool skip = p.skip_first_load != 0 && blockIdx.x == 0;
        bool ok = true;
        bool first_lap = true;   // every stage starts free: no wait on the first lap
        // bytes of one K block: tile_rows rows of B (the box) and NC rows of A
        const uint32_t kb_bytes = static_cast<uint32_t>(p.tile_rows * kBKBytes + kXBytes);
        int t = t_begin, kb0 = kb_begin;
        for (int64_t left = n_units; left > 0 && ok; ++t, kb0 = 0) {
            const int kb_end = static_cast<int>(min(static_cast<int64_t>(KB), kb0 + left));
            left -= kb_end - kb0;
            for (int kb = kb0; kb < kb_end; kb += KPS) {
                const int nk = min(KPS, kb_end - kb);
                if (!first_lap && !wait_bounded(&empty[stage], phase ^ 1u, ctl)) { ok = false; break; }
                if (skip) {
                    skip = false;   // leave this stage unloaded
                } else {
                    mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(nk) * kb_bytes);
#pragma unroll
                    for (int i = 0; i < KPS; ++i) {
                        if (i < nk) {
                            tma_load_2d(sW + stage * C::kStageW + i * kWBytes, &tmap_w, &full[stage],
                                        (kb + i) * kBK, t * p.tile_rows);
                            tma_load_2d(sX + stage * C::kStageX + i * kXBytes, &tmap_x, &full[stage],
                                        (kb + i) * kBK, 0);
                        }
                    }
                    issued_mask |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                }
                if (++stage == kStages) { stage = 0; phase ^= 1u; first_lap = false; }
            }
        }
        // Let every issued copy land before the CTA exits (immediate after a
        // normal run; after an abort, copies still in flight finish).
        for (int s = 0; s < kStages; ++s)
            if (issued_mask & (1u << s))
                wait_bounded(&full[s], (issued_phase >> s) & 1u, ctl, false);
    } else if (warp == 1 && lane == 0) {
        // ------------------------------------------------ MMA issuer
        int stage = 0;
        uint32_t phase = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        bool issued_any = false;
        int kb0 = kb_begin;
        for (int64_t left = n_units; left > 0 && ok; kb0 = 0) {
            const int kb_end = static_cast<int>(min(static_cast<int64_t>(KB), kb0 + left));
            left -= kb_end - kb0;
            if (!wait_bounded(&acc_empty[acc], acc_phase ^ 1u, ctl)) break;
            tc_fence_after_sync();
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * NC);
            for (int kb = kb0; kb < kb_end; kb += KPS) {
                const int nk = min(KPS, kb_end - kb);
                if (!wait_bounded(&full[stage], phase, ctl)) { ok = false; break; }
                tc_fence_after_sync();
#pragma unroll
                for (int i = 0; i < KPS; ++i) {
                    if (i < nk) {
                        const uint32_t a0 = smem_addr(sW + stage * C::kStageW + i * kWBytes);
                        const uint32_t b0 = smem_addr(sX + stage * C::kStageX + i * kXBytes);
#pragma unroll
                        for (int kk = 0; kk < kBKBytes / 32; ++kk) {
                            const uint64_t ad = sdesc_k_major_sw128(a0 + kk * 32);
                            const uint64_t bd = sdesc_k_major_sw128(b0 + kk * 32);
                            const uint32_t accum = (kb > kb0 || i > 0 || kk > 0) ? 1u : 0u;
                            if constexpr (kFp16In)
                                mma_f16(d_tmem, ad, bd, C::kIdesc, accum);
                            else
                                mma_f8f6f4(d_tmem, ad, bd, C::kIdesc, accum);
                        }
                    }
                }
                issued_any = true;
                mma_commit(&empty[stage]);
                if (++stage == kStages) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            mma_commit(&acc_full[acc]);
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
        if (issued_any) {
            mma_commit(drain);
            wait_bounded(drain, 0, ctl, false);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------ epilogue
        // Thread (q, lane) owns row r = 32 q + lane of each tile (its tensor-
        // memory lane) and that row's 16 accumulator columns, one per row of A.
        const int q = warp & 3;
        const int r = q * 32 + lane;
        const int me = static_cast<int>(blockIdx.x);
        float ab = 1.0f;   // (a fused epilogue has scales of its own)
        if (!kFused && p.sa != nullptr) ab = p.sa[0] * p.sb[0];
        const float alpha = !kFused && p.out_kind == kOutE4M3 ? __fdiv_rn(ab, p.sd[0]) : ab;
        ByScale out{1.0f, 1.0f};
        FusedColumn column;
        if constexpr (kFused) {
            out = output_scale(p.out_kind, p.sd);
            if (r < NC) {
                const ScaleParts row = scale_parts(p.sa != nullptr && r < p.M ? ld_float(p.sa + r * p.epi.sa_step) : 1.0f);
                row_scales[r] = row.rest;
                row_scales[NC + r] = row.whole;
            }
            named_bar_sync(kEpiBar, kEpiThreads);   // (the helpers' reads come after a hand-off)
        }
        uint32_t amax_bits = 0u;
        bool released = false;   // the last tile handed to warps 0-3 (thread 128)
        int acc = 0;
        uint32_t acc_phase = 0;
        int t = t_begin, kb0 = kb_begin;
        for (int64_t left = n_units; left > 0; ++t, kb0 = 0) {
            const int kb_end = static_cast<int>(min(static_cast<int64_t>(KB), kb0 + left));
            left -= kb_end - kb0;
            // Which CTAs share tile t, and their slots (before the wait).
            const int64_t tile_u0 = static_cast<int64_t>(t) * KB;
            const int c_first = cta_of_unit(tile_u0, G, units);
            const int c_last = cta_of_unit(tile_u0 + KB - 1, G, units);
            const int first_slot =
                range_start(c_first, G, units) == tile_u0 ? 2 * c_first : 2 * c_first + 1;
            if constexpr (kFused) {
                const int n0 = t * p.tile_rows + r;
                column = fused_column(p, r < p.tile_rows && n0 < p.N, n0);
                if (p.epi.residual != nullptr) {
                    if (t != t_begin) named_bar_sync(kEpiBar, kEpiThreads);   // the last tile's has been read
                    stage_residual(p, residual_tile, t, r);
                }
            }
            // The four warps continue or leave together (named barriers below).
            const bool got = wait_bounded(&acc_full[acc], acc_phase, ctl);
            if constexpr (kFused) asm volatile("cp.async.wait_all;" ::: "memory");
            if (!named_bar_and(kEpiBar, kEpiThreads, got)) break;
            tc_fence_after_sync();
            // Columns [c0, c0 + 16) of this row's accumulator, 16 at a time;
            // only chunks that hold rows of A (c0 < M) are read.
            const uint32_t tacc = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                  static_cast<uint32_t>(acc * NC);
            const int n = t * p.tile_rows + r;
            float first[16];   // chunk 0, kept from the partial pass
            bool finish = true;
            int my_slot = 0;
            if (c_last > c_first) {
                // Split tile: publish this partial, count the arrival.
                my_slot = me == c_first ? first_slot : 2 * me;
                float4* ws = reinterpret_cast<float4*>(p.partials) +
                             static_cast<int64_t>(my_slot) * (NC / 4) * kRows;
#pragma unroll 1
                for (int c0 = 0; c0 < NC && c0 < p.M; c0 += 16) {
                    uint32_t raw[16];
                    __syncwarp();
                    tmem_load_16cols(tacc + static_cast<uint32_t>(c0), raw);
                    tmem_load_wait(raw);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (c0 == 0) first[j] = __uint_as_float(raw[j]);
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        if (c0 + 4 * g < p.M)
                            __stcg(ws + ((c0 >> 2) + g) * kRows + r,
                                   make_float4(__uint_as_float(raw[4 * g]), __uint_as_float(raw[4 * g + 1]),
                                               __uint_as_float(raw[4 * g + 2]),
                                               __uint_as_float(raw[4 * g + 3])));
                    }
                }
                named_bar_sync(kEpiBar, kEpiThreads);
                if (threadIdx.x == 4 * 32) {
                    const uint32_t old = atom_add_acq_rel_gpu(&p.counts[t], 1u);
                    const bool last = old == static_cast<uint32_t>(c_last - c_first);
                    if (last) atomicExch(&p.counts[t], 0u);   // zero for the next launch
                    *last_flag = last ? 1 : 0;
                }
                named_bar_sync(kEpiBar, kEpiThreads);
                finish = *last_flag != 0;
            }
            // When this is the CTA's last segment its ring of K blocks is idle:
            // one thread bulk-copies every other segment's partial tile into
            // it on one barrier, and the sum below reads shared memory instead
            // of making L2 round trips for each 16 columns and each four
            // segments.  At NC = 16 with at most three other segments (one
            // chunk, one group of direct loads) the loads measured as fast.
            const int others = c_last - c_first;
            const int quads = (min(p.M, NC) + 3) >> 2;   // column quads that hold rows of A
            const uint32_t slot_bytes = static_cast<uint32_t>(quads) * kRows * 16u;
            const bool staged = (NC >= 32 || others >= 4) && finish && others > 0 && left == 0 &&
                                static_cast<int64_t>(others + 1) * slot_bytes <=
                                    static_cast<int64_t>(kRingKBlocks) * kKBBytes;
            if (staged) {
                if (threadIdx.x == 4 * 32) {
                    // the partials were published through the generic proxy
                    // and acquired by this thread's arrival atomic
                    fence_proxy_async_global();
                    mbar_arrive_expect_tx(fix_bar, static_cast<uint32_t>(others) * slot_bytes);
                    // segment c goes to position c - c_first; the own position
                    // is filled from tensor memory below
                    for (int c = c_first; c <= c_last; ++c) {
                        if (c == me) continue;
                        const int slot = c == c_first ? first_slot : 2 * c;
                        bulk_load_g2s(smem + static_cast<uint32_t>(c - c_first) * slot_bytes,
                                      reinterpret_cast<const float4*>(p.partials) +
                                          static_cast<int64_t>(slot) * (NC / 4) * kRows,
                                      slot_bytes, fix_bar);
                    }
                }
                const bool landed = wait_bounded(fix_bar, 0, ctl);
                if (!named_bar_and(kEpiBar, kEpiThreads, landed)) {
                    // let the copies land before the CTA's shared memory is released
                    if (threadIdx.x == 4 * 32) wait_bounded(fix_bar, 0, ctl, false);
                    break;
                }
            }
            // The CTA's last tile: with more than one chunk, warps 0-3 (idle
            // by now, each reading the same tensor-memory lanes as its twin
            // among warps 4-7) take the odd chunks.  The hand-off is an
            // mbarrier with bounded waits, released on every exit path.
            const bool helped = NC >= 32 && finish && left == 0;
            if (left == 0 && threadIdx.x == 4 * 32) {
                help[1] = t;
                help[2] = acc;
                help[3] = c_first;
                help[4] = c_last;
                help[5] = first_slot;
                help[6] = staged ? 1 : 0;
                help[0] = helped ? 1 : 0;
                mbar_arrive(help_bar);
                released = true;
            }
            if (finish)
                finish_chunks<NC, kFused>(p, smem, tacc, r, n, 0, helped ? 32 : 16, me, c_first, c_last,
                                  first_slot, staged, quads, first, alpha, amax_bits, column, out, row_scales, residual_tile);
            // The accumulator is free once every chunk has been read.
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
            (void)my_slot;
        }
        // Every exit (including a timed-out wait) releases warps 0-3.
        if (threadIdx.x == 4 * 32 && !released) {
            help[0] = 0;
            mbar_arrive(help_bar);
        }
        // max |sa*sb*acc| of this warp's stored outputs (monotone rounding:
        // fl(max|acc| * c) is the exact maximum of fl(|acc| * c)).
        if (p.amax_out != nullptr) {
            __syncwarp();
            const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, amax_bits);
            if (lane == 0 && bits != 0u)
                atomicMax(p.amax_out, __float_as_uint(__uint_as_float(bits) * ab) & 0x7FFFFFFFu);
        }
    }
    if constexpr (NC >= 32) {
        if (warp < 4) {
            // ------------------------------------------------ helpers
            // Warps 0-3, once their own roles are done, take the odd
            // 16-column chunks of the CTA's last tile when it finishes one.
            __syncwarp();
            ByScale out{1.0f, 1.0f};
            FusedColumn column;
            if constexpr (kFused) {   // of the CTA's last tile
                const int t_last = static_cast<int>((u_begin + n_units - 1) / KB), n = t_last * p.tile_rows + warp * 32 + lane;
                out = output_scale(p.out_kind, p.sd);
                column = fused_column(p, warp * 32 + lane < p.tile_rows && n < p.N, n);
            }
            const bool go = wait_bounded(help_bar, 0, ctl) && help[0] != 0;
            if (__all_sync(0xFFFFFFFFu, go)) {
                const int t = help[1], acc = help[2], c_first = help[3], c_last = help[4];
                const int first_slot = help[5];
                const bool staged = help[6] != 0;
                tc_fence_after_sync();
                const bool landed = !staged || wait_bounded(fix_bar, 0, ctl);
                if (__all_sync(0xFFFFFFFFu, landed)) {
                    const int q = warp;   // the same tensor-memory lanes as warp q + 4
                    const int r = q * 32 + lane;
                    const uint32_t tacc = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                          static_cast<uint32_t>(acc * NC);
                    float ab = 1.0f;   // (a fused epilogue has scales of its own)
                    if (!kFused && p.sa != nullptr) ab = p.sa[0] * p.sb[0];
                    const float alpha = !kFused && p.out_kind == kOutE4M3 ? __fdiv_rn(ab, p.sd[0]) : ab;
                    const int quads = (min(p.M, NC) + 3) >> 2;
                    const float none[16] = {};   // chunk 0 is not among the odd ones
                    uint32_t amax_bits = 0u;
                    finish_chunks<NC, kFused>(p, smem, tacc, r, t * p.tile_rows + r, 16, 32,
                                      static_cast<int>(blockIdx.x), c_first, c_last, first_slot,
                                      staged, quads, none, alpha, amax_bits, column, out, row_scales, residual_tile);
                    if (p.amax_out != nullptr) {
                        __syncwarp();
                        const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, amax_bits);
                        if (lane == 0 && bits != 0u)
                            atomicMax(p.amax_out,
                                      __float_as_uint(__uint_as_float(bits) * ab) & 0x7FFFFFFFu);
                    }
                }
            }
        }
    }

    // Warps whose lane 0 ran a role alone may arrive diverged: the barrier
    // before tensor memory is freed is the non-aligned one.
    tc_fence_before_sync();
    cta_sync_diverged();
    tc_fence_after_sync();
    if (warp == 2) tmem_dealloc<C::kTmemCols>(tmem_base);
}

// ------------------------------------------------------------- host side

// B boxes each CTA prefetches into L2 before its dependency wait:
// DG_SPLITK_PREFETCH=n (sweeps, 0..256), default one ring.
int splitk_prefetch_kblocks(int ring) {
    const int n = knobs().splitk_prefetch;
    return n >= 0 ? n : ring;
}

template <bool kFp16In, int KPS, int NC, bool kFused>
cudaError_t launch_sk(const TcLaunch& L, float* partials, uint32_t* counts, cudaStream_t s) {
    using C = SkCfg<NC, KPS>;
    static std::mutex mu;
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        if (!attr_done[dev]) {
            e = cudaFuncSetAttribute(gemm_skinny_kernel<kFp16In, KPS, NC, kFused>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kFused ? C::kFusedSmemBytes : C::kSmemBytes);
            if (e != cudaSuccess) return e;
            attr_done[dev] = true;
        }
    }
    CUtensorMap tw, tx;
    const int tile_rows = L.plan->block_n;
    if (!make_map(&tw, L.B, L.N, L.K, kFp16In, tile_rows) ||
        !make_map(&tx, L.A, L.M, L.K, kFp16In, NC))
        return cudaErrorInvalidValue;
    SkParams prm;
    prm.D = L.D;
    prm.M = L.M;
    prm.N = L.N;
    prm.K = L.K;
    prm.sa = L.sa;
    prm.sb = L.sb;
    prm.sd = L.sd;
    prm.out_kind = L.out_kind;
    prm.status = L.status;
    prm.timeout_ns = wait_timeout_ns();
    prm.skip_first_load = take_skip_first_load() ? 1 : 0;
    prm.amax_out = L.amax_out;
    prm.partials = partials;
    prm.counts = counts;
    prm.tiles = L.plan->tiles;
    prm.tile_rows = tile_rows;
    const int bk = kFp16In ? 64 : 128;
    prm.kblocks = (L.K + bk - 1) / bk;
    prm.prefetch_kblocks = splitk_prefetch_kblocks(C::kRing);
    if (L.epi != nullptr) prm.epi = *L.epi;
    return launch_kernel(gemm_skinny_kernel<kFp16In, KPS, NC, kFused>, dim3(L.plan->grid), dim3(kThreads),
                         kFused ? C::kFusedSmemBytes : C::kSmemBytes, s, tw, tx, prm);
}

// K blocks per stage: DG_SPLITK_KPS=1|2 (sweeps), default 2.
int splitk_kps() { return knobs().splitk_kps; }

// MMA N for M rows of A: M rounded up to 16, 32, 64 or 128.
int nc_for(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

int smem_for_nc(int nc) {
    switch (nc) {
        case 16: return SkCfg<16, 2>::kSmemBytes;
        case 32: return SkCfg<32, 2>::kSmemBytes;
        case 64: return SkCfg<64, 2>::kSmemBytes;
        default: return SkCfg<128, 2>::kSmemBytes;
    }
}

template <bool kFp16In, int NC, bool kFused>
cudaError_t launch_nc(const TcLaunch& L, float* partials, uint32_t* counts, cudaStream_t s) {
    if (SkCfg<NC, 1>::kRing == L.plan->stages)
        return launch_sk<kFp16In, 1, NC, kFused>(L, partials, counts, s);
    return launch_sk<kFp16In, 2, NC, kFused>(L, partials, counts, s);
}

template <bool kFp16In, bool kFused>
cudaError_t launch_in(const TcLaunch& L, float* partials, uint32_t* counts, cudaStream_t s) {
    switch (nc_for(L.M)) {
        case 16: return launch_nc<kFp16In, 16, kFused>(L, partials, counts, s);
        case 32: return launch_nc<kFp16In, 32, kFused>(L, partials, counts, s);
        case 64: return launch_nc<kFp16In, 64, kFused>(L, partials, counts, s);
        default: return launch_nc<kFp16In, 128, kFused>(L, partials, counts, s);
    }
}

}  // namespace
}  // namespace dg
