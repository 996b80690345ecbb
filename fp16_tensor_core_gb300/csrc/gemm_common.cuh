// gemm_common.cuh -- pieces shared by the single-CTA and CTA-pair
// tensor-core GEMM kernels: launch parameters, tile raster, the fused
// scale/convert epilogue store and TMA tensor-map creation.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "activation.cuh"
#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "gemm_smem.h"

namespace dg {

struct Params {
    void* D;
    int M, N, K;
    const float* sa;
    const float* sb;
    const float* sd;
    int out_kind;
    int out_elem;
    int vec_ok;
    uint32_t* status;
    uint64_t timeout_ns;
    int skip_first_load;
    int group_m;   // tiles are rastered in groups of group_m M-tiles sweeping N
    uint32_t* amax_out;  // optional: running max |sa*sb*acc| as float bits
    // Grouped GEMM: group g covers rows [group_off[g], group_off[g+1]) of A
    // and D and rows [g*N, g*N + N) of B; sa/sb/sd hold one scale per group.
    const int* group_off;
    int groups;
    int early_release;   // release the next kernel once every CTA is on its last tile
    int staged;          // epilogue through staging boxes and bulk tensor stores (tmap_d)
    // CTA-pair kernel, split tail: the tiles left after the last full wave
    // are cut into tail_split K ranges (>= 2; 1 = no split), one per pair.
    int tail_split;
    float* tail_ws;         // partial tiles: [slot][2 CTAs][BN / 4][128] float4
    uint32_t* tail_counts;  // per tail tile and CTA: arrivals of the later parts
    // Single-CTA kernel: bytes of one A box and one B box (128 and BN rows
    // x 128 bytes), and of the shorter boxes of the edge tiles: tiles whose
    // A rows start at a_edge_row or later (B rows at b_edge_row or later)
    // load through the edge maps, boxes of the rows left rounded up to 8
    // (INT_MAX: no edge).  The MMA still reads 128 and BN rows; the rows
    // past a box only reach output rows past M or columns past N, which are
    // not stored.
    int a_box_bytes;
    int b_box_bytes;
    int a_edge_bytes;
    int b_edge_bytes;
    int a_edge_row;
    int b_edge_row;
    Epilogue epi;   // of the fused kernels only
};

constexpr int kMaxGroups = 1024;

// CTA-pair kernel (k_gemm_tc2.cu): shared memory and stage count of the
// 256 x bn pair tile, and its launcher.
int pair_smem_for(int bn, int kps);   // kps: K blocks per stage (1 or 2)
int pair_stages(int bn, int kps);
cudaError_t launch_gemm_tc_pair(const TcLaunch& L, const Params& prm, cudaStream_t s);
// The same kernels with a fused epilogue (L.epi).
cudaError_t launch_gemm_tc_pair_fused(const TcLaunch& L, const Params& prm, cudaStream_t s);
cudaError_t launch_gemm_tc_fused(const TcLaunch& L, const Params& prm, cudaStream_t s);

namespace {

constexpr int kThreads = 256;   // warps: 0 TMA, 1 MMA, 2 TMEM owner, 3 idle, 4-7 epilogue
constexpr int gemm_threads(bool fused) { return 128 + 32 * epilogue_warps(fused); }

constexpr uint32_t pow2_at_least(uint32_t v) {
    uint32_t p = 32;
    while (p < v) p <<= 1;
    return p;
}

__device__ __forceinline__ void tile_coords(int t, int num_m, int num_n, int group_m, int& mt,
                                            int& nt) {
    const int group = group_m * num_n;
    const int g = t / group;
    const int first_m = g * group_m;
    const int gm = min(num_m - first_m, group_m);
    const int r = t - g * group;
    mt = first_m + r % gm;
    nt = r / gm;
}

__device__ __forceinline__ void st_global_v4(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};"
                 :: "l"(p), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Convert and store 32 consecutive output columns of one row, `ncols` (at
// most 32) of them inside D.
__device__ __forceinline__ void store_values(const Params& p, int row, int ncols, int col0,
                                             const float (&v)[32]) {
    const int64_t off = static_cast<int64_t>(row) * p.N + col0;
    if (p.out_kind == kOutE4M3) {
        uint8_t* dst = static_cast<uint8_t*>(p.D) + off;
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = static_cast<uint32_t>(f32x2_to_e4m3x2(v[4 * j], v[4 * j + 1])) |
                   (static_cast<uint32_t>(f32x2_to_e4m3x2(v[4 * j + 2], v[4 * j + 3])) << 16);
        if (ncols == 32 && p.vec_ok) {
            st_global_v4(dst, w[0], w[1], w[2], w[3]);
            st_global_v4(dst + 16, w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < ncols) dst[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
        }
    } else {
        uint16_t* dst = static_cast<uint16_t*>(p.D) + off;
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            w[j] = p.out_kind == kOutFP16 ? f32x2_to_f16x2(v[2 * j], v[2 * j + 1])
                                          : f32x2_to_bf16x2(v[2 * j], v[2 * j + 1]);
        if (ncols == 32 && p.vec_ok) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                st_global_v4(dst + 8 * j, w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < ncols) dst[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// Scale, convert and store 32 consecutive accumulator columns of one row.
// Returns max |acc| over the stored elements as ordered bits (the bit
// pattern of a non-negative float; NaN above every number), 0 if none.
__device__ __forceinline__ uint32_t store_chunk(const Params& p, int row, int row_end, int col0,
                                                const uint32_t (&r)[32], float alpha) {
    if (row >= row_end) return 0u;
    const int ncols = min(32, p.N - col0);
    if (ncols <= 0) return 0u;
    uint32_t amax_bits = 0u;
    if (p.amax_out != nullptr) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < ncols) amax_bits = max(amax_bits, r[i] & 0x7FFFFFFFu);
    }
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * alpha;
    store_values(p, row, ncols, col0, v);
    return amax_bits;
}

// Staged epilogue: each epilogue warp converts 32 rows x 32 columns of the
// accumulator into a box in shared memory laid out as the output tensor map
// expects (64-byte swizzle for 2-byte outputs, 32-byte for E4M3) and writes
// it with one bulk tensor store, which moves whole lines and clips rows >= M
// and columns >= N.

// Thread `lane` converts one row's 32 values into its line of `box`.
__device__ __forceinline__ void stage_values(const Params& p, uint8_t* box, const float (&v)[32],
                                             int lane) {
    if (p.out_kind == kOutE4M3) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = static_cast<uint32_t>(f32x2_to_e4m3x2(v[4 * j], v[4 * j + 1])) |
                   (static_cast<uint32_t>(f32x2_to_e4m3x2(v[4 * j + 2], v[4 * j + 3])) << 16);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int ph = k ^ ((lane >> 2) & 1);   // 32-byte swizzle: 16-byte halves
            st_shared_v4(smem_addr(box + lane * 32 + ph * 16), w[4 * k], w[4 * k + 1], w[4 * k + 2],
                         w[4 * k + 3]);
        }
    } else {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            w[j] = p.out_kind == kOutFP16 ? f32x2_to_f16x2(v[2 * j], v[2 * j + 1])
                                          : f32x2_to_bf16x2(v[2 * j], v[2 * j + 1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int ph = k ^ ((lane >> 1) & 3);   // 64-byte swizzle: 16-byte quarters
            st_shared_v4(smem_addr(box + lane * 64 + ph * 16), w[4 * k], w[4 * k + 1], w[4 * k + 2],
                         w[4 * k + 3]);
        }
    }
}

// Thread `lane` converts accumulator row `row`, columns col0 .. col0 + 31,
// into its line of `box`.  Returns max |acc| over the columns < N of a row
// < row_end (ordered bits) when p.amax_out is set, else 0.
__device__ __forceinline__ uint32_t stage_box(const Params& p, uint8_t* box, int row, int row_end,
                                              int col0, const uint32_t (&r)[32], float alpha,
                                              int lane) {
    uint32_t amax_bits = 0u;
    if (p.amax_out != nullptr && row < row_end) {
        const int ncols = min(32, p.N - col0);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < ncols) amax_bits = max(amax_bits, r[i] & 0x7FFFFFFFu);
    }
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * alpha;
    stage_values(p, box, v, lane);
    return amax_bits;
}

// ---- the fused epilogue: act(scale_a[m] scale_b[n] acc + bias[n]) + residual[m, n]

// 32 elements of one row of the residual, 16 bits each (zeros past column N
// and without a residual); N a multiple of 8.  Not the read-only path: D may
// be the residual, each element read by the warp that later writes it.
__device__ __forceinline__ void load_residual(const Params& p, int row, bool row_ok, int col0,
                                              uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 0u;
    if (p.epi.residual == nullptr || !row_ok || col0 >= p.N) return;
    const uint16_t* src = p.epi.residual + static_cast<int64_t>(row) * p.N + col0;
    if (col0 + 32 <= p.N) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                         : "l"(src + 8 * i));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col0 + 8 * i < p.N)
                asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                             : "l"(src + 8 * i));
    }
}

// Rows that are not whole 16-byte pieces: a warp's 32 x 32 elements pass
// through its staging box, so that each access to memory is 32 neighbours of
// one row and not 32 rows (200 x 1001 x 1040 E4M3 13.3 -> 6.9 us).  A row's
// words lie permuted by its number: neither side meets a bank twice.
__device__ __forceinline__ uint32_t* box_word(uint8_t* box, int row, int words, int at) {
    return reinterpret_cast<uint32_t*>(box) + row * words + (at ^ (row & (words - 1)));
}

__device__ __forceinline__ void load_residual_odd(const Params& p, uint8_t* box, int row0, int row_end, int col0,
                                                  int lane, uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 0u;
    if (p.epi.residual == nullptr || col0 >= p.N) return;   // the whole warp
    const uint16_t* src = p.epi.residual + static_cast<int64_t>(row0) * p.N + col0 + lane;
    __syncwarp();   // the box's last use
#pragma unroll 1   // (code that is not there does not have to be fetched)
    for (int i0 = 0; i0 < 32; i0 += 16) {
        uint32_t e[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            e[i] = 0u;
            if (row0 + i0 + i < row_end && col0 + lane < p.N)
                asm volatile("ld.global.u16 %0, [%1];" : "=r"(e[i]) : "l"(src + static_cast<int64_t>(i0 + i) * p.N));
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
            reinterpret_cast<uint16_t*>(box_word(box, i0 + i, 16, lane >> 1))[lane & 1] = static_cast<uint16_t>(e[i]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = *box_word(box, lane, 16, i);
    __syncwarp();
}

// Converts and stores a warp's 32 rows of 32 columns, thread `lane` the
// values v of row row0 + lane.
__device__ __forceinline__ void store_box_odd(const Params& p, uint8_t* box, int row0, int row_end, int col0,
                                              const float (&v)[32], int lane) {
    if (col0 >= p.N) return;   // the whole warp
    const int64_t at = static_cast<int64_t>(row0) * p.N + col0 + lane;
    const bool inside = col0 + lane < p.N;
    if (p.out_kind == kOutE4M3) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *box_word(box, lane, 8, i) = static_cast<uint32_t>(f32x2_to_e4m3x2(v[4 * i], v[4 * i + 1])) |
                                         static_cast<uint32_t>(f32x2_to_e4m3x2(v[4 * i + 2], v[4 * i + 3])) << 16;
        __syncwarp();
        uint8_t* dst = static_cast<uint8_t*>(p.D) + at;
#pragma unroll 4
        for (int i = 0; i < 32; ++i)
            if (inside && row0 + i < row_end)
                dst[static_cast<int64_t>(i) * p.N] = reinterpret_cast<uint8_t*>(box_word(box, i, 8, lane >> 2))[lane & 3];
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            *box_word(box, lane, 16, i) = p.out_kind == kOutFP16 ? f32x2_to_f16x2(v[2 * i], v[2 * i + 1])
                                                                 : f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]);
        __syncwarp();
        uint16_t* dst = static_cast<uint16_t*>(p.D) + at;
#pragma unroll 4
        for (int i = 0; i < 32; ++i)
            if (inside && row0 + i < row_end)
                dst[static_cast<int64_t>(i) * p.N] = reinterpret_cast<uint16_t*>(box_word(box, i, 16, lane >> 1))[lane & 1];
    }
    __syncwarp();   // before the box is written again
}

// The columns' scales of B and biases (laid out as kColumnFloats says) into
// shared memory while the main loop runs, zeros past N: chunks first, first +
// 2, ... of the tile whose columns start at col0.  What is kept of a scale is
// its rest (scale_parts); returns whether any column's scale is more than that.
template <int BN>
__device__ __forceinline__ bool stage_columns(const Params& p, float* columns, int col0, int first, int lane) {
    bool parts = false;
    constexpr int kChunks = fused_chunks(BN);
    float s[kChunks], b[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int n = col0 + 32 * (first + 2 * i) + lane;
        s[i] = p.sb == nullptr ? 1.0f : 0.0f;
        b[i] = 0.0f;
        if (n < p.N && p.sb != nullptr) {
            const float sb = ld_float(p.sb + static_cast<int64_t>(n) * p.epi.sb_step);
            s[i] = scale_parts(sb).rest;
            parts |= !scale_is_rest(sb);
        }
        if (n < p.N && p.epi.bias != nullptr) b[i] = ld_float(p.epi.bias + n);
    }
    __syncwarp();   // every lane has read the last tile's
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int at = kColumnFloats * i + 2 * (lane & ~1) + (lane & 1);
        columns[at] = s[i];
        columns[at + 2] = b[i];
    }
    __syncwarp();
    return __any_sync(0xFFFFFFFFu, parts);
}

// Multiplies 32 accumulator columns by what stage_columns left out of their
// scales.
__device__ __forceinline__ void apply_wholes(const Params& p, int col0, int lane, uint32_t (&r)[32]) {
    const int n = col0 + lane;
    const float s = n < p.N && p.sb != nullptr ? ld_float(p.sb + static_cast<int64_t>(n) * p.epi.sb_step) : 1.0f;
    const float column = scale_parts(s).whole;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        r[i] = __float_as_uint(__uint_as_float(r[i]) * __shfl_sync(0xFFFFFFFFu, column, i));
}

// The same of a warp's chunks of a tile (first, first + 2, ...), in tensor
// memory, before its epilogue: there a branch at every chunk took 1 us more
// of 4096 x 4096 x 4096 E4M3's 49.
template <int BN>
__device__ __forceinline__ void apply_wholes_to_tile(const Params& p, uint32_t taddr, int col0, int first, int lane) {
#pragma unroll 1
    for (int c = first; c < BN / 32; c += 2) {
        uint32_t r[32];
        __syncwarp();
        tmem_load_32cols(taddr + c * 32, r);
        tmem_load_wait(r);
        apply_wholes(p, col0 + c * 32, lane, r);
        tmem_store_32cols(taddr + c * 32, r);
    }
    tmem_store_wait();
}

// Moves a tile row's residual (this warp's lines of 64 columns: the first half
// or the second) into L2.
template <int BN>
__device__ __forceinline__ void prefetch_residual(const Params& p, int row, bool row_ok, int col0, int half) {
    if (p.epi.residual == nullptr || !row_ok) return;
    const uint16_t* src = p.epi.residual + static_cast<int64_t>(row) * p.N + col0;
#pragma unroll
    for (int i = 0; i < BN; i += 128)
        if (i + 64 * half < BN && col0 + i + 64 * half < p.N)
            asm volatile("prefetch.global.L2 [%0];" :: "l"(src + i + 64 * half));
}

// The values of 32 accumulator columns of one row; sa: the row's scale in its
// parts, columns: the rests of theirs (stage_columns).  Returns their largest magnitude inside D
// (ordered bits) when it is wanted, before the division by the output's scale.
__device__ __forceinline__ uint32_t fuse32(const Params& p, bool row_ok, int col0, const uint32_t (&r)[32],
                                           const uint32_t (&res)[16], ScaleParts sa, const float* columns, ByScale out,
                                           float (&f)[32]) {
    pair v[16];
    const pair row_scale = pair_of(sa.rest), row_whole = pair_of(sa.whole);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const ulonglong2 c = reinterpret_cast<const ulonglong2*>(columns)[i];
        const pair acc = pair_mul(pair_of(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), row_whole);
        v[i] = pair_fma(acc, pair_mul(row_scale, c.x), c.y);
    }
    with_activation(p.epi.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = activation(act.value, v[i]);
    });
    if (p.epi.residual != nullptr) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float2 x;
            if (p.epi.residual_fp16 != 0)
                x = f16x2_to_f32x2(res[i]);
            else
                x = make_float2(__uint_as_float(res[i] << 16), __uint_as_float(res[i] & 0xFFFF0000u));
            v[i] = pair_add(v[i], pair_of(x.x, x.y));
        }
    }
    float top = 0.0f;
    if (p.amax_out != nullptr && row_ok) {
        if (col0 + 32 <= p.N) {
#pragma unroll
            for (int i = 0; i < 16; ++i) top = pair_top(v[i], top);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 x = floats_of(v[i]);
                if (col0 + 2 * i < p.N) top = pair_top(pair_of(x.x), top);
                if (col0 + 2 * i + 1 < p.N) top = pair_top(pair_of(x.y), top);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (p.out_kind == kOutE4M3) v[i] = pair_mul(pair_mul(v[i], pair_of(out.pre)), pair_of(out.inv));
        const float2 x = floats_of(v[i]);
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
    return __float_as_uint(top);
}

// A row's scale of A (1 without scales, and for rows outside).
__device__ __forceinline__ float scale_of_row(const Params& p, int row, bool row_ok) {
    return p.sa == nullptr || !row_ok ? 1.0f : ld_float(p.sa + static_cast<int64_t>(row) * p.epi.sa_step);
}

__device__ __forceinline__ ByScale output_scale(int out_kind, const float* sd) {
    return out_kind == kOutE4M3 ? by_scale(ld_float(sd)) : ByScale{1.0f, 1.0f};
}

// The fused kernels' maximum, one warp's: already of the values themselves.
__device__ __forceinline__ void publish_top(uint32_t* amax_out, uint32_t top) {
    if (amax_out == nullptr) return;
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0 && top != 0u) atomicMax(amax_out, top);
}

// Waits until every bulk store this thread committed has finished reading
// shared memory (the staging box may then be rewritten).
__device__ __forceinline__ void bulk_wait_read_all() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// The output tensor map of the staged epilogue: D (M x N of the output
// type), 32 x 32 boxes, swizzled to the width of one box line.  False if the
// rows of D are not 16-byte multiples (then the epilogue stores directly).
inline bool make_out_map(CUtensorMap* map, const TcLaunch& L);

// Publishes one warp's running max |acc| (ordered bits) as
// max |acc| * (sa * sb) into p.amax_out.  Rounding is monotone, so
// fl(max|acc| * c) = max fl(|acc| * c) exactly.  Whole warp, converged.
__device__ __forceinline__ void publish_amax(const Params& p, uint32_t amax_bits) {
    if (p.amax_out == nullptr) return;
    amax_bits = __reduce_max_sync(0xFFFFFFFFu, amax_bits);
    if ((threadIdx.x & 31) == 0 && amax_bits != 0u) {
        float ab = 1.0f;
        if (p.sa != nullptr) ab = (*p.sa) * (*p.sb);
        const float v = __uint_as_float(amax_bits) * ab;
        atomicMax(p.amax_out, __float_as_uint(v) & 0x7FFFFFFFu);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// 2-D map over a rows x k row-major matrix, box = box_rows x 128 bytes,
// 128-byte swizzle, zero fill outside the matrix.
bool make_map(CUtensorMap* map, const void* base, int rows, int k, bool fp16, int box_rows) {
    auto encode = get_encode_fn();
    if (!encode) return false;
    const int elem = fp16 ? 2 : 1;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(k) * elem};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(kBKBytes / elem), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = encode(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                              2, const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

inline bool make_out_map(CUtensorMap* map, const TcLaunch& L) {
    if ((static_cast<int64_t>(L.N) * L.out_elem) % 16 != 0) return false;
    auto encode = get_encode_fn();
    if (!encode) return false;
    const bool e4 = L.out_kind == kOutE4M3;
    const CUtensorMapDataType dt = e4 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                  : (L.out_kind == kOutFP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(L.N), static_cast<cuuint64_t>(L.M)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(L.N) * L.out_elem};
    cuuint32_t box[2] = {32, 32};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, dt, 2, L.D, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  e4 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace dg
