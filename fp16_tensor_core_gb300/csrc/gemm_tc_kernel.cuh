// gemm_tc_kernel.cuh -- the single-CTA tensor-core kernel that k_gemm_tc.cu
// describes, as a template: k_gemm_tc.cu holds the plain and grouped forms,
// k_gemm_tc_fused.cu those with a fused epilogue (kFused: row and column
// scales, bias, activation, residual in place of one scale).
#pragma once

#include <algorithm>
#include <climits>
#include <mutex>

#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "gemm_common.cuh"

namespace dg {
namespace {

constexpr int kBM = 128;

// Shared memory for the grouped variant's per-group tile prefix.
constexpr int kGroupSmem = 4 * (kMaxGroups + 1) + 12;

// Staging boxes of the epilogue: one 32 x 32 box per epilogue warp.
constexpr int staging_bytes(bool fused) { return epilogue_warps(fused) * kBoxBytes; }

// Stage count = what fits in 227 KB beside the barrier block (1 KB, keeping
// the staging boxes 1024-byte aligned), the staging boxes, the grouped
// variant's tile prefix and the fused one's columns, at most 8 (4 with two K blocks per stage).
constexpr int stages_for(int bn, bool grouped = false, int kps = 1, bool fused = false) {
    const int st = (kSmemLimit - 1024 - 1024 - staging_bytes(fused) - (grouped ? kGroupSmem : 0) -
                    (fused ? columns_bytes(bn) : 0)) /
                   (kps * (kBM * kBKBytes + bn * kBKBytes));
    return st > 8 / kps ? 8 / kps : st;
}

// KPS: K blocks per pipeline stage (1, or 2: each stage holds two adjacent
// 128-byte K blocks of every row, so a row's 256 bytes are requested
// together).
template <int BN, int STAGES, bool kFp16In, bool kGrouped = false, int KPS = 1, bool kFused = false>
struct Cfg {
    static constexpr int kBK = kFp16In ? 64 : 128;        // K elements per K block
    static constexpr int kABox = kBM * kBKBytes;          // 16 KB
    static constexpr int kBBox = BN * kBKBytes;
    static constexpr int kABytes = KPS * kABox;
    static constexpr int kBBytes = KPS * kBBox;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr uint32_t kTmemCols = pow2_at_least(2 * BN);  // two accumulators
    static constexpr int kBarBytes = 256;
    static constexpr int kStagingOff = STAGES * kStageBytes + 1024;   // after the barriers
    static constexpr int kGroupOff = kStagingOff + staging_bytes(kFused);     // grouped: tile prefix
    static constexpr int kColumnsOff = kGroupOff + (kGrouped ? kGroupSmem : 0);   // fused: its columns' scales, bias
    static constexpr int kSmemBytes = 1024 + kColumnsOff + (kFused ? columns_bytes(BN) : 0);
    static constexpr uint32_t kIdesc = idesc_f32acc(kBM, BN, 0, 0);
    static_assert(BN % 32 == 0 && BN >= 64 && BN <= 256,
                  "BN: MMA N (multiple of 16, <= 256) and 32-column epilogue chunks");
    static_assert(kTmemCols <= 512, "TMEM columns");
    static_assert(kSmemBytes <= kSmemLimit, "shared memory");
    static_assert(kBBytes % 1024 == 0, "1024-byte aligned B stages (128-byte swizzle atoms)");
    static_assert(STAGES * kStageBytes >= 4 * (BN / 32) * kBoxBytes,
                  "every output box of a tile fits in the ring");
};

// Output tile t of this launch: A rows from a_row, B rows from b_row,
// output rows [a_row, row_end) and columns from col0.
struct Tile {
    int a_row, b_row, row_end, col0, g;
};

template <int BN, int STAGES, bool kFp16In, bool kGrouped = false, int KPS = 1, bool kFused = false>
__global__ void __launch_bounds__(gemm_threads(kFused), 1)
gemm_tc_kernel(const __grid_constant__ CUtensorMap tmap_a,
               const __grid_constant__ CUtensorMap tmap_b,
               const __grid_constant__ CUtensorMap tmap_d,
               const __grid_constant__ CUtensorMap tmap_a_edge,
               const __grid_constant__ CUtensorMap tmap_b_edge, const Params p) {
    using C = Cfg<BN, STAGES, kFp16In, kGrouped, KPS, kFused>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + STAGES * C::kABytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::kStageBytes);
    uint64_t* empty = full + STAGES;
    uint64_t* acc_full = empty + STAGES;   // [2]
    uint64_t* acc_empty = acc_full + 2;    // [2]
    uint64_t* drain = acc_empty + 2;       // [1]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
    // grouped only: tile_start[g] = first tile of group g (G + 1 entries)
    int* tile_start = reinterpret_cast<int*>(smem + C::kGroupOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], epilogue_warps(kFused));
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmap_a);
        tma_prefetch_desc(&tmap_b);
        tma_prefetch_desc(&tmap_a_edge);
        tma_prefetch_desc(&tmap_b_edge);
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
    const int num_m = (p.M + kBM - 1) / kBM;
    const int num_n = (p.N + BN - 1) / BN;
    int num_tiles = num_m * num_n;
    // pipeline steps per tile (KPS K blocks each; a block past K loads zeros)
    const int num_kb = ((p.K + C::kBK - 1) / C::kBK + KPS - 1) / KPS;
    // The prologue overlaps the preceding kernel's tail; the grouped tile
    // prefix reads the device offsets, so there the wait comes first, while
    // the plain kernel forms its first tile before it (below).
    if constexpr (kGrouped) pdl_wait();
    if constexpr (kGrouped) {
        // Tiles of group g: ceil(M_g / 128) x num_n, numbered group by group.
        // The offsets are validated here; invalid ones store nothing.
        if (warp == 3) {
            const int G = p.groups;
            bool valid = p.group_off[0] == 0 && p.group_off[G] == p.M;
            int base = 0;
            for (int g0 = 0; g0 < G; g0 += 32) {
                const int g = g0 + lane;
                int n_tiles = 0;
                if (g < G) {
                    const int m_g = p.group_off[g + 1] - p.group_off[g];
                    if (m_g < 0) valid = false;
                    n_tiles = (max(m_g, 0) + kBM - 1) / kBM * num_n;
                }
                int incl = n_tiles;   // inclusive warp scan
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                    if (lane >= o) incl += v;
                }
                if (g < G) tile_start[g] = base + incl - n_tiles;
                base += __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
            valid = __all_sync(0xFFFFFFFFu, valid);
            if (lane == 0) {
                tile_start[G] = valid ? base : 0;
                if (!valid) atomicOr(p.status, kStatusBadArgument);
            }
            if (!valid)
                for (int g = lane; g < G; g += 32) tile_start[g] = 0;
        }
        __syncthreads();
        num_tiles = tile_start[p.groups];
    }
    // Tile coordinates for tile t (cursor g only moves forward: every role
    // visits its tiles in increasing t).
    auto tile_of = [&](int t, int& g) -> Tile {
        Tile T;
        if constexpr (kGrouped) {
            while (t >= tile_start[g + 1]) ++g;
            const int local = t - tile_start[g];
            const int mt = local / num_n, nt = local - mt * num_n;
            T.a_row = p.group_off[g] + mt * kBM;
            T.row_end = p.group_off[g + 1];
            T.b_row = g * p.N + nt * BN;
            T.col0 = nt * BN;
            T.g = g;
        } else {
            int mt, nt;
            tile_coords(t, num_m, num_n, p.group_m, mt, nt);
            T.a_row = mt * kBM;
            T.row_end = p.M;
            T.b_row = nt * BN;
            T.col0 = nt * BN;
            T.g = 0;
        }
        return T;
    };
    // The producer's first tile depends only on the launch: formed before the
    // dependency wait while the preceding kernel drains (the empty asm keeps
    // it there).
    Tile T0{};
    if constexpr (!kGrouped) {
        if (warp == 0 && lane == 0 && static_cast<int>(blockIdx.x) < num_tiles) {
            int g0 = 0;
            T0 = tile_of(static_cast<int>(blockIdx.x), g0);
            asm volatile("" :: "r"(T0.a_row), "r"(T0.b_row), "r"(T0.row_end), "r"(T0.col0) : "memory");
        }
        pdl_wait();
    }

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------ TMA producer
        int stage = 0;
        uint32_t phase = 0;
        uint32_t issued_mask = 0;          // stages with a load ever issued
        uint32_t issued_phase = 0;         // parity of each stage's last load
        bool skip = p.skip_first_load != 0 && blockIdx.x == 0;
        bool ok = true;
        bool first_lap = true;   // every stage starts free: no wait on the first lap
        int gcur = 0;
        for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
            const Tile T = (!kGrouped && t == static_cast<int>(blockIdx.x)) ? T0 : tile_of(t, gcur);
            for (int kb = 0; kb < num_kb; ++kb) {
                if (!first_lap && !wait_bounded(&empty[stage], phase ^ 1u, ctl)) { ok = false; break; }
                if (skip) {
                    skip = false;           // leave this stage unloaded
                } else {
                    // edge tiles load shorter boxes through their own maps
                    const bool ae = T.a_row >= p.a_edge_row, be = T.b_row >= p.b_edge_row;
                    mbar_arrive_expect_tx(&full[stage], KPS * ((ae ? p.a_edge_bytes : p.a_box_bytes) +
                                                               (be ? p.b_edge_bytes : p.b_box_bytes)));
#pragma unroll
                    for (int j = 0; j < KPS; ++j) {
                        const int x = (kb * KPS + j) * C::kBK;
                        tma_load_2d(sA + stage * C::kABytes + j * C::kABox,
                                    ae ? &tmap_a_edge : &tmap_a, &full[stage], x, T.a_row);
                        tma_load_2d(sB + stage * C::kBBytes + j * C::kBBox,
                                    be ? &tmap_b_edge : &tmap_b, &full[stage], x, T.b_row);
                    }
                    issued_mask |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                }
                if (++stage == STAGES) { stage = 0; phase ^= 1u; first_lap = false; }
            }
        }
        // Every load this thread issued must have landed before the CTA can
        // exit.  After a normal run they all have (the MMA thread consumed
        // each one) and these waits return at once; after an abort they let
        // copies still in flight finish.
        for (int s = 0; s < STAGES; ++s)
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
        for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
            if (!wait_bounded(&acc_empty[acc], acc_phase ^ 1u, ctl)) { ok = false; break; }
            tc_fence_after_sync();
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
            for (int kb = 0; kb < num_kb; ++kb) {
                if (!wait_bounded(&full[stage], phase, ctl)) { ok = false; break; }
                tc_fence_after_sync();
#pragma unroll
                for (int j = 0; j < KPS; ++j) {
                    const uint32_t a0 = smem_addr(sA + stage * C::kABytes + j * C::kABox);
                    const uint32_t b0 = smem_addr(sB + stage * C::kBBytes + j * C::kBBox);
#pragma unroll
                    for (int kk = 0; kk < kBKBytes / 32; ++kk) {
                        const uint64_t ad = sdesc_k_major_sw128(a0 + kk * 32);
                        const uint64_t bd = sdesc_k_major_sw128(b0 + kk * 32);
                        const uint32_t accum = (kb > 0 || j > 0 || kk > 0) ? 1u : 0u;
                        if constexpr (kFp16In)
                            mma_f16(d_tmem, ad, bd, C::kIdesc, accum);
                        else
                            mma_f8f6f4(d_tmem, ad, bd, C::kIdesc, accum);
                    }
                }
                issued_any = true;
                mma_commit(&empty[stage]);   // frees the stage when these MMAs finish
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            mma_commit(&acc_full[acc]);      // accumulator ready for the epilogue
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
        if (issued_any) {
            // Tensor memory is freed below: wait for every MMA this thread
            // issued (normal end or abort alike).
            mma_commit(drain);
            wait_bounded(drain, 0, ctl, false);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------ epilogue
        const int q = warp & 3;              // TMEM lane quarter of this warp
        // its chunks of 32 columns: every one, or every second from `half` on
        constexpr int kChunkStep = epilogue_warps(kFused) / 4;
        const int half = kFused ? (warp - 4) >> 2 : 0;
        auto alpha_of = [&](int g) {
            float a = 1.0f;
            if (kFused) return a;
            if (p.sa != nullptr) a = p.sa[g] * p.sb[g];
            if (p.out_kind == kOutE4M3) a = __fdiv_rn(a, p.sd[g]);
            return a;
        };
        float alpha = alpha_of(0);
        int alpha_g = 0;
        float* columns = reinterpret_cast<float*>(smem + C::kColumnsOff) +
                         (warp - 4) * fused_chunks(BN) * kColumnFloats;
        const ByScale out_scale = kFused ? output_scale(p.out_kind, p.sd) : ByScale{1.0f, 1.0f};
        uint32_t amax_bits = 0u;
        int acc = 0;
        uint32_t acc_phase = 0;
        int gcur = 0;
        for (int t = blockIdx.x; t < num_tiles; t += gridDim.x) {
            const Tile T = tile_of(t, gcur);
            if (T.g != alpha_g) {
                alpha = alpha_of(T.g);
                alpha_g = T.g;
            }
            // The next kernel in the stream may be scheduled once every CTA
            // is on its last tile (it still waits for this grid's memory).
            const bool last_tile = t + static_cast<int>(gridDim.x) >= num_tiles;
            if (p.early_release && last_tile && warp == 4 && lane == 0) pdl_launch_dependents();
            const int row = T.a_row + q * 32 + lane;
            const int row0 = T.a_row + q * 32;
            // The fused epilogue's own operands, on their way while the main
            // loop runs; the residual one 32-column chunk ahead.
            const bool row_ok = row < T.row_end;
            ScaleParts sa{1.0f, 1.0f};
            bool parts = false;
            uint32_t res[16];
            if constexpr (kFused) {
                sa = scale_parts(scale_of_row(p, row, row_ok));
                if ((p.N & 7) == 0) load_residual(p, row, row_ok, T.col0 + 32 * half, res);
                prefetch_residual<BN>(p, row, row_ok, T.col0, half);
                parts = stage_columns<BN>(p, columns, T.col0, half, lane);
            }
            // Every lane waits; the vote reconverges the warp (tcgen05.ld is
            // .sync.aligned) and makes the whole warp leave together.
            const bool got = wait_bounded(&acc_full[acc], acc_phase, ctl);
            if (!__all_sync(0xFFFFFFFFu, got)) break;
            tc_fence_after_sync();
            const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                   static_cast<uint32_t>(acc * BN);
            if constexpr (kFused) {
                if (parts) apply_wholes_to_tile<BN>(p, tbase, T.col0, half, lane);
            }
            // Staged bulk stores (whole lines, M / N edges clipped by the
            // tensor map) unless the warp's 32 rows cross a group's end,
            // which the tensor map cannot clip: those rows store directly.
            // One staging box per warp while later tiles' main loops run;
            // on the last tile the ring of stages is idle and every box has
            // a place of its own in it, so the stores go out back to back.
            const bool staged = p.staged && (!kGrouped || row0 + 32 <= T.row_end);
#pragma unroll 1
            for (int c = half; c < BN / 32; c += kChunkStep) {
                uint32_t r[32];
                __syncwarp();
                tmem_load_32cols(tbase + c * 32, r);
                if (staged) {
                    uint8_t* box = last_tile ? smem + (q * (BN / 32) + c) * kBoxBytes
                                             : smem + C::kStagingOff + (warp - 4) * kBoxBytes;
                    if (!last_tile && lane == 0) bulk_wait_read_all();   // the box is free again
                    __syncwarp();
                    tmem_load_wait(r);
                    const int col0 = T.col0 + c * 32;
                    if constexpr (kFused) {
                        float v[32];
                        amax_bits = max(amax_bits, fuse32(p, row_ok, col0, r, res, sa, columns + kColumnFloats * (c / kChunkStep), out_scale, v));
                        if (c + kChunkStep < BN / 32) load_residual(p, row, row_ok, col0 + 32 * kChunkStep, res);
                        stage_values(p, box, v, lane);
                    } else {
                        amax_bits = max(amax_bits, stage_box(p, box, row, T.row_end, col0, r, alpha, lane));
                    }
                    if (last_tile) continue;   // stored together below
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && row0 < T.row_end && col0 < p.N) {
                        tma_store_2d(&tmap_d, box, col0, row0);
                        bulk_commit();
                    }
                } else {
                    tmem_load_wait(r);
                    const int col0 = T.col0 + c * 32;
                    if constexpr (kFused) {
                        uint8_t* box = smem + C::kStagingOff + (warp - 4) * kBoxBytes;
                        if ((p.N & 7) != 0) load_residual_odd(p, box, row0, T.row_end, col0, lane, res);
                        float v[32];
                        amax_bits = max(amax_bits, fuse32(p, row_ok, col0, r, res, sa, columns + kColumnFloats * (c / kChunkStep), out_scale, v));
                        if ((p.N & 7) == 0 && c + kChunkStep < BN / 32)
                            load_residual(p, row, row_ok, col0 + 32 * kChunkStep, res);
                        store_box_odd(p, box, row0, T.row_end, col0, v, lane);
                    } else {
                        amax_bits = max(amax_bits, store_chunk(p, row, T.row_end, col0, r, alpha));
                    }
                }
            }
            if (staged && last_tile) {
                // every box of the warp is in the idle ring: one fence, then
                // all of its stores
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && row0 < T.row_end) {
                    for (int c = half; c < BN / 32 && T.col0 + c * 32 < p.N; c += kChunkStep)
                        tma_store_2d(&tmap_d, smem + (q * (BN / 32) + c) * kBoxBytes, T.col0 + c * 32,
                                     row0);
                    bulk_commit();
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
        // The staging box must have been written out before the CTA exits.
        if (lane == 0) bulk_wait_all();
        __syncwarp();
        if constexpr (kFused)
            publish_top(p.amax_out, amax_bits);
        else
            publish_amax(p, amax_bits);
    }

    // Warps 0 and 1 may arrive diverged (their lane 0 ran a role alone): the
    // barrier before tensor memory is freed is the non-aligned one.
    tc_fence_before_sync();
    cta_sync_diverged();
    tc_fence_after_sync();
    if (warp == 2) tmem_dealloc<C::kTmemCols>(tmem_base);
}

// ------------------------------------------------------------- host side

template <int BN, int STAGES, bool kFp16In, bool kGrouped = false, int KPS = 1, bool kFused = false>
cudaError_t launch_cfg(const TcLaunch& L, const Params& prm, cudaStream_t s) {
    using C = Cfg<BN, STAGES, kFp16In, kGrouped, KPS, kFused>;
    static std::mutex mu;
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        if (!attr_done[dev]) {
            e = cudaFuncSetAttribute(gemm_tc_kernel<BN, STAGES, kFp16In, kGrouped, KPS, kFused>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
            if (e != cudaSuccess) return e;
            attr_done[dev] = true;
        }
    }
    CUtensorMap ta, tb, td;
    const int b_rows = kGrouped ? L.N * L.groups : L.N;   // grouped: B is (G*N) x K
    // Edge boxes: the last tile of an operand that ends inside a tile (128
    // rows of A, BN of B) loads boxes of the rows left rounded up to 8, so
    // no box reaches far past the tensor's end.  Those rows still cross
    // into the SM and slow every load: E4M3 17 x 11008 x 4096 17.3 -> 12.5
    // us, 33 x 12288 x 1040 9.9 -> 7.0, 48 x 11008 x 1040 9.3 -> 7.2 with
    // the short box; no change at 4096-deep K for 33..120 rows.
    // DG_TC_SHORT_BOX=0 keeps full boxes everywhere, =1 narrows only an
    // operand of at most 32 rows (sweeps).  Grouped B rows are slices of
    // one tall tensor: full boxes.
    const int sb = knobs().tc_short_box;
    auto edge = [&](int rows, int full, int* edge_row, int* edge_box) {
        const int left = rows % full;
        *edge_row = INT_MAX;
        *edge_box = full;
        if (kGrouped || left == 0 || sb == 0 || (sb == 1 && rows > 32)) return;
        *edge_row = rows - left;
        *edge_box = (left + 7) / 8 * 8;
    };
    int a_edge_row, a_edge_box, b_edge_row, b_edge_box;
    edge(L.M, kBM, &a_edge_row, &a_edge_box);
    edge(L.N, BN, &b_edge_row, &b_edge_box);
    // (an operand without an edge tile passes its full map twice: no
    // second encoding on the host)
    CUtensorMap tae, tbe;
    if (!make_map(&ta, L.A, L.M, L.K, kFp16In, kBM) ||
        !make_map(&tb, L.B, b_rows, L.K, kFp16In, BN))
        return cudaErrorInvalidValue;
    tae = ta;
    tbe = tb;
    if ((a_edge_row != INT_MAX && !make_map(&tae, L.A, L.M, L.K, kFp16In, a_edge_box)) ||
        (b_edge_row != INT_MAX && !make_map(&tbe, L.B, b_rows, L.K, kFp16In, b_edge_box)))
        return cudaErrorInvalidValue;
    Params prm2 = prm;
    prm2.a_box_bytes = kBM * kBKBytes;
    prm2.b_box_bytes = BN * kBKBytes;
    prm2.a_edge_bytes = a_edge_box * kBKBytes;
    prm2.b_edge_bytes = b_edge_box * kBKBytes;
    prm2.a_edge_row = a_edge_row;
    prm2.b_edge_row = b_edge_row;
    // Output map of the staged epilogue (else the epilogue stores directly).
    if (!prm2.staged || !make_out_map(&td, L)) {
        prm2.staged = 0;
        td = ta;
    }
    return launch_kernel(gemm_tc_kernel<BN, STAGES, kFp16In, kGrouped, KPS, kFused>, dim3(L.plan->grid),
                         dim3(gemm_threads(kFused)), C::kSmemBytes, s, ta, tb, td, tae, tbe, prm2);
}

template <bool kFp16In, bool kFused>
cudaError_t launch_in(const TcLaunch& L, const Params& prm, cudaStream_t s) {
    switch (L.plan->block_n) {
        // two K blocks per stage: block_k is twice the K block
        case 64:
            if (L.plan->block_k == 2 * (kFp16In ? 64 : 128))
                return launch_cfg<64, stages_for(64, false, 2, kFused), kFp16In, false, 2, kFused>(L, prm, s);
            return launch_cfg<64, stages_for(64, false, 1, kFused), kFp16In, false, 1, kFused>(L, prm, s);
        case 96:
            if (L.plan->block_k == 2 * (kFp16In ? 64 : 128))
                return launch_cfg<96, stages_for(96, false, 2, kFused), kFp16In, false, 2, kFused>(L, prm, s);
            return launch_cfg<96, stages_for(96, false, 1, kFused), kFp16In, false, 1, kFused>(L, prm, s);
        case 128:
            if (L.plan->block_k == 2 * (kFp16In ? 64 : 128))
                return launch_cfg<128, stages_for(128, false, 2, kFused), kFp16In, false, 2, kFused>(L, prm, s);
            return launch_cfg<128, stages_for(128, false, 1, kFused), kFp16In, false, 1, kFused>(L, prm, s);
        case 160: return launch_cfg<160, stages_for(160, false, 1, kFused), kFp16In, false, 1, kFused>(L, prm, s);
        case 192: return launch_cfg<192, stages_for(192, false, 1, kFused), kFp16In, false, 1, kFused>(L, prm, s);
        case 224: return launch_cfg<224, stages_for(224, false, 1, kFused), kFp16In, false, 1, kFused>(L, prm, s);
        default: return launch_cfg<256, stages_for(256, false, 1, kFused), kFp16In, false, 1, kFused>(L, prm, s);
    }
}

}  // namespace
}  // namespace dg
