// k_gemm_tc.cu -- the tensor-core GEMM for M > 16 (E4M3 or FP16 inputs,
// FP32 accumulation in tensor memory, fused scale/convert epilogue).
//
// Page shorthands: [FP8-guide] = "DeepGEMM实战：FP8矩阵乘法与JIT编译优化指南";
// [DG-FP16] = the DeepGEMM FP16/WMMA deep-dive page; [HGEMM-L2] =
// "HGEMM优化：深度学习中的矩阵乘法性能提升策略".
//
// What the pages prescribe, and how it maps onto sm_103a:
//  * block tiling of C with a K-blocked main loop ([FP8-guide] §3.1) ->
//    128 x BN output tiles, 128-byte K blocks, one tcgen05.mma (M=128,
//    N=BN, K=32 bytes) per 32 bytes of K, accumulating in tensor memory;
//  * loader warps separate from compute warps ([DG-FP16] §2.2) and a
//    multi-stage prefetch pipeline ([FP8-guide] §2.3, §4.4; [HGEMM-L2]
//    §3.2-§3.3) -> one TMA producer thread, one MMA-issuing thread and four
//    epilogue warps, joined by full/empty mbarriers over a STAGES-deep
//    shared-memory ring; single-wave plans up to 128 wide over at least 12
//    K blocks hold two adjacent K blocks per stage (256 contiguous bytes of
//    every operand row per request, half the barrier round trips);
//  * bank-conflict-free shared-memory layout ([DG-FP16] §3.2) -> TMA's
//    128-byte swizzle, which the MMA's shared-memory descriptors read
//    natively;
//  * scale_A * scale_B applied once to the accumulator on write-back, and
//    the output scale divided out for FP8 output ([FP8-guide] §3.2);
//  * M/N edges by predication and K tails by zero fill, in one kernel
//    ([FP8-guide] §3.3) -> TMA fills out-of-range box elements with zeros,
//    and epilogue stores are predicated on m < M, n < N; an operand that
//    ends inside a tile loads that last tile through a second tensor map
//    whose box is the rows left rounded up to 8, since rows of a box past
//    the tensor's end still cross into the SM.
// The kernel is persistent (one CTA per SM, tiles strided by the grid) and
// double-buffers the accumulator in tensor memory so that the epilogue of
// one tile overlaps the main loop of the next; the epilogue writes each
// warp's 32 x 32 output boxes through a staging box in shared memory with
// bulk tensor stores (whole lines; direct stores only for a grouped tile's
// rows that cross its group's end).  Every mbarrier wait is
// bounded: on a timeout the CTA raises its abort flag, records
// kStatusTimeout, lets in-flight copies and MMAs land, frees its tensor
// memory and returns.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <mutex>

#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "gemm_common.cuh"
#include "gemm_tc_kernel.cuh"

namespace dg {
namespace {

int smem_for(int bn) {
    switch (bn) {
        case 64: return Cfg<64, stages_for(64), false>::kSmemBytes;
        case 96: return Cfg<96, stages_for(96), false>::kSmemBytes;
        case 128: return Cfg<128, stages_for(128), false>::kSmemBytes;
        case 160: return Cfg<160, stages_for(160), false>::kSmemBytes;
        case 192: return Cfg<192, stages_for(192), false>::kSmemBytes;
        case 224: return Cfg<224, stages_for(224), false>::kSmemBytes;
        default: return Cfg<256, stages_for(256), false>::kSmemBytes;
    }
}

}  // namespace

void plan_tc(int64_t M, int64_t N, int64_t K, bool fp16_in, int sm_count, dg_plan* p) {
    // Per-shape tile choice ([FP8-guide] §3.1, §3.3; [HGEMM-L2] §3.1):
    // estimate each candidate's time as (waves of tiles over the SMs) x
    // (tile width / relative MMA efficiency of that width) and keep the
    // cheapest; narrow tiles win when the grid would otherwise leave SMs
    // idle or strand a partial last wave.
    const int64_t num_m = (M + kBM - 1) / kBM;
    // Relative throughput per CTA of a 128 x BN tile.  Each 32-byte K step
    // reads 4 KB of A and BN*32 B of B from shared memory while the MMA runs
    // for BN/2 cycles, so narrow tiles need more shared-memory bandwidth per
    // flop (8192/BN + 64 B/clk).  Measured on GB300 (8192^3 E4M3): BN 256 ->
    // 1.0, 128 -> 0.72, 64 -> 0.36; the widths in between are interpolated
    // along that demand curve.  The 96-wide tile (last-but-one candidate)
    // takes part only in the one-wave rule below.
    constexpr int kCand = 7;
    const int cand[kCand] = {256, 224, 192, 160, 128, 96, 64};
    const double eff[kCand] = {1.0, 0.95, 0.88, 0.80, 0.72, 0.0, 0.36};
    int best = 256;
    double best_cost = 0.0;
    for (int i = 0; i < kCand; ++i) {
        if (cand[i] == 96) continue;
        const int bn = cand[i];
        const int64_t tiles = num_m * ((N + bn - 1) / bn);
        const int64_t waves = (tiles + sm_count - 1) / sm_count;
        const double cost = static_cast<double>(waves) * bn / eff[i];
        if (i == 0 || cost < best_cost) { best = bn; best_cost = cost; }
    }
    // A width that puts every tile in one wave (K up to 64 K blocks, up to
    // 32 for widths above 128): the launch is bound by latency and each
    // SM's own operand stream rather than by MMA efficiency, so the
    // narrowest such tile (most CTAs, fewest bytes per CTA) wins, and CTA
    // pairs only add cluster start-up.  Measured on GB300 (BF16 out,
    // graph-replayed), against the estimate below: 256^3 3.2 us (128 x 64)
    // vs 5.2 (pairs 256 x 128); 1024^3 5.9 vs 8.1; 129 x 1000 x 1040 6.8 vs
    // 7.7; 1024 x 1024 x 8192 20.9 vs 24.0; FP16 1024^3 8.1 vs 10.3;
    // 1024 x 4096 x 4096 15.5 vs 17.2 (128 x 224); equal at 256 x 12288 x
    // 4096.  DG_ONE_WAVE=0 turns the rule off and DG_ONE_WAVE_KB sets its
    // K-block limit (sweeps).
    const int64_t kblocks = (K + (fp16_in ? 64 : 128) - 1) / (fp16_in ? 64 : 128);
    const Knobs& kn = knobs();
    bool one_wave = false;
    if (kn.one_wave && kblocks <= kn.one_wave_kb) {
        for (int i = kCand - 1; i >= 0; --i) {   // narrowest first
            if (num_m * ((N + cand[i] - 1) / cand[i]) <= sm_count) {
                // past 32 K blocks a wide tile is MMA-bound enough for the
                // pairs' efficiency to win (2048^2 x 8192: 26.1 us as pairs
                // vs 27.6 as 128 x 256 single tiles)
                if (kblocks <= 32 || cand[i] <= 128) {
                    best = cand[i];
                    one_wave = true;
                }
                break;
            }
        }
    }
    // DG_FORCE_BLOCK_N=64|96|128|160|192|224|256 pins the tile width (sweeps).
    {
        const int v = kn.force_block_n;
        for (int i = 0; i < kCand; ++i)
            if (v == cand[i]) best = v;
    }
    const int64_t tiles = num_m * ((N + best - 1) / best);
    p->block_m = kBM;
    p->block_n = best;
    p->block_k = fp16_in ? 64 : 128;
    p->stages = stages_for(best);
    p->tiles = static_cast<int>(tiles);
    p->grid = static_cast<int>(tiles < sm_count ? tiles : sm_count);
    p->smem_bytes = smem_for(best);
    // Single-wave plans up to 128 wide over at least 12 K blocks take two K
    // blocks per stage: each stage then requests 256 contiguous bytes of
    // every row of B, which streams better, and the barrier round trips per
    // K block halve.  Measured on GB300 (graph-replayed, us, one -> two):
    // E4M3 32 x 12288 x 4096 12.87 -> 12.27, 128 x 12288 x 4096 13.28 ->
    // 12.82, 96 x 8192 x 2048 7.84 -> 6.86, 32 x 8192 x 3072 9.73 -> 8.27,
    // 48 x 12288 x 1536 7.28 -> 6.96, 256 x 4096 x 11008 26.59 -> 23.73,
    // 2048 x 1024 x 11008 27.12 -> 22.47, 512 x 2048 x 8192 20.40 -> 16.15;
    // FP16 1024 x 1024 x 8192 37.85 -> 32.20; over 9 K blocks no gain and up
    // to 4% lost on latency-bound shapes (129 x 1000 x 1040 5.33 -> 5.53).
    // DG_TC_KPS=1|2 pins one or two for every such plan (sweeps).
    const bool kps2 = kn.tc_kps == 2 || (kn.tc_kps == 0 && kblocks >= 12);
    if (tiles <= sm_count && kps2 && best <= 128) {
        p->block_k *= 2;
        p->stages = stages_for(best, false, 2);
        p->smem_bytes = best == 64 ? Cfg<64, stages_for(64, false, 2), false, false, 2>::kSmemBytes
                        : best == 96 ? Cfg<96, stages_for(96, false, 2), false, false, 2>::kSmemBytes
                                     : Cfg<128, stages_for(128, false, 2), false, false, 2>::kSmemBytes;
    }

    // CTA pairs (256 x BN tiles over sm_count / 2 clusters), for M >= 256.
    // Per-SM throughput relative to the single-CTA 128 x 256 tile: each SM
    // stores and reads only half of the tile's B rows.  Measured on GB300:
    // 8192^3 E4M3 3607 vs 3399 TFLOP/s (1.06).  With one K block per stage
    // a pair tile cost about the same whatever its N (4096^3 E4M3,
    // interleaved: 45.6 / 45.7 / 53.4 / 61.3 / 70.3 us at BN 256 / 224 /
    // 192 / 160 / 128 over 4 / 4 / 5 / 6 / 7 waves): the per-K-block
    // barrier round trip set the pace, so the narrower widths' relative
    // rates were below their share of 256; two K blocks per stage raise
    // them (below).  A partial last wave whose tiles the kernel splits along
    // K (two to four K ranges per tile over idle pairs) counts as that
    // fraction of a wave.  Pairs are used when their estimate is no worse;
    // DG_2CTA=0 disables them, DG_2CTA=1 forces them for M >= 256.
    const bool pairs_off = kn.two_cta == 0;
    const bool pairs_forced = kn.two_cta == 1;
    if (!pairs_off && (!one_wave || pairs_forced) && M >= 256 && sm_count >= 2) {
        const int64_t pm = (M + 255) / 256;
        const int slots = sm_count / 2;
        const int pcand[5] = {256, 224, 192, 160, 128};
        // Narrower widths with two K blocks per stage (12 K blocks on):
        // 4096^3 E4M3, 4 / 4 / 5 / 6 / 7 rounds: 43.5 / 42.5 / 46.9 / 51.2 /
        // 58.0 us at BN 256 / 224 / 192 / 160 / 128.  The plans this moves
        // from single-CTA to pair tiles of the same width, measured (us,
        // single -> pair): 3072 x 2240 x 11008 54.07 -> 50.65, 512 x 5120 x
        // 11008 28.00 -> 26.04, 1536 x 7168 x 8192 62.14 -> 59.94, 768 x
        // 7168 x 4096 22.51 -> 21.61, FP16 256 x 11008 x 4096 23.37 ->
        // 23.05; 256 x 12288 x 8192 25.97 -> 26.48 and 1024 x 5120 x 2048
        // 13.76 -> 13.92 the other way.
        const bool pk2 = kn.pair_kps == 2 || (kn.pair_kps == 0 && kblocks >= 12);
        const double peff[5] = {1.06, 0.95, pk2 ? 0.92 : 0.83, pk2 ? 0.84 : 0.72, pk2 ? 0.68 : 0.58};
        int pbest = 256;
        double pcost = 0.0;
        for (int i = 0; i < 5; ++i) {
            const int bn = pcand[i];
            const int64_t pt = pm * ((N + bn - 1) / bn);
            const int64_t full = pt / slots, rem = pt % slots;
            const int64_t split = rem > 0 ? std::min<int64_t>(slots / rem, 4) : 0;
            double waves = static_cast<double>(full);
            if (rem > 0)
                waves += (kn.split_tail && split >= 2 && kblocks >= split)
                             ? 1.0 / static_cast<double>(split) : 1.0;
            const double cost = waves * bn / peff[i];
            if (i == 0 || cost < pcost) { pbest = bn; pcost = cost; }
        }
        {
            const int v = kn.force_block_n;
            if (v == 128 || v == 160 || v == 192 || v == 224 || v == 256) pbest = v;
        }
        if (pairs_forced || pcost <= best_cost) {
            const int64_t pt = pm * ((N + pbest - 1) / pbest);
            p->block_m = 256;
            p->block_n = pbest;
            // Two K blocks per stage from 12 K blocks on, as for single-CTA
            // tiles: fewer barrier round trips per K block.  Measured on GB300
            // (graph-replayed, us, one -> two): E4M3 4096^3 45.92 -> 43.58,
            // HGEMM 4096^3 83.14 -> 79.59, 4096 x 4096 x 8192 85.31 ->
            // 82.31, FP16 1024 x 4096 x 4096 25.82 -> 24.83; the 8192^3 bench
            // step's GEMM 0.304-0.307 -> 0.298-0.301 ms.  DG_PAIR_KPS=1|2
            // pins either (sweeps).
            const int pkps = kn.pair_kps != 0 ? kn.pair_kps : (kblocks >= 12 ? 2 : 1);
            p->block_k = (fp16_in ? 64 : 128) * pkps;
            p->stages = pair_stages(pbest, pkps);
            p->tiles = static_cast<int>(pt);
            p->grid = static_cast<int>(2 * (pt < slots ? pt : slots));
            p->smem_bytes = pair_smem_for(pbest, pkps);
        }
    }
}

Params make_params(const TcLaunch& L) {
    Params prm;
    prm.D = L.D;
    prm.M = L.M;
    prm.N = L.N;
    prm.K = L.K;
    prm.sa = L.sa;
    prm.sb = L.sb;
    prm.sd = L.sd;
    prm.out_kind = L.out_kind;
    prm.out_elem = L.out_elem;
    prm.vec_ok = ((static_cast<int64_t>(L.N) * L.out_elem) % 16 == 0) ? 1 : 0;
    prm.staged = prm.vec_ok && knobs().staged_epilogue ? 1 : 0;   // confirmed by the launcher
    prm.early_release = knobs().early_release ? 1 : 0;
    prm.tail_split = 1;   // set by the CTA-pair launcher when the tail is split
    prm.tail_ws = nullptr;
    prm.tail_counts = nullptr;
    prm.status = L.status;
    prm.timeout_ns = wait_timeout_ns();
    prm.skip_first_load = take_skip_first_load() ? 1 : 0;
    prm.amax_out = L.amax_out;
    // Raster: groups of 32 M-tiles when there are many (8192^3: 3361 vs 3285
    // TFLOP/s at 16, measured), 8 otherwise (4096^3: 2865 vs 2830).
    prm.group_m = ((L.M + kBM - 1) / kBM) >= 48 ? 32 : 8;
    if (L.plan->block_m == 256) prm.group_m /= 2;   // pair tiles are 256 rows
    // DG_GROUP_M=<n> overrides the raster group size (sweeps).
    if (knobs().group_m != 0) prm.group_m = knobs().group_m;
    if (L.epi != nullptr) prm.epi = *L.epi;
    prm.group_off = L.group_off;
    prm.groups = L.groups;
    prm.a_box_bytes = kBM * kBKBytes;   // the single-CTA launcher sets the edge boxes
    prm.b_box_bytes = L.plan->block_n * kBKBytes;
    prm.a_edge_bytes = prm.a_box_bytes;
    prm.b_edge_bytes = prm.b_box_bytes;
    prm.a_edge_row = INT_MAX;
    prm.b_edge_row = INT_MAX;
    return prm;
}

cudaError_t launch_gemm_tc(const TcLaunch& L, cudaStream_t s) {
    const Params prm = make_params(L);
    if (L.plan->block_m == 256)
        return L.epi != nullptr ? launch_gemm_tc_pair_fused(L, prm, s) : launch_gemm_tc_pair(L, prm, s);
    if (L.epi != nullptr) return launch_gemm_tc_fused(L, prm, s);
    return L.fp16_in ? launch_in<true, false>(L, prm, s) : launch_in<false, false>(L, prm, s);
}

cudaError_t launch_gemm_tc_grouped(const TcLaunch& L, cudaStream_t s) {
    if (L.fp16_in || L.groups < 1 || L.groups > kMaxGroups) return cudaErrorInvalidValue;
    const Params prm = make_params(L);
    if (L.plan->block_n == 128)
        return launch_cfg<128, stages_for(128, true), false, true>(L, prm, s);
    return launch_cfg<256, stages_for(256, true), false, true>(L, prm, s);
}

}  // namespace dg
