// k_gemm_tc2.cu -- CTA-pair variant of the tensor-core GEMM (M >= 256).
//
// Page shorthands: [FP8-guide] = "DeepGEMM实战：FP8矩阵乘法与JIT编译优化指南";
// [DG-FP16] = the DeepGEMM FP16/WMMA deep-dive page.
//
// Same computation and epilogue as k_gemm_tc.cu ([FP8-guide] §2.3, §3.1-§3.3;
// [DG-FP16] §2.2), but two CTAs on two SMs (a cluster of 2) share one
// 256 x BN output tile.  Each CTA holds its own 128 rows of A and half of the
// tile's BN rows of B; one pair MMA (M = 256) reads A from both CTAs and B
// from both CTAs, and writes each CTA's 128 rows of the accumulator into that
// CTA's tensor memory.  Per SM this halves the B bytes that TMA writes into
// shared memory and that the MMA reads from it, the traffic that limits the
// single-CTA kernel with 128 x 256 tiles.
//
// From 12 K blocks on a stage holds two adjacent K blocks (KPS = 2): half
// the full/empty round trips per K block, which with one per stage set a
// floor on the time per K block above the MMA's own for tiles under 256
// wide.
//
// Signalling (all waits bounded):
//  * each CTA's producer loads its halves into its own shared memory; every
//    box completes on the even CTA's `full` barrier of the stage, whose
//    producer arms it for the bytes of both CTAs (of the stage's K blocks
//    within the item's K range);
//  * the even CTA's MMA thread issues the pair MMAs and frees a stage in both
//    CTAs with one multicast commit to `empty`; at the end of a tile it
//    commits to `acc_full` in both CTAs;
//  * both CTAs' epilogue warps release an accumulator buffer by arriving on
//    the even CTA's `acc_empty` (count 8: four warps per CTA; 16 when fused);
//  * a final multicast commit to `drain` tells both CTAs that no pair MMA
//    still reads their shared memory or writes their tensor memory; only
//    then is tensor memory freed (collectively) and the CTAs exit;
//  * the epilogue (which overlaps the next tile's main loop) stages each
//    warp's 32 x 32 output boxes in a buffer of its own (TMA's 64- or 32-byte
//    swizzle) and writes them with bulk tensor stores -- whole lines, edges
//    clipped by the tensor map -- instead of one scattered 16-byte row piece
//    per lane, whose many partial-line writes slowed the concurrent main
//    loop by ~1 us per tile at 4096^3;
//  * once every CTA is on its last tile the grid lets the next kernel in the
//    stream be scheduled, so that its CTAs start as these exit.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <mutex>

#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "gemm_common.cuh"
#include "gemm_pair_kernel.cuh"

namespace dg {

int pair_smem_for(int bn, int kps) {
    if (kps == 2) {
        switch (bn) {
            case 128: return PairCfg<128, pair_stages_for(128, 2), false, 2>::kSmemBytes;
            case 160: return PairCfg<160, pair_stages_for(160, 2), false, 2>::kSmemBytes;
            case 192: return PairCfg<192, pair_stages_for(192, 2), false, 2>::kSmemBytes;
            case 224: return PairCfg<224, pair_stages_for(224, 2), false, 2>::kSmemBytes;
            default: return PairCfg<256, pair_stages_for(256, 2), false, 2>::kSmemBytes;
        }
    }
    switch (bn) {
        case 128: return PairCfg<128, pair_stages_for(128), false>::kSmemBytes;
        case 160: return PairCfg<160, pair_stages_for(160), false>::kSmemBytes;
        case 192: return PairCfg<192, pair_stages_for(192), false>::kSmemBytes;
        case 224: return PairCfg<224, pair_stages_for(224), false>::kSmemBytes;
        default: return PairCfg<256, pair_stages_for(256), false>::kSmemBytes;
    }
}

int pair_stages(int bn, int kps) { return pair_stages_for(bn, kps); }

cudaError_t launch_gemm_tc_pair(const TcLaunch& L, const Params& prm, cudaStream_t s) {
    return L.fp16_in ? launch_pair_in<true, false>(L, prm, s) : launch_pair_in<false, false>(L, prm, s);
}

}  // namespace dg
