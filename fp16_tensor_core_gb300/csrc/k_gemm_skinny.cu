// k_gemm_skinny.cu -- the tensor-core path for skinny GEMMs (M <= 128 with
// few output tiles): split-K over every SM, with the operands swapped so that
// the long side fills the 128-row MMA.
//
// Page shorthands: [FP8-guide] = "DeepGEMM实战：FP8矩阵乘法与JIT编译优化指南";
// [DG-FP16] = the DeepGEMM FP16/WMMA deep-dive page.
//
// For a decode-style product (a handful of activation rows against a large
// weight matrix) the weight B is read once and the work is bound by HBM
// ([DG-FP16] §2.1, weight-aware tiling).  A 128 x BN output tile with
// M <= 16 would leave 7/8 of each MMA empty and give N/BN tiles -- too few
// to occupy 152 SMs.  Here instead:
//  * operands are swapped: the MMA computes D^T = B * A^T, its M side (128)
//    is 128 rows of B and its N side (NC = 16, 32, 64 or 128) the M rows of
//    A rounded up, zero-filled by TMA past M ([FP8-guide] §3.3's edge
//    handling);
//  * the K blocks of all tiles form one sequence of `units` (tile, k block)
//    that is cut into gridDim.x equal contiguous ranges, one per CTA, so every
//    SM streams the same number of bytes (split-K, balanced);
//  * a CTA's range splits at tile boundaries into segments.  A segment that
//    covers a whole tile writes D directly; otherwise the CTA stores its FP32
//    partial tile in a workspace slot and bumps the tile's arrival counter,
//    and the CTA that arrives last adds the partials in segment order (fixed,
//    so the result does not depend on arrival order), applies
//    scale_A * scale_B (/ scale_D for E4M3 out, [FP8-guide] §3.2), stores D
//    and resets the counter to zero.  No CTA waits for another.
// Pipeline: one TMA thread, one MMA thread, four epilogue warps, a ring of
// K blocks (16 KB of B + NC x 128 bytes of A each; 12 of them for NC = 16,
// 6 for NC = 128; 1 or 2 blocks per stage) and two NC-column accumulators in
// tensor memory.  Partial tiles are kept as FP32 column quads (16 bytes per
// row and 4 columns).  The finishing CTA adds them in segment order: from its
// idle ring, bulk-copied there, when the tile is its last segment and they
// fit, else four segments' quads at a time from L2; for its last tile, warps
// 0-3 (done with their own roles) take the odd 16-column chunks.  With at
// least two CTAs per tile the grid is a whole multiple of the tile count.
// Row ranges (DG_SPLITK_ROWS=1): when N fits 128 rows per SM, a tile may
// instead be a range of tile_rows = ceil(N / SMs) rows, one CTA per range
// over the whole of K (grid = tiles): every SM streams the same share of B
// with no tile split, so no partial tile, workspace or finishing pass.  TMA
// loads tile_rows rows of B per K block; the MMA still spans 128 rows, and
// the accumulator rows past tile_rows (stale shared memory) are never
// stored.  Measured on GB300 no faster than 128-row tiles at the decode QKV
// shape (16 x 12288 x 4096: 11.48 against 11.58 us) and much slower for
// short ranges over a long K (16 x 4096 x 11008, 27 rows per CTA: 22.1
// against 11.2 us, too few bytes per box in flight), so not the default.
// Launch overlap: before its
// dependency wait a CTA prefetches its first ring of B into L2, and right
// after it the grid lets the next kernel take over SMs as CTAs exit, so the
// start-up of one launch hides in the straggling tail of the one before.
// All mbarrier waits are bounded as in the other GEMMs.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "gemm_common.cuh"
#include "gemm_skinny_kernel.cuh"

namespace dg {

void plan_skinny(int64_t M, int64_t N, int64_t K, bool fp16_in, int sm_count, dg_plan* p) {
    const int bk = fp16_in ? 64 : 128;
    const int nc = nc_for(M);
    // rows of B per tile: 128, or DG_SPLITK_TILE_ROWS (sweeps; the MMA still
    // spans 128 rows and the rows past the tile are not stored)
    const int tile_rows = knobs().splitk_tile_rows;
    const int64_t tiles = (N + tile_rows - 1) / tile_rows;
    const int64_t units = tiles * ((K + bk - 1) / bk);
    p->block_m = nc;
    p->block_n = tile_rows;
    p->block_k = bk;
    p->stages = ring_kblocks(nc) / splitk_kps();
    // Row ranges (see the file comment): N within 128 rows per SM.
    const int64_t range = (N + sm_count - 1) / sm_count;
    const int rows_knob = knobs().splitk_rows;
    if (range <= kRows && knobs().splitk_grid == 0 && rows_knob == 1) {
        p->block_n = static_cast<int>(range);
        p->tiles = static_cast<int>((N + range - 1) / range);
        p->grid = p->tiles;
        p->smem_bytes = smem_for_nc(nc);
        return;
    }
    p->tiles = static_cast<int>(tiles);
    // With room for at least two CTAs per tile, launch a whole multiple of
    // the tile count, so every CTA covers the same fraction of one tile (one
    // segment each, the same number of segments in every tile); otherwise
    // every SM, with ranges that cross tile edges.
    const int64_t per_tile = sm_count / tiles;
    const int64_t g = per_tile >= 2 ? per_tile * tiles : sm_count;
    p->grid = static_cast<int>(units < g ? units : g);
    if (const int64_t g = knobs().splitk_grid) {   // sweeps: CTAs per launch
        if (g <= sm_count && g <= units) p->grid = static_cast<int>(g);
    }
    p->smem_bytes = smem_for_nc(nc);
}

cudaError_t launch_gemm_skinny(const TcLaunch& L, float* partials, uint32_t* counts, int max_cols,
                               cudaStream_t s) {
    const int rows = L.plan->block_n;
    if (L.M < 1 || L.M > kSplitkMaxCols || nc_for(L.M) > max_cols || rows < 1 || rows > kRows ||
        L.plan->tiles > kSkinnyMaxTiles ||
        static_cast<int64_t>(L.plan->tiles) * rows < L.N)
        return cudaErrorInvalidValue;
    // Tiles may be split over CTAs (workspace needed) unless there is one CTA
    // per tile (grid = tiles: each CTA's range is exactly one tile).
    if (L.plan->grid != L.plan->tiles && (partials == nullptr || counts == nullptr))
        return cudaErrorInvalidValue;
    if (L.epi != nullptr) return launch_gemm_skinny_fused(L, partials, counts, s);
    return L.fp16_in ? launch_in<true, false>(L, partials, counts, s)
                     : launch_in<false, false>(L, partials, counts, s);
}

}  // namespace dg
