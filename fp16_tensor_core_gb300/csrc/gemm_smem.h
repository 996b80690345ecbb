// gemm_smem.h -- sizes in shared memory of the tiled GEMMs, and where the
// CTA-pair kernel puts what it finishes a tile with.  Plain C++, so that a
// host program can go through every width.
#pragma once

namespace dg {

// Shared memory per CTA available to a kernel (227 KB).
constexpr int kSmemLimit = 232448;
constexpr int kBKBytes = 128;     // one 128-byte swizzle row of K per stage
constexpr int kBoxBytes = 2048;   // an epilogue box: 32 x 32 two-byte elements (E4M3 uses half)

// The fused tiled kernels have eight epilogue warps (4-11): two take the 32
// columns of a chunk in turn, so that one's arithmetic runs while the other
// waits for its loads and stores.  With four the epilogue was longer than the
// main loop at K = 4096 (4096 x 11008 x 4096 E4M3, SiLU and bias: 139 us,
// with eight 128).
constexpr int epilogue_warps(bool fused) { return fused ? 8 : 4; }

// What a fused epilogue warp holds of its chunks of a tile in shared memory:
// each column's scale of B and bias, as pairs of columns {scale, scale, bias,
// bias} so that one 16-byte read serves two columns.
constexpr int kColumnFloats = 64;   // of a chunk
constexpr int fused_chunks(int bn) { return (bn / 32 + 1) / 2; }   // a warp's, at most
constexpr int columns_bytes(int bn) { return epilogue_warps(true) * fused_chunks(bn) * kColumnFloats * 4; }

// ---- CTA pairs: 256 x bn tiles, 128 rows of A and half of B's rows per CTA

constexpr int kPairRows = 128;   // of a CTA
constexpr int kPairMaxParts = 4; // K ranges of a split tile, at most

// Staging boxes of the epilogue: one 32 x 32 box per epilogue warp.
constexpr int pair_staging_bytes(bool fused) { return epilogue_warps(fused) * kBoxBytes; }
constexpr int pair_stage_bytes(int bn, int kps) { return kps * (kPairRows + bn / 2) * kBKBytes; }

// Stage count: what fits in 227 KB beside the barrier block (1 KB, keeping
// the staging boxes 1024-byte aligned), the staging boxes and a fused
// epilogue's columns, at most 8 (4 with two K blocks per stage).
constexpr int pair_stages_for(int bn, int kps = 1, bool fused = false) {
    const int st = (kSmemLimit - 1024 - 1024 - pair_staging_bytes(fused) - (fused ? columns_bytes(bn) : 0)) /
                   pair_stage_bytes(bn, kps);
    return st > 8 / kps ? 8 / kps : st;
}
constexpr int pair_ring_bytes(int bn, int kps, bool fused) {
    return pair_stages_for(bn, kps, fused) * pair_stage_bytes(bn, kps);
}

// On a CTA's last item its ring is idle.  It then holds, one behind another,
// the partial tiles of a split tile's other parts (FP32, kPairRows x bn each)
// and the tile's output boxes -- when they all fit; else the partial tiles are
// read from L2 and the boxes start at 0.
constexpr int pair_partial_bytes(int bn) { return kPairRows * bn * 4; }
constexpr int pair_boxes_bytes(int bn) { return kPairRows / 32 * (bn / 32) * kBoxBytes; }
constexpr bool pair_parts_in_ring(int ring_bytes, int bn, int parts) {
    return (parts - 1) * pair_partial_bytes(bn) + pair_boxes_bytes(bn) <= ring_bytes;
}
// Where the boxes begin behind the partial tiles of the other parts.
constexpr int pair_boxes_at(int bn, int parts) { return (parts - 1) * pair_partial_bytes(bn); }

}  // namespace dg
