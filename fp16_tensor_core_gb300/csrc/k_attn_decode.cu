// k_attn_decode.cu -- attention of a few new tokens per request over the
// paged E4M3 key/value cache, with an optional prefix shared by the batch.
//
// For one query row and the tokens t it sees, with codes kc, vc and scales
// sk, sv of one cached row each (k_t = sk_t kc_t, v_t = sv_t vc_t):
//   x_t = scale sk_t (q . kc_t)                the score
//   w_t = exp(x_t + ln sv_t - m),  m = max_t (x_t + ln sv_t) - 15 ln 2
//   acc = sum_t w_t vc_t,          l = sum_t w_t / sv_t
//   o   = acc / l,                 lse = m + ln l
// The value's scale sits inside the exponential, so a weight costs one
// exponential.  It goes to the second product as FP16, rounded to 11 bits
// (more would take a second FP16 operand and twice the MMAs; against codes
// of 4 bits they are not what limits an output); l takes it before that
// rounding.  The reference m lies 2^15 below the row's largest contribution,
// so that weights use FP16's whole range: one below 2^-29 of the largest
// keeps an absolute error of 2^-40 of it, and a long tail behind a single
// heavy token is not lost (with m at the largest, tokens below 2^-25 of it
// were).  E4M3 codes are exact in FP16; sums, maxima and the state are FP32.
//
// A cached element is read once and takes 4 flop per row, so for the few
// rows that share a key head the kernel is bound by HBM: it streams codes
// through shared memory with asynchronous copies and takes both products on
// warp-level MMAs with the cached operand on their 16-row side and 8 query
// rows on the other (tcgen05's 128 rows would be idle).
//
// Split: all (request, key head, row tile) units are laid end to end in
// 32-token tiles, with room for the cost of taking up a unit before each,
// and every warp of the grid takes an equal run of them, so
// ragged lengths balance and one long cache spreads over all SMs.  A warp
// writes the units that lie inside its run; the pieces of a unit that
// crosses warps are joined in shared memory, and those of a unit that
// crosses blocks through scratch by a second, small kernel.  Every join goes
// in token order: results do not depend on timing.
//
// Measured: 3 requests of up to 120001 tokens, 32/8 heads of 128: 85 us
// (5.5 TB/s, 0.82 of a copy); 64 of up to 4099: 55 us (0.75).  Heads of 256:
// 178 (0.77) and 111 (0.73).  The loop runs
// at what HBM gives; the rest is the start (lengths, pages, first tiles: 5
// us), the join (4), and SMs that end at different times: four groups of ten
// SMs get an eighth less of the bandwidth than the others and end 8 us later,
// always the same ones.  Runs handed out as warps become free would even that
// out, but each piece more costs a state (as many bytes as a quarter of a
// tile) to write and join, which takes the gain back.
//
// Units of 8 or 16 rows read and convert the cache once each, so many rows a
// key head are this kernel's weak side: a prompt's own 2048 tokens as q_len
// (32/8 heads of 128) 410 us, 0.04 of the tensor rate; 96 requests behind
// 2000 and 12000 shared tokens with 256-wide heads, which the tcgen05 kernel
// does not hold, 100 and 351 us (38 and 58 with heads of 128 there).
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "attn_common.cuh"
#include "dg_internal.h"
#include "dg_ptx.cuh"

namespace dg {
namespace {

constexpr int kTile = 32;        // tokens per warp step
constexpr int kMaxUnitRows = 16; // query rows of a unit
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kHeadroom = 15.0f;   // log2 of the largest weight (FP16 ends at 2^16)

struct AttnArgs {
    const uint16_t* q;
    int64_t q_ts, q_hs;
    uint16_t* out;
    int64_t o_ts, o_hs;
    float* lse;                // [tokens, q_heads] or null
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    int64_t pages;
    int kv_heads;
    int page_shift;
    const int32_t* page_table; // row per request, or the prefix's pages
    int64_t table_stride;
    int max_len;               // tokens a row of page_table can name
    const int32_t* kv_lens;    // null: every request has max_len tokens
    int batch;
    int q_len;
    int group;                 // query heads per key head
    int rows;                  // q_len * group
    int row_tiles;
    int ranks_log2;            // of the blocks (a cluster) that share a unit, where units are taken whole
    int q_heads;
    bool causal;
    bool behind;               // started behind the kernel that leaves a.prefix, which ends later
    float scale_log2;          // softmax scale * log2(e)
    float* slots;              // two states of kRows rows per block
    int4* crossings;           // per block: the unit that goes on past it
    const float* prefix;       // states of the prefix, per (token, head), or null
    float* states;             // where this call leaves states instead of outputs, or null
    uint32_t* status;
};

constexpr int kMaxRanks = 8;   // blocks of a cluster

// Reads of another block's shared memory (addresses of map_to_rank).
__device__ __forceinline__ float2 load_peer2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 load_peer4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
// The transpose of an 8 x 8 matrix of 16-bit values held two to a lane (row
// lane / 4, columns 2 (lane % 4), + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shapes per head width D and number of 8-row tiles NT.  A lane with
// lane % 4 == c holds dims c * kDims .. of each kSpan-wide part of the head
// in the first product, one with lane / 4 == g dims g * kSpan / 8 .. in the
// second.
template <int D, int NT, int W = D == 256 ? 4 : 8>
struct Shape {
    static constexpr int kRows = 8 * NT;             // query rows per unit
    static constexpr int kWarps = W;                 // of a block
    static constexpr int kPerSm = (D == 128 && NT == 2 ? 8 : D == 256 ? 8 : 16) / W;   // resident blocks (registers)
    static constexpr int kStages = D == 64 || (D == 128 && NT == 2) ? 2 : 1;
    static constexpr int kParts = D == 256 ? 2 : 1;
    static constexpr int kSpan = D / kParts;         // 64 or 128
    static constexpr int kDims = kSpan / 4;          // 16 or 32
    static constexpr int kTileBytes = kTile * D;     // keys or values of a tile
    static constexpr int kState = D + 4;             // m, l, 2 unused, acc[D]
    static constexpr int kStashBytes = kRows * kState * 4;
    // per warp: stages of keys, of values, of scales; log2 and reciprocal of
    // the value scales in use
    static constexpr int kScaleAt = 2 * kStages * kTileBytes;
    static constexpr int kLogAt = kScaleAt + kStages * 2 * kTile * 4;
    static constexpr int kRingBytes = kLogAt + 2 * kTile * 4;
    // a run's last piece is stashed over the warp's (drained) stages
    static_assert(kRingBytes >= kStashBytes, "a tail piece fits the ring");
    static constexpr int kSmem = kWarps * (kRingBytes + kStashBytes);
};

// Row r (0 .. 31) of a tile's MMA operands is token 4 (r % 8) + r / 8, so
// that a lane's four tokens are neighbours (their scales are one 16-byte
// read).  Byte offset of 16-byte chunk `chunk` of token t in a tile: the
// chunks of a 128-byte line are permuted by the token so that neither
// product's reads meet in a bank (a quarter warp reads 4 chunks of tokens t
// and t + 4 of the keys, and 2 chunks of tokens t, t + 8, t + 16, t + 24 of
// the values).
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int t, int chunk) {
    if constexpr (D == 64)
        return (t >> 1) * 128 +
               ((((t & 1) * 4 + chunk) ^ ((((t >> 3) & 3) << 1) ^ (t & 4))) * 16);
    else
        return t * D + (chunk >> 3) * 128 + (((chunk & 7) ^ ((t >> 2) & 7)) * 16);
}

// A place in the flat order of tiles.  Units are laid out with kUnitCost
// tiles' worth of room before their first tile: about what a warp spends on
// taking up a unit and leaving it.
constexpr int kUnitCost = 1;
struct Cursor {
    int b;       // request
    int h, rt;   // unit: key head, row tile
    int tile;
    int ntile;   // tiles of the request's units
    int len;     // its tokens
    int stop;    // the run's end in this unit: its last tile + 1
};

// Where a row's result goes and what it is joined with: factors for its
// partial sums, so that out = x * wx (+ prefix state * wp).
struct RowEnd {
    float* state;          // raw state wanted: there
    const float* prefix;   // state to join with, or null
    uint16_t* out;
    float wx, wp;
};

template <int D>
__device__ __forceinline__ RowEnd row_end(const AttnArgs& a, int64_t token, int head, float m, float l,
                                          bool leader) {
    RowEnd e;
    const int64_t row = token * a.q_heads + head;
    e.state = nullptr;
    e.prefix = nullptr;
    if (a.states != nullptr) {
        e.state = a.states + row * (D + 4);
        if (leader) *reinterpret_cast<float2*>(e.state) = make_float2(m, l);
        return e;
    }
    e.out = a.out + token * a.o_ts + head * a.o_hs;
    e.wx = 1.0f;
    e.wp = 0.0f;
    if (a.prefix != nullptr) {
        e.prefix = a.prefix + row * (D + 4);
        const float2 p = *reinterpret_cast<const float2*>(e.prefix);
        const float top = fmaxf(m, p.x);
        const float base = top == -INFINITY ? 0.0f : top;
        e.wx = ex2(m - base);
        e.wp = ex2(p.x - base);
        m = top;
        l = e.wx * l + e.wp * p.y;
    }
    const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
    e.wx *= inv;
    e.wp *= inv;
    if (leader && a.lse != nullptr)
        a.lse[row] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
    return e;
}

// Dims d .. d + 3 of a row.
template <int D, bool kFp16>
__device__ __forceinline__ void emit4(const RowEnd& e, int d, float4 x) {
    if (e.state != nullptr) {
        *reinterpret_cast<float4*>(e.state + 4 + d) = x;
        return;
    }
    x = scaled(x, e.wx);
    if (e.prefix != nullptr)
        x = plus_scaled(x, e.wp, *reinterpret_cast<const float4*>(e.prefix + 4 + d));
    uint2 o;
    if constexpr (kFp16) {
        o = make_uint2(f32x2_to_f16x2(x.x, x.y), f32x2_to_f16x2(x.z, x.w));
    } else {
        o = make_uint2(f32x2_to_bf16x2(x.x, x.y), f32x2_to_bf16x2(x.z, x.w));
    }
    *reinterpret_cast<uint2*>(e.out + d) = o;
}

// Row r (0 .. rows-1) of request b's key head h: its token and query head.
__device__ __forceinline__ void row_place(const AttnArgs& a, int b, int h, int r, int64_t* token,
                                          int* head) {
    const int i = r / a.group;
    *token = static_cast<int64_t>(b) * a.q_len + i;
    *head = h * a.group + (r - i * a.group);
}

// Tokens of request b; a length the page table cannot hold counts as none.
__device__ __forceinline__ int request_len(const AttnArgs& a, int b) {
    if (a.kv_lens == nullptr) return a.max_len;
    const int n = a.kv_lens[b];
    if (n < 0 || n > a.max_len) {
        atomicOr(a.status, kStatusBadArgument);
        return 0;
    }
    return n;
}

// cum[b] = room of one unit of each of requests 0 .. b-1 (its tiles and the
// unit's cost; nothing for an empty request), and the requests' lengths;
// over the whole block.
template <int kThreads>
__device__ __forceinline__ void scan_tiles(const AttnArgs& a, uint32_t* cum, int* lens, uint32_t* warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t carry = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        const int len = b < a.batch ? request_len(a, b) : 0;
        if (b < a.batch) lens[b] = len;
        uint32_t n = (len + kTile - 1) / kTile;
        if (n > 0) n += kUnitCost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, n, o);
            if (lane >= o) n += up;
        }
        if (lane == 31) warp_sum[warp] = n;
        __syncthreads();
        uint32_t before = carry, all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += warp_sum[w];
            all += warp_sum[w];
        }
        if (b < a.batch) cum[b + 1] = before + n;
        carry += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) cum[0] = 0;
    __syncthreads();
}

// a / b for non-negative a, in 32 bits where they suffice (as they do but for
// the largest calls): a 64-bit division is a hundred instructions.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 31) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// Room a warp takes: an equal share of all, at least one tile beside a
// unit's cost.
__device__ __forceinline__ int64_t room_per_warp(int64_t total, int64_t warps) {
    return max(static_cast<int64_t>(kUnitCost + 1), quotient(total + warps - 1, warps));
}

// The request whose room holds position f (which is below the total), by a
// whole warp: 32 places a step.
__device__ __forceinline__ int find_request(const uint32_t* cum, int batch, int64_t units, int64_t f, int lane) {
    int lo = 0, n = batch;   // it is one of lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const bool starts_before = lane * step < n && static_cast<int64_t>(cum[lo + lane * step]) * units <= f;
        const int k = 31 - __clz(__ballot_sync(0xFFFFFFFFu, starts_before));   // lane 0's always does
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// kWhole: every block, or cluster of blocks, takes one whole unit
// instead (its warps equal runs of the unit's tiles): nothing to search for,
// and the blocks' pieces meet in shared memory, without another launch.
template <int D, int NT, int W, bool kFp16, bool kWhole>
__global__ void __launch_bounds__(W * 32, Shape<D, NT, W>::kPerSm)
attn_split_kernel(const AttnArgs a) {
    using S = Shape<D, NT, W>;
    constexpr int kWarps = S::kWarps, kThreads = kWarps * 32, kStages = S::kStages, kRows = S::kRows;
    constexpr int kParts = D > 128 ? 2 : 1;   // float4s of a row a lane
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t warp_sum[kWarps];
    __shared__ int piece_b[2 * kWarps], piece_unit[2 * kWarps];   // request (-1: no piece), unit
    uint32_t* cum = reinterpret_cast<uint32_t*>(smem + S::kSmem);
    int* lens = reinterpret_cast<int*>(cum + a.batch + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    // A prefix's kernel reads nothing of the one before it but a.prefix.
    if (!a.behind) pdl_wait();
    pdl_launch_dependents();
    const int units = a.kv_heads * a.row_tiles;
    Cursor unit;                // kWhole: this block's
    int64_t run, block0, block1, f0, f1;   // room, or the unit's tiles
    int rank = 0;               // kWhole: this block's in its cluster
    if constexpr (kWhole) {
        int u = static_cast<int>(blockIdx.x);
        rank = u & ((1 << a.ranks_log2) - 1);
        u >>= a.ranks_log2;
        unit.b = u / units;
        u -= unit.b * units;
        unit.h = a.row_tiles == 1 ? u : u / a.row_tiles;
        unit.rt = u - unit.h * a.row_tiles;
        unit.len = request_len(a, unit.b);
        unit.ntile = (unit.len + kTile - 1) / kTile;
        // One tile has one warp's row ends, none at all is written here: by
        // the first block alone.
        if (unit.ntile <= 1 && rank > 0) return;
        if (unit.ntile == 0) {
            const int r0 = unit.rt * kRows;
            for (int i = threadIdx.x; i < min(kRows, a.rows - r0) * (D / 4); i += kThreads) {
                const int r = i / (D / 4), d = 4 * (i % (D / 4));
                int64_t token;
                int head;
                row_place(a, unit.b, unit.h, r0 + r, &token, &head);
                emit4<D, kFp16>(row_end<D>(a, token, head, -INFINITY, 0.0f, d == 0), d, make_float4(0, 0, 0, 0));
            }
            return;
        }
        run = ((unit.ntile + kWarps - 1) / kWarps + (1 << a.ranks_log2) - 1) >> a.ranks_log2;
        block0 = min(static_cast<int64_t>(unit.ntile), rank * kWarps * run);
        block1 = min(static_cast<int64_t>(unit.ntile), block0 + kWarps * run);
        f0 = min(block1, block0 + warp * run);
        f1 = min(block1, f0 + run);
    } else {
        scan_tiles<kThreads>(a, cum, lens, warp_sum);
        const int64_t total = static_cast<int64_t>(cum[a.batch]) * units;
        run = room_per_warp(total, static_cast<int64_t>(gridDim.x) * kWarps);
        block0 = min(total, static_cast<int64_t>(blockIdx.x) * kWarps * run);
        block1 = min(total, block0 + kWarps * run);
        f0 = min(total, block0 + warp * run);
        f1 = min(total, f0 + run);

        // Requests without a token of their own: nothing below reaches them.
        // A warp a row (rows are counted in 32 bits, their elements are not).
        for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
            if (cum[b + 1] != cum[b]) continue;
            for (int row = warp; row < a.q_len * a.q_heads; row += kWarps) {
                const int i = row / a.q_heads;
                const RowEnd e = row_end<D>(a, static_cast<int64_t>(b) * a.q_len + i, row - i * a.q_heads, -INFINITY,
                                            0.0f, lane == 0);
                if (D >= 128 || 4 * lane < D) {
#pragma unroll
                    for (int k = 0; k < kParts; ++k) emit4<D, kFp16>(e, 4 * lane + 128 * k, make_float4(0, 0, 0, 0));
                }
            }
        }
    }

    uint8_t* mine = smem + warp * S::kRingBytes;
    const uint32_t ring = smem_addr(mine);
    float* logs = reinterpret_cast<float*>(mine + S::kLogAt);
    float* head_stash =
        reinterpret_cast<float*>(smem + kWarps * S::kRingBytes + warp * S::kStashBytes);
    float* tail_stash = reinterpret_cast<float*>(mine);
    if (lane == 0) piece_b[2 * warp] = piece_b[2 * warp + 1] = -1;

    if (f0 < f1) {
        // ---- the run's tiles: from the one at f0 up to the one at f1
        // Sets u.stop; whether u (at its unit's first tile of the run) is in the run.
        auto settle = [&](Cursor& u) {
            if constexpr (kWhole) {
                u.stop = static_cast<int>(f1);
                return u.tile < u.stop;
            }
            const int64_t tiles_at = static_cast<int64_t>(cum[u.b]) * units +
                                     static_cast<int64_t>(u.h * a.row_tiles + u.rt) * (u.ntile + kUnitCost) + kUnitCost;
            u.stop = static_cast<int>(min(max(f1 - tiles_at, static_cast<int64_t>(0)), static_cast<int64_t>(u.ntile)));
            return u.tile < u.stop;
        };
        // The next tile; whether it is in the run.
        auto advance = [&](Cursor& u) {
            if (++u.tile < u.stop) return true;
            if (kWhole || u.stop < u.ntile) return false;
            u.tile = 0;
            if (++u.rt == a.row_tiles) {
                u.rt = 0;
                if (++u.h == a.kv_heads) {
                    u.h = 0;
                    do ++u.b; while (u.b < a.batch && cum[u.b + 1] == cum[u.b]);
                    if (u.b == a.batch) return false;
                    u.ntile = static_cast<int>(cum[u.b + 1] - cum[u.b]) - kUnitCost;
                    u.len = lens[u.b];
                }
            }
            return settle(u);
        };
        Cursor at;
        if constexpr (kWhole) {
            at = unit;
            at.tile = static_cast<int>(f0);
        } else {
            at.b = find_request(cum, a.batch, units, f0, lane);
            const int room = static_cast<int>(cum[at.b + 1] - cum[at.b]);
            at.ntile = room - kUnitCost;
            at.len = lens[at.b];
            const int64_t in_b = f0 - static_cast<int64_t>(cum[at.b]) * units;
            const int unit = static_cast<int>(quotient(in_b, room));
            at.tile = max(0, static_cast<int>(in_b - static_cast<int64_t>(unit) * room) - kUnitCost);
            at.h = a.row_tiles == 1 ? unit : unit / a.row_tiles;
            at.rt = unit - at.h * a.row_tiles;
        }
        bool running = settle(at);
        Cursor in = at;

        // ---- loads: this lane's token of the tile to load next
        const int in_page = (1 << a.page_shift) - 1;
        constexpr int kPerRow = D / 16, kPerStep = 32 / kPerRow;   // 16-byte copies of a row; rows a step
        const int chunk = lane % kPerRow, row_in = lane / kPerRow;
        // The page is asked for when the tile's turn comes up and first looked
        // at when its keys are loaded, a product later.
        int page = -1;
        int64_t token_row = -1;   // its row in the cache, or -1
        auto find_page = [&]() {
            const int t = in.tile * kTile + lane;
            page = t < in.len ? a.page_table[in.b * a.table_stride + (t >> a.page_shift)] : -1;
        };
        auto find_row = [&]() {
            const int t = in.tile * kTile + lane;
            token_row = -1;
            if (page >= 0 && page < a.pages) {
                token_row = ((static_cast<int64_t>(page) * a.kv_heads + in.h) << a.page_shift) + (t & in_page);
            } else if (t < in.len) {
                atomicOr(a.status, kStatusBadArgument);
            }
        };
        auto load_codes = [&](const uint8_t* codes, uint32_t base) {
            if (a.page_shift >= 5 && in.tile * kTile + kTile <= in.len) {
                // a whole tile inside one page: one address for all of it
                const int64_t first = __shfl_sync(0xFFFFFFFFu, token_row, 0);
                const uint8_t* p = codes + (max(first, static_cast<int64_t>(0)) + row_in) * D + chunk * 16;
                const uint32_t n = first < 0 ? 0 : 16;
#pragma unroll
                for (int i = 0; i < kTile / kPerStep; ++i)
                    cp_async16(base + chunk_at<D>(i * kPerStep + row_in, chunk), p + i * kPerStep * D, n);
            } else {
#pragma unroll
                for (int i = 0; i < kTile / kPerStep; ++i) {
                    const int t = i * kPerStep + row_in;
                    const int64_t r = __shfl_sync(0xFFFFFFFFu, token_row, t);
                    cp_async16(base + chunk_at<D>(t, chunk),
                               codes + max(r, static_cast<int64_t>(0)) * D + chunk * 16, r < 0 ? 0 : 16);
                }
            }
        };
        auto load_keys = [&](int stage) {   // and both scales
            find_row();
            load_codes(a.k, ring + stage * S::kTileBytes);
            const uint32_t sc = ring + S::kScaleAt + stage * (2 * kTile * 4) + lane * 4;
            const int64_t r = max(token_row, static_cast<int64_t>(0));
            cp_async4(sc, a.k_scale + r, token_row < 0 ? 0 : 4);
            cp_async4(sc + kTile * 4, a.v_scale + r, token_row < 0 ? 0 : 4);
        };
        auto load_values = [&](int stage) {
            load_codes(a.v, ring + (kStages + stage) * S::kTileBytes);
        };

        // This unit's queries as the first product's B operand (row 8 n + g
        // of the unit), and per row 8 n + 2c + i of this lane's scores:
        uint32_t qb[NT][D / 16][2];
        float qscale[NT][2];      // factor from MMA sums to base-2 scores
        int seen[NT][2];          // tokens the row sees
        float m[NT][2], l[NT][2]; // running reference; this lane's part of l
        float acc[D / 16][NT][4]; // [.][n][i]: dim pair's first, [.][n][2 + i]: second
        int seen_min = 0, stage = 0, first_tile = 0;
        // The queries of unit `at`: rows 8 n + g.
        auto load_queries = [&](uint4 (&w)[NT][D / 32]) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = at.rt * kRows + 8 * n + g;
                int64_t token = 0;
                int head = 0;
                if (r < a.rows) row_place(a, at.b, at.h, r, &token, &head);
                const uint16_t* src = a.q + token * a.q_ts + head * a.q_hs + c * S::kDims;
#pragma unroll
                for (int p = 0; p < S::kParts; ++p)
#pragma unroll
                    for (int i = 0; i < S::kDims / 8; ++i)
                        w[n][p * (S::kDims / 8) + i] =
                            r < a.rows ? *reinterpret_cast<const uint4*>(src + p * S::kSpan + 8 * i)
                                       : make_uint4(0, 0, 0, 0);
            }
        };
        // Makes `at` the current unit, with those queries.
        auto take_up = [&](uint4 (&w)[NT][D / 32]) {
            first_tile = at.tile;
            seen_min = at.len;
            const int r0 = at.rt * kRows;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float mul = 1.0f, factor = a.scale_log2;
                if constexpr (!kFp16) {
                    uint32_t top = 0;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) top = max(top, top_abs_bf16(w[n][k]));
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    const PowerOfTwo p = query_scale(top);
                    mul = p.inverse;
                    factor *= p.value;
                }
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    const uint4 v = kFp16 ? w[n][k] : bf16_to_half8(w[n][k], mul);
                    // dims 8k + 2i, +1 of the lane's run: MMA step 2k + i/2
                    qb[n][2 * k][0] = v.x;
                    qb[n][2 * k][1] = v.y;
                    qb[n][2 * k + 1][0] = v.z;
                    qb[n][2 * k + 1][1] = v.w;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int rr = r0 + 8 * n + 2 * c + i;
                    qscale[n][i] = __shfl_sync(0xFFFFFFFFu, factor, 4 * (2 * c + i));
                    seen[n][i] = rr >= a.rows || !a.causal ? at.len
                                                           : max(0, at.len - a.q_len + 1 + rr / a.group);
                    seen_min = min(seen_min, seen[n][i]);
                    m[n][i] = -INFINITY;
                    l[n][i] = 0.0f;
                }
            }
            seen_min = __reduce_min_sync(0xFFFFFFFFu, seen_min);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][n][i] = 0.0f;
        };

        // ---- the first unit's queries travel with the first tiles
        bool more = running;   // `in` is a tile of this run
        {
            uint4 w[NT][D / 32];
            if (more) find_page();
            if (running) load_queries(w);
#pragma unroll 1
            for (int s = 0; s < kStages; ++s) {
                if (more) load_keys(s);
                cp_commit();
                if (more) {
                    load_values(s);
                    more = advance(in);
                    if (more) find_page();
                }
                cp_commit();
            }
            if (running) take_up(w);
        }
        bool fresh = false;

        while (running) {
            if (fresh) {
                uint4 w[NT][D / 32];
                load_queries(w);
                take_up(w);
                fresh = false;
            }

            // ---- scores: s[t][n][..] of tokens 4g + 2t (first two) and 4g + 2t + 1
            cp_wait<2 * kStages - 1>();
            __syncwarp();
            const uint32_t kb = ring + stage * S::kTileBytes, vb = ring + (kStages + stage) * S::kTileBytes;
            const float* sc = reinterpret_cast<const float*>(mine + S::kScaleAt + stage * (2 * kTile * 4));
            {   // this lane's token: log2 and reciprocal of the value's scale
                const float sv = sc[kTile + lane];
                const float safe = sv < 0x1p-100f ? 0x1p-100f : sv;
                logs[lane] = __log2f(safe);
                logs[kTile + lane] = rcp(safe);
            }
            const float4 sk4 = *reinterpret_cast<const float4*>(sc + 4 * g);
            float s[2][NT][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][n][i] = 0.0f;
#pragma unroll
                for (int p = 0; p < D / 64; ++p) {
                    const int ch = D == 64 ? c : 8 * (p >> 1) + 2 * c + (p & 1);
                    const uint4 x = lds128(kb + chunk_at<D>(4 * g + 2 * t, ch));
                    const uint4 y = lds128(kb + chunk_at<D>(4 * g + 2 * t + 1, ch));
                    const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t a0, a1, a2, a3;
                        codes_to_halves(wx[i], &a0, &a2);
                        codes_to_halves(wy[i], &a1, &a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816(s[t][n], a0, a1, a2, a3, qb[n][4 * p + i][0], qb[n][4 * p + i][1]);
                    }
                }
            }
            __syncwarp();   // the keys are read, the logs written
            if (more) load_keys(stage);
            cp_commit();

            // ---- softmax
            const float4 lg4 = *reinterpret_cast<const float4*>(logs + 4 * g);
            const float4 rs4 = *reinterpret_cast<const float4*>(logs + kTile + 4 * g);
            const float kk[4] = {sk4.x, sk4.y, sk4.z, sk4.w}, lg[4] = {lg4.x, lg4.y, lg4.z, lg4.w};
            const float rsv[4] = {rs4.x, rs4.y, rs4.z, rs4.w};
            const int t0 = at.tile * kTile + 4 * g;   // this lane's tokens: t0 .. t0 + 3
            const bool masked = at.tile * kTile + kTile > seen_min;
            float top[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float& y = s[q >> 1][n][2 * (q & 1) + i];
                        // both factors first: the sum times a large one alone could pass FP32
                        y = fmaf(y, kk[q] * qscale[n][i], lg[q]);
                    }
                    if (masked) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (t0 + q >= seen[n][i]) s[q >> 1][n][2 * (q & 1) + i] = -INFINITY;
                    }
                    top[n][i] = fmaxf(fmaxf(s[0][n][i], s[0][n][2 + i]), fmaxf(s[1][n][i], s[1][n][2 + i]));
                }
            bool grew = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[n][i] = fmaxf(top[n][i], __shfl_xor_sync(0xFFFFFFFFu, top[n][i], 4));
                    top[n][i] = fmaxf(top[n][i], __shfl_xor_sync(0xFFFFFFFFu, top[n][i], 8));
                    top[n][i] = fmaxf(top[n][i], __shfl_xor_sync(0xFFFFFFFFu, top[n][i], 16));
                    // rounded up: no weight passes 2^kHeadroom
                    top[n][i] = __fadd_ru(top[n][i], -kHeadroom);
                    grew |= top[n][i] > m[n][i];
                }
            if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float to = fmaxf(m[n][i], top[n][i]);
                        const float by = to == -INFINITY ? 1.0f : ex2(m[n][i] - to);
                        m[n][i] = to;
                        l[n][i] *= by;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            acc[j][n][i] *= by;
                            acc[j][n][2 + i] *= by;
                        }
                    }
            }
            // weights, turned from (token, row) to the second product's B
            // operand (row, token pair)
            uint32_t wt[2][NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float w[4][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float base = m[n][i] == -INFINITY ? 0.0f : m[n][i];
                    float part = 0.0f;
#pragma unroll
                    for (int q = 0; q < 4; ++q) w[q][i] = ex2(s[q >> 1][n][2 * (q & 1) + i] - base);
                    if (masked) {   // a token that a row does not see adds nothing, whatever its scale holds
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (t0 + q < seen[n][i]) part = fmaf(w[q][i], rsv[q], part);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) part = fmaf(w[q][i], rsv[q], part);
                    }
                    l[n][i] += part;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    wt[q >> 1][n][q & 1] = transpose8x8(f32x2_to_f16x2(w[q][0], w[q][1]));
            }

            // ---- values: k columns 2c, 2c + 1 of MMA t are tokens 8c + 2t, 8c + 4 + 2t,
            // columns 2c + 8, + 9 the tokens after them; dims of chunk g
            cp_wait<2 * kStages - 1>();
            __syncwarp();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tok = 8 * c + 2 * t;
                auto words = [&](int j, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
                    uint32_t p[4], q[4];   // dims of bytes 0..3: token pairs 0, 1 and 2, 3
                    codes_to_halves(__byte_perm(x0, x1, 0x5140), &p[0], &p[1]);
                    codes_to_halves(__byte_perm(x0, x1, 0x7362), &p[2], &p[3]);
                    codes_to_halves(__byte_perm(x2, x3, 0x5140), &q[0], &q[1]);
                    codes_to_halves(__byte_perm(x2, x3, 0x7362), &q[2], &q[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816(acc[j][n], p[0], p[1], q[0], q[1], wt[t][n][0], wt[t][n][1]);
                        mma16816(acc[j + 1][n], p[2], p[3], q[2], q[3], wt[t][n][0], wt[t][n][1]);
                    }
                };
                if constexpr (D == 64) {
                    const int ch = g >> 1, part = (g & 1) * 8;
                    const uint2 x0 = lds64(vb + chunk_at<D>(tok, ch) + part);
                    const uint2 x1 = lds64(vb + chunk_at<D>(tok + 4, ch) + part);
                    const uint2 x2 = lds64(vb + chunk_at<D>(tok + 1, ch) + part);
                    const uint2 x3 = lds64(vb + chunk_at<D>(tok + 5, ch) + part);
                    words(0, x0.x, x1.x, x2.x, x3.x);
                    words(2, x0.y, x1.y, x2.y, x3.y);
                } else {
#pragma unroll
                    for (int p = 0; p < S::kParts; ++p) {
                        const uint4 x0 = lds128(vb + chunk_at<D>(tok, 8 * p + g));
                        const uint4 x1 = lds128(vb + chunk_at<D>(tok + 4, 8 * p + g));
                        const uint4 x2 = lds128(vb + chunk_at<D>(tok + 1, 8 * p + g));
                        const uint4 x3 = lds128(vb + chunk_at<D>(tok + 5, 8 * p + g));
                        words(8 * p, x0.x, x1.x, x2.x, x3.x);
                        words(8 * p + 2, x0.y, x1.y, x2.y, x3.y);
                        words(8 * p + 4, x0.z, x1.z, x2.z, x3.z);
                        words(8 * p + 6, x0.w, x1.w, x2.w, x3.w);
                    }
                }
            }
            __syncwarp();
            if (more) {
                load_values(stage);
                more = advance(in);
                if (more) find_page();
            }
            cp_commit();
            stage = stage + 1 == kStages ? 0 : stage + 1;

            // ---- the unit's (or the run's) end
            const bool unit_end = at.tile + 1 == at.ntile;
            const Cursor was = at;
            running = advance(at);
            if (unit_end || !running) {
                fresh = true;
                const int r0 = was.rt * kRows;
                const bool whole = unit_end && first_tile == 0;
                if (whole && a.behind) pdl_wait();
                // first piece of the run when its unit began before it, else the last one
                const bool is_head = !whole && first_tile != 0;
                float* stash = is_head ? head_stash : tail_stash;
                if (!whole && !is_head) {   // over the ring: nothing is in flight any more
                    cp_wait<0>();
                    __syncwarp();
                }
                if (!whole && lane == 0) {
                    piece_b[2 * warp + (is_head ? 0 : 1)] = was.b;
                    piece_unit[2 * warp + (is_head ? 0 : 1)] = was.h * a.row_tiles + was.rt;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 4);
                        l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 8);
                        l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 16);
                        const int rr = 8 * n + 2 * c + i;
                        if (r0 + rr >= a.rows) continue;
                        RowEnd e;
                        if (whole) {
                            int64_t token;
                            int head;
                            row_place(a, was.b, was.h, r0 + rr, &token, &head);
                            e = row_end<D>(a, token, head, m[n][i], l[n][i], g == 0);
                        } else {
                            e.state = stash + rr * S::kState;
                            if (g == 0) {
                                e.state[0] = m[n][i];
                                e.state[1] = l[n][i];
                            }
                        }
                        // dims of chunk g, two per MMA tile
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            const float4 x = make_float4(acc[2 * k][n][i], acc[2 * k][n][2 + i],
                                                         acc[2 * k + 1][n][i], acc[2 * k + 1][n][2 + i]);
                            const int part = k / (S::kSpan / 32), in_part = k % (S::kSpan / 32);
                            emit4<D, kFp16>(e, part * S::kSpan + g * (S::kSpan / 8) + 4 * in_part, x);
                        }
                    }
            }
        }
        cp_wait<0>();
    }
    __syncthreads();
    if (a.behind) pdl_wait();

    // ---- join the pieces of each unit, in warp (token) order.  Lane p of
    // every warp looks at piece p; a unit's pieces are neighbours among those
    // that exist, and its rows are dealt out over the warps.
    static_assert(2 * kWarps <= 32, "a lane per piece");
    const int my_b = lane < 2 * kWarps ? piece_b[lane] : -1;
    const int my_unit = my_b >= 0 ? piece_unit[lane] : 0;
    const uint32_t exist = __ballot_sync(0xFFFFFFFFu, my_b >= 0);
    const uint32_t below = exist & ((1u << lane) - 1u);
    const int prev = below != 0 ? 31 - __clz(below) : lane;
    const int prev_b = __shfl_sync(0xFFFFFFFFu, my_b, prev), prev_unit = __shfl_sync(0xFFFFFFFFu, my_unit, prev);
    uint32_t starts = __ballot_sync(0xFFFFFFFFu, my_b >= 0 && (below == 0 || prev_b != my_b || prev_unit != my_unit));
    const float* my_piece = reinterpret_cast<const float*>(
        (lane & 1) ? smem + (lane >> 1) * S::kRingBytes
                   : smem + kWarps * S::kRingBytes + (lane >> 1) * S::kStashBytes);
    // What lane p knows of the unit whose pieces begin with piece p.
    const bool is_start = (starts >> lane & 1u) != 0;
    int my_h = 0, my_r0 = 0, my_rows = 0, my_to = 2, my_n = 0;   // my_n: blocks from this one on
    if (is_start) {
        my_h = a.row_tiles == 1 ? my_unit : my_unit / a.row_tiles;
        my_r0 = (my_unit - my_h * a.row_tiles) * kRows;
        my_rows = min(kRows, a.rows - my_r0);
        if constexpr (!kWhole) {
            const int64_t room = cum[my_b + 1] - cum[my_b], per_block = kWarps * run;
            const int64_t u0 = static_cast<int64_t>(cum[my_b]) * units + my_unit * room, u1 = u0 + room;
            const bool begins = block0 <= u0 + kUnitCost, ends = u1 <= block1;
            if (!(begins && ends)) {
                // slot 1 when it goes on in a later block, 0 when it began in an earlier one
                my_to = begins ? 1 : 0;
                if (begins) my_n = static_cast<int>(quotient(u1 - 1, per_block)) - static_cast<int>(blockIdx.x) + 1;
            }
        }
    }
    if (!kWhole && warp == 0) {
        // what the joining kernel needs to know of this block's end
        const bool goes_on = is_start && my_to == 1;
        if (goes_on) a.crossings[blockIdx.x] = make_int4(my_b, my_unit, my_n, 0);
        if (!__any_sync(0xFFFFFFFFu, goes_on) && lane == 0) a.crossings[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    int turn = 0;   // (unit, row) pairs so far
    while (starts != 0) {
        const int p = __ffs(starts) - 1;
        starts &= starts - 1;
        const uint32_t upto = starts != 0 ? (starts & -starts) - 1u : 0xFFFFFFFFu;
        const uint32_t chain = exist & upto & ~((1u << p) - 1u);
        const int b = __shfl_sync(0xFFFFFFFFu, my_b, p), h = __shfl_sync(0xFFFFFFFFu, my_h, p);
        const int r0 = __shfl_sync(0xFFFFFFFFu, my_r0, p), rows = __shfl_sync(0xFFFFFFFFu, my_rows, p);
        const int to = __shfl_sync(0xFFFFFFFFu, my_to, p);
        const bool mine_too = (chain >> lane & 1u) != 0;
#pragma unroll 1
        for (int r = (warp - turn) & (kWarps - 1); r < rows; r += kWarps) {
            const float2 ml = mine_too ? reinterpret_cast<const float2*>(my_piece)[r * (S::kState / 2)]
                                       : make_float2(-INFINITY, 0.0f);
            float m = ml.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const float w = mine_too ? ex2(ml.x - (m == -INFINITY ? 0.0f : m)) : 0.0f;
            float l = mine_too ? w * ml.y : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
            float4 x[kParts];
#pragma unroll
            for (int k = 0; k < kParts; ++k) x[k] = make_float4(0, 0, 0, 0);
#pragma unroll 1
            for (uint32_t left = chain; left != 0; left &= left - 1) {
                const int q = __ffs(left) - 1;
                const float wq = __shfl_sync(0xFFFFFFFFu, w, q);
                const uint8_t* base = (q & 1) ? smem + (q >> 1) * S::kRingBytes
                                              : smem + kWarps * S::kRingBytes + (q >> 1) * S::kStashBytes;
                if (D >= 128 || 4 * lane < D) {
#pragma unroll
                    for (int k = 0; k < kParts; ++k)
                        x[k] = plus_scaled(x[k], wq, reinterpret_cast<const float4*>(base)[(r * S::kState + 4) / 4 + lane + 32 * k]);
                }
            }
            RowEnd e;
            if (kWhole && a.ranks_log2 > 0) {   // over the row of the first piece: its readers are these lanes
                e.state = reinterpret_cast<float*>(smem + (p == 1 ? 0 : kWarps * S::kRingBytes)) + r * S::kState;
                if (lane == 0) *reinterpret_cast<float2*>(e.state) = make_float2(m, l);
            } else if (to == 2) {
                int64_t token;
                int head;
                row_place(a, b, h, r0 + r, &token, &head);
                e = row_end<D>(a, token, head, m, l, lane == 0);
            } else {
                e.state = a.slots + ((2 * static_cast<int64_t>(blockIdx.x) + to) * kRows + r) * S::kState;
                if (lane == 0) *reinterpret_cast<float2*>(e.state) = make_float2(m, l);
            }
            if (D >= 128 || 4 * lane < D) {
#pragma unroll
                for (int k = 0; k < kParts; ++k) emit4<D, kFp16>(e, 4 * lane + 128 * k, x[k]);
            }
        }
        turn += rows;
    }
    if constexpr (kWhole) {
        if (a.ranks_log2 == 0 || unit.ntile <= 1) return;
        // ---- join the blocks' states in token order.  A block's first piece
        // is its first warp's: the tail of the unit's first run (over the
        // ring) in the first block, a head in the others.
        cluster_sync_all_diverged();
        const int blocks = static_cast<int>((unit.ntile + kWarps * run - 1) / (kWarps * run));   // with tiles
        const int r0 = unit.rt * kRows, rows = min(kRows, a.rows - r0);
#pragma unroll 1
        for (int r = rank * kWarps + warp; r < rows; r += kWarps << a.ranks_log2) {
            auto state_of = [&](int q) {
                return map_to_rank(smem + (q == 0 ? 0 : kWarps * S::kRingBytes) + r * S::kState * 4, q);
            };
            float2 ml = make_float2(-INFINITY, 0.0f);
            if (lane < blocks) ml = load_peer2(state_of(lane));
            float m = ml.x;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            m = __shfl_sync(0xFFFFFFFFu, m, 0);
            const float w = ex2(ml.x - (m == -INFINITY ? 0.0f : m));
            float l = w * ml.y;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
            l = __shfl_sync(0xFFFFFFFFu, l, 0);
            float4 x[kParts], y[kMaxRanks][kParts];
#pragma unroll
            for (int q = 0; q < kMaxRanks; ++q)
                if (q < blocks && (D >= 128 || 4 * lane < D)) {
#pragma unroll
                    for (int k = 0; k < kParts; ++k) y[q][k] = load_peer4(state_of(q) + 16 + 16 * (lane + 32 * k));
                }
#pragma unroll
            for (int k = 0; k < kParts; ++k) x[k] = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < kMaxRanks; ++q) {
                const float wq = __shfl_sync(0xFFFFFFFFu, w, q);
                if (q < blocks && (D >= 128 || 4 * lane < D)) {
#pragma unroll
                    for (int k = 0; k < kParts; ++k) x[k] = plus_scaled(x[k], wq, y[q][k]);
                }
            }
            int64_t token;
            int head;
            row_place(a, unit.b, unit.h, r0 + r, &token, &head);
            const RowEnd e = row_end<D>(a, token, head, m, l, lane == 0);
            if (D >= 128 || 4 * lane < D) {
#pragma unroll
                for (int k = 0; k < kParts; ++k) emit4<D, kFp16>(e, 4 * lane + 128 * k, x[k]);
            }
        }
        cluster_sync_all_diverged();   // until nobody reads this block's states
    }
}

// Joins the units that cross blocks: block x of the grid takes the unit that
// begins in block x of the split kernel and goes on past it, warp y one of
// its rows.
template <int D, int NT, bool kFp16>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnArgs a) {
    constexpr int kState = Shape<D, NT>::kState, kRows = Shape<D, NT>::kRows, kParts = D > 128 ? 2 : 1;
    pdl_wait();
    const int4 unit = a.crossings[blockIdx.x];   // request, number, blocks
    if (unit.x < 0) return;
    const int h = unit.y / a.row_tiles, r0 = (unit.y - h * a.row_tiles) * kRows;
    const int r = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r0 + r >= a.rows) return;
    int64_t token;
    int head;
    row_place(a, unit.x, h, r0 + r, &token, &head);
    // slot 1 of the first block, then slot 0 of each later one
    constexpr int64_t kBlock = 2 * kRows * kState;
    const float* first = a.slots + blockIdx.x * kBlock + (kRows + r) * kState;
    float4 x[kParts], y[kParts];
    float m, l;
    const bool live = 4 * lane < D;
    const float2 ml = *reinterpret_cast<const float2*>(first);
    if (live) {
#pragma unroll
        for (int k = 0; k < kParts; ++k) x[k] = *reinterpret_cast<const float4*>(first + 4 + 4 * lane + 128 * k);
    }
    join_states<D>(first + (kBlock - kRows * kState), kBlock, unit.z - 1, lane, &m, &l, y);
    const float top = fmaxf(m, ml.x), base = top == -INFINITY ? 0.0f : top;
    const float w0 = ex2(ml.x - base), w1 = ex2(m - base);
    const RowEnd e = row_end<D>(a, token, head, top, w0 * ml.y + w1 * l, lane == 0);
    if (live) {
#pragma unroll
        for (int k = 0; k < kParts; ++k)
            emit4<D, kFp16>(e, 4 * lane + 128 * k, plus_scaled(scaled(x[k], w0), w1, y[k]));
    }
}

// The end of a call whose prefix was cut into shares on the tensor cores: a
// row's shares, in token order, and the state of its own tokens (a.prefix;
// addition is the same either way).  One warp a row.
struct PrefixShares {
    const float* slots;   // per share, row tile and row
    int splits, row_tiles, tile_rows, rows;
};
template <int D, bool kFp16>
__global__ void __launch_bounds__(128) attn_prefix_join_kernel(const AttnArgs a, const PrefixShares p) {
    constexpr int kState = D + 4;
    static_assert(D <= 128, "a lane holds 4 dims");
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int r = static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5), h = blockIdx.y;
    if (r >= p.rows) return;
    const int rt = r / p.tile_rows;
    const int64_t stride = static_cast<int64_t>(p.row_tiles) * p.tile_rows * kState;   // from share to share
    const float* first = p.slots + ((static_cast<int64_t>(h) * p.splits * p.row_tiles + rt) * p.tile_rows +
                                    (r - rt * p.tile_rows)) * kState;
    float m, l;
    float4 x;
    join_states<D>(first, stride, p.splits, lane, &m, &l, &x);
    int64_t token;
    int head;
    row_place(a, 0, h, r, &token, &head);
    const RowEnd e = row_end<D>(a, token, head, m, l, lane == 0);
    if (4 * lane < D) emit4<D, kFp16>(e, 4 * lane, x);
}

// Most blocks of a launch: the two that an SM holds.  (A block spends 10 us
// on its start, its joins and its end, so more and smaller runs, handed to
// the SMs that are done first, cost more than their evenness gains: 3 x
// 120001 tokens 85 us with 2 blocks per SM, 97 with 3, 88 with 4.)
int attn_blocks(int sm_count) { return 2 * sm_count; }

// The crossings' room in floats.
int64_t crossing_floats(int sm_count) { return static_cast<int64_t>(attn_blocks(sm_count)) * 4; }

// Whole units, one per cluster of 1 << a.ranks_log2 blocks of W warps.
template <int D, int NT, int W, bool kFp16>
cudaError_t run_whole(const AttnArgs& a, int64_t units, cudaStream_t s) {
    const auto kernel = attn_split_kernel<D, NT, W, kFp16, true>;
    const cudaError_t e = allow_smem(kernel, Shape<D, NT, W>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_clusters(kernel, dim3(static_cast<unsigned>(units << a.ranks_log2)), dim3(W * 32), 1 << a.ranks_log2,
                           Shape<D, NT, W>::kSmem, s, a);
}

template <int D, int NT, bool kFp16>
cudaError_t run_split_nt(AttnArgs a, int sm_count, cudaStream_t s) {
    using S = Shape<D, NT>;
    a.row_tiles = (a.rows + S::kRows - 1) / S::kRows;
    // Whole units while a unit is at most four tiles a warp, by the page
    // table's width (the lengths are not known here), over clusters of as many
    // blocks as fit the GPU at once, until most warps have a single tile.
    // Measured with 32/8 heads of 128, us, whole units (blocks a cluster)
    // against equal runs: 1 x 300 tokens 6.7 (1) / 10.6, 1 x 1000 7.0 (4) /
    // 10.5, 1 x 8000 12.0 (8) / 14.5, 8 x 2000 11.3 (4) / 13.0, 16 x 2000
    // 15.2 (2) / 16.2, 64 x 1000 21.8 (1) / 23.1, 64 x 2000 (8 tiles a warp)
    // 36.2 (1) / 33.6.  Clusters past one wave lose: 64 x 400 16.5 (1), 29.6
    // (2), 51.5 (4).
    const int blocks = S::kPerSm * sm_count;
    const int64_t units = static_cast<int64_t>(a.batch) * a.kv_heads * a.row_tiles;
    const int64_t tiles = (static_cast<int64_t>(a.max_len) + kTile - 1) / kTile;
    int ranks = 1;
    for (a.ranks_log2 = 0; ranks < kMaxRanks && 2 * tiles > 3 * ranks * S::kWarps && units * ranks * 2 <= blocks;
         ++a.ranks_log2)
        ranks *= 2;
    if (tiles <= 4 * ranks * S::kWarps && units <= INT_MAX) {
        // More units than blocks at once: half as many warps a block, twice as
        // many blocks, whose starts and joins overlap (64 x 400 tokens 13.0
        // against 16.5 us, 64 x 1000 21.8 / 23.8; but 8 x 1000 9.2 / 8.7).
        if constexpr (S::kWarps == 8) {
            if (units > blocks) return run_whole<D, NT, 4, kFp16>(a, units, s);
        }
        return run_whole<D, NT, S::kWarps, kFp16>(a, units, s);
    }
    // Equal runs: 16 warps an SM, in two blocks, but 16-row units of 64-wide
    // heads in one (24 x 5 x 2500 tokens of 16/4 heads 22.7 / 23.8 us, 2 x 8 x
    // 30000 25.8 / 28.4; 8-row units 13.9 / 12.8 for 24 x 2500).
    using F = Shape<D, NT, D == 64 && NT == 2 ? 16 : S::kWarps>;
    const int run_blocks = F::kPerSm * sm_count;
    const size_t cum = sizeof(uint32_t) * (2 * a.batch + 1);
    const auto kernel = attn_split_kernel<D, NT, F::kWarps, kFp16, false>;
    const cudaError_t e =
        allow_smem(kernel, F::kSmem + static_cast<int>(sizeof(uint32_t)) * (2 * kAttnMaxBatch + 1));
    if (e != cudaSuccess) return e;
    const cudaError_t k = launch_kernel(kernel, dim3(run_blocks), dim3(F::kWarps * 32), F::kSmem + cum, s, a);
    if (k != cudaSuccess) return k;
    return launch_kernel(attn_join_kernel<D, NT, kFp16>, dim3(run_blocks, (std::min(S::kRows, a.rows) + 3) / 4),
                         dim3(128), 0, s, a);
}

// 8-row units while a key head's rows fit one (a 16-row one would idle half
// of its MMAs and registers), else 16-row ones; 256-wide heads leave no
// registers for a second row tile.
template <int D, bool kFp16>
cudaError_t run_split(const AttnArgs& a, int sm_count, cudaStream_t s) {
    if constexpr (D < 256) {
        if (a.rows > 8) return run_split_nt<D, 2, kFp16>(a, sm_count, s);
    }
    return run_split_nt<D, 1, kFp16>(a, sm_count, s);
}

template <int D, bool kFp16>
cudaError_t run_attn(const AttnLaunch& L, cudaStream_t s) {
    AttnArgs a{};
    a.q = static_cast<const uint16_t*>(L.q->data);
    a.q_ts = L.q->token_stride;
    a.q_hs = L.q->head_stride;
    a.out = static_cast<uint16_t*>(L.out->data);
    a.o_ts = L.out->token_stride;
    a.o_hs = L.out->head_stride;
    a.lse = L.lse;
    a.k = L.cache->k;
    a.v = L.cache->v;
    a.k_scale = L.cache->k_scale;
    a.v_scale = L.cache->v_scale;
    a.pages = L.cache->pages;
    a.kv_heads = L.cache->kv_heads;
    while ((1 << a.page_shift) < L.cache->page_size) ++a.page_shift;
    a.q_heads = L.q_heads;
    a.group = L.q_heads / a.kv_heads;
    a.scale_log2 = static_cast<float>(L.scale * 1.4426950408889634074);
    a.crossings = static_cast<int4*>(L.scratch);
    a.slots = static_cast<float*>(L.scratch) + crossing_floats(L.sm_count);
    a.status = L.status;
    float* states = a.slots + attn_slot_floats(L.sm_count, D);
    AttnArgs own = a;
    own.page_table = L.page_table;
    own.table_stride = L.table_stride;
    own.max_len = static_cast<int>(L.max_len);
    own.kv_lens = L.kv_lens;
    own.batch = L.batch;
    own.q_len = L.q_len;
    own.rows = L.q_len * a.group;
    own.causal = true;
    if (L.prefix_len == 0) return run_split<D, kFp16>(own, L.sm_count, s);

    // The rows' states over one part of their tokens go to scratch, the other
    // part's kernel joins them with its own (addition is the same either
    // way).  The own tokens come first where the prefix's kernel can start
    // while their last blocks run: its first reads need nothing of theirs.
    const int rows = L.batch * L.q_len * a.group;
    const bool on_tensor_cores = attn_prefix_on_tensor_cores(rows, D);
    const int splits = on_tensor_cores ? attn_prefix_splits(rows, a.kv_heads, L.prefix_len, L.sm_count) : 0;
    if (splits == 1) {
        const cudaError_t e = launch_attn_prefix(L, nullptr, states, s);
        if (e != cudaSuccess) return e;
        own.prefix = states;
        return run_split<D, kFp16>(own, L.sm_count, s);
    }
    own.states = states;
    const cudaError_t e = run_split<D, kFp16>(own, L.sm_count, s);
    if (e != cudaSuccess) return e;
    a.prefix = states;
    if constexpr (D <= 128) {
        if (on_tensor_cores) {
            float* shares = states + attn_state_floats(L.batch, L.q_len, L.q_heads, D);
            const cudaError_t k = launch_attn_prefix(L, shares, nullptr, s);
            if (k != cudaSuccess) return k;
            const PrefixShares p{shares, splits, (rows + kPrefixTileRows - 1) / kPrefixTileRows, kPrefixTileRows, rows};
            return launch_kernel(attn_prefix_join_kernel<D, kFp16>, dim3((rows + 3) / 4, a.kv_heads), dim3(128), 0, s,
                                 a, p);
        }
    }
    // The prefix as one request that every query row of the batch asks.
    a.page_table = L.prefix_pages;
    a.max_len = static_cast<int>(L.prefix_len);
    a.batch = 1;
    a.q_len = L.batch * L.q_len;
    a.rows = rows;
    a.behind = true;
    return run_split<D, kFp16>(a, L.sm_count, s);
}

}  // namespace

int64_t attn_slot_floats(int sm_count, int head_dim) {
    return static_cast<int64_t>(2) * attn_blocks(sm_count) * kMaxUnitRows * (head_dim + 4);
}

int64_t attn_state_floats(int batch, int q_len, int q_heads, int head_dim) {
    return static_cast<int64_t>(batch) * q_len * q_heads * (head_dim + 4);
}

// Rows of a key head from which the prefix goes to the tcgen05 kernel (which
// holds heads of 64 and 128).
bool attn_prefix_on_tensor_cores(int64_t rows, int head_dim) { return head_dim < 256 && rows > 32; }

int64_t attn_scratch_bytes(int batch, int q_len, int q_heads, int head_dim, int64_t prefix_len,
                           int sm_count) {
    int64_t n = crossing_floats(sm_count) + attn_slot_floats(sm_count, head_dim);
    if (prefix_len > 0)
        n += attn_state_floats(batch, q_len, q_heads, head_dim) + attn_prefix_slot_floats(sm_count, head_dim);
    return n * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_attn_decode(const AttnLaunch& L, cudaStream_t s) {
    switch (L.cache->head_dim) {
        case 64: return L.fp16 ? run_attn<64, true>(L, s) : run_attn<64, false>(L, s);
        case 128: return L.fp16 ? run_attn<128, true>(L, s) : run_attn<128, false>(L, s);
        default: return L.fp16 ? run_attn<256, true>(L, s) : run_attn<256, false>(L, s);
    }
}

}  // namespace dg
