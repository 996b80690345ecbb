// k_attn_decode.cu -- attention of a few new tokens per request over the
// paged E4M3 key/value cache, with an optional prefix shared by the batch.
//
// For one query row and the tokens t it sees, with codes kc, vc and scales
// sk, sv of one cached row each (k_t = sk_t kc_t, v_t = sv_t vc_t):
//   x_t = scale sk_t (q . kc_t)                the score
//   w_t = exp(x_t + ln sv_t - m),  m = max_t (x_t + ln sv_t)
//   acc = sum_t w_t vc_t,          l = sum_t w_t / sv_t
//   o   = acc / l,                 lse = m + ln l
// The value's scale sits inside the exponential, so a weight costs one
// exponential, w is at most 1 (exactly 1 for the row's largest) and goes to
// the second product as FP16 with 11 bits: a weight below 2^-14 of the
// largest contribution keeps an absolute error of 2^-25 of it.  E4M3 codes
// are exact in FP16; sums, maxima and the state are FP32.
//
// A cached element is read once and takes 4 flop per row, so for the few
// rows that share a key head the kernel is bound by HBM: it streams codes
// through shared memory with asynchronous copies and takes both products on
// warp-level MMAs (16 rows; tcgen05's 128 would be idle).
//
// Split: all (request, key head, 16-row tile) units are laid end to end in
// 32-token tiles, and every warp of the grid takes an equal run of them, so
// ragged lengths balance and one long cache spreads over all SMs.  A warp
// writes the units that lie inside its run; the pieces of a unit that
// crosses warps are joined in shared memory, and those of a unit that
// crosses blocks through scratch by a second, small kernel.  Every join goes
// in token order: results do not depend on timing.
#include <cuda_runtime.h>

#include <algorithm>

#include "dg_internal.h"
#include "dg_ptx.cuh"

namespace dg {
namespace {

constexpr int kTile = 32;      // tokens per warp step
constexpr int kRows = 16;      // query rows per unit (the MMA's M side)
constexpr float kLn2 = 0.69314718055994531f;

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
    int q_heads;
    bool causal;
    float scale_log2;          // softmax scale * log2(e)
    float* slots;              // two states of 16 rows per block
    const float* prefix;       // states of the prefix, per (token, head), or null
    float* states;             // where this call leaves states instead of outputs, or null
    uint32_t* status;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                 :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

__device__ __forceinline__ uint32_t half2_of(uint32_t codes, int hi) {
    return e4m3x2_to_f16x2(static_cast<uint16_t>(hi ? codes >> 16 : codes));
}

// Shapes per head width.  kDims: dims of one lane quarter in a run (a lane
// with lane % 4 == c owns dims c * kDims .. of each kSpan-wide part of the
// head, in both products).
template <int D>
struct Shape {
    static constexpr int kWarps = D == 256 ? 4 : 8;
    static constexpr int kStages = D == 64 ? 4 : 2;
    static constexpr int kParts = D == 256 ? 2 : 1;
    static constexpr int kSpan = D / kParts;        // 64 or 128
    static constexpr int kDims = kSpan / 4;         // 16 or 32
    static constexpr int kStageBytes = kTile * D * 2 + kTile * 8;
    static constexpr int kState = D + 4;            // m, l, 2 unused, acc[D]
    static constexpr int kStashBytes = kRows * kState * 4;
    // tail pieces are stashed over the warp's (drained) stages
    static constexpr int kRingBytes = kStages * kStageBytes;
    static_assert(kRingBytes >= kStashBytes, "a tail piece fits the ring");
    static constexpr int kSmem = kWarps * (kRingBytes + kStashBytes) + 256;
};

// Byte offset of 16-byte chunk `chunk` of token t in a tile: the chunks of a
// 128-byte line are permuted by the token so that neither product's reads
// meet in a bank (key reads: 2 tokens x 4 chunks a quarter warp; value
// reads: 4 even tokens x 2 chunks).
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int t, int chunk) {
    if constexpr (D == 64)
        return (t >> 1) * 128 + ((((t & 1) * 4 + chunk) ^ (((t >> 1) & 3) << 1)) * 16);
    else
        return t * D + (chunk >> 3) * 128 + (((chunk & 7) ^ (t & 7)) * 16);
}

// A place in the flat order of tiles.
struct Cursor {
    int b;       // request
    int unit;    // key head * row_tiles + row tile
    int tile;
    int ntile;   // tiles of the request's units
    int len;     // its tokens
};

// A warp's state of one unit: rows g and g + 8 of the lane.
template <int D>
struct State {
    float m[2], l[2];
    float acc[D / 8][4];
};

// Final output (or state) of 4 dims of one row from its joined state.
template <int D, bool kFp16>
__device__ __forceinline__ void emit4(const AttnArgs& a, int64_t token, int head, int d, float m,
                                      float l, float4 x) {
    if (a.states != nullptr) {
        float* s = a.states + (token * a.q_heads + head) * (D + 4);
        *reinterpret_cast<float4*>(s + 4 + d) = x;
        if (d == 0) {
            s[0] = m;
            s[1] = l;
        }
        return;
    }
    if (a.prefix != nullptr) {
        const float* s = a.prefix + (token * a.q_heads + head) * (D + 4);
        const float pm = s[0], pl = s[1];
        const float4 p = *reinterpret_cast<const float4*>(s + 4 + d);
        const float top = fmaxf(m, pm);
        const float base = top == -INFINITY ? 0.0f : top;
        const float wm = ex2(m - base), wp = ex2(pm - base);
        m = top;
        l = wm * l + wp * pl;
        x.x = wm * x.x + wp * p.x;
        x.y = wm * x.y + wp * p.y;
        x.z = wm * x.z + wp * p.z;
        x.w = wm * x.w + wp * p.w;
    }
    const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
    uint2 o;
    if constexpr (kFp16) {
        o = make_uint2(f32x2_to_f16x2(x.x * inv, x.y * inv), f32x2_to_f16x2(x.z * inv, x.w * inv));
    } else {
        o = make_uint2(f32x2_to_bf16x2(x.x * inv, x.y * inv), f32x2_to_bf16x2(x.z * inv, x.w * inv));
    }
    *reinterpret_cast<uint2*>(a.out + token * a.o_ts + head * a.o_hs + d) = o;
    if (d == 0 && a.lse != nullptr)
        a.lse[token * a.q_heads + head] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
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

// cum[b] = tiles of one unit of requests 0 .. b-1, over the whole block.
template <int kThreads>
__device__ __forceinline__ void scan_tiles(const AttnArgs& a, uint32_t* cum, uint32_t* warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t carry = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        uint32_t n = b < a.batch ? (request_len(a, b) + kTile - 1) / kTile : 0;
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

// Tiles a warp takes: an equal share of all.
__device__ __forceinline__ int64_t tiles_per_warp(int64_t total, int64_t warps) {
    return max(static_cast<int64_t>(1), (total + warps - 1) / warps);
}

// The request whose tiles hold flat position f (which is below the total).
__device__ __forceinline__ int find_request(const uint32_t* cum, int batch, int64_t units, int64_t f) {
    int lo = 0, hi = batch;   // cum[lo] * units <= f < cum[hi] * units
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<int64_t>(cum[mid]) * units <= f) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int D, bool kFp16>
__global__ void __launch_bounds__(Shape<D>::kWarps * 32, 1)
attn_split_kernel(const AttnArgs a) {
    using S = Shape<D>;
    constexpr int kWarps = S::kWarps, kThreads = kWarps * 32, kStages = S::kStages;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t warp_sum[kWarps];
    __shared__ int piece_b[2 * kWarps], piece_unit[2 * kWarps];   // request (-1: no piece), unit
    uint32_t* cum = reinterpret_cast<uint32_t*>(smem + S::kSmem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    pdl_wait();
    scan_tiles<kThreads>(a, cum, warp_sum);

    const int units = a.kv_heads * a.row_tiles;
    const int64_t total = static_cast<int64_t>(cum[a.batch]) * units;
    const int64_t run = tiles_per_warp(total, static_cast<int64_t>(gridDim.x) * kWarps);
    const int64_t block0 = static_cast<int64_t>(blockIdx.x) * kWarps * run;
    const int64_t block1 = min(total, block0 + kWarps * run);
    const int64_t f0 = min(total, block0 + warp * run), f1 = min(total, f0 + run);

    // Requests without a token of their own: nothing below reaches them.
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
        if (cum[b + 1] != cum[b]) continue;
        for (int i = threadIdx.x; i < a.q_len * a.q_heads * (D / 4); i += kThreads) {
            const int row = i / (D / 4);
            emit4<D, kFp16>(a, static_cast<int64_t>(b) * a.q_len + row / a.q_heads, row % a.q_heads,
                            4 * (i % (D / 4)), -INFINITY, 0.0f, make_float4(0, 0, 0, 0));
        }
    }

    const uint32_t ring = smem_addr(smem) + warp * S::kRingBytes;
    float* head_stash =
        reinterpret_cast<float*>(smem + kWarps * S::kRingBytes + warp * S::kStashBytes);
    float* tail_stash = reinterpret_cast<float*>(smem + warp * S::kRingBytes);
    if (lane == 0) piece_b[2 * warp] = piece_b[2 * warp + 1] = -1;

    if (f0 < f1) {
        // ---- producer side: the next tile to load, and its tokens' pages
        auto start = [&](int64_t f) {
            Cursor u;
            u.b = find_request(cum, a.batch, units, f);
            u.ntile = static_cast<int>(cum[u.b + 1] - cum[u.b]);
            u.len = request_len(a, u.b);
            const int64_t in = f - static_cast<int64_t>(cum[u.b]) * units;
            u.unit = static_cast<int>(in / u.ntile);
            u.tile = static_cast<int>(in - static_cast<int64_t>(u.unit) * u.ntile);
            return u;
        };
        auto advance = [&](Cursor& u) {
            if (++u.tile < u.ntile) return;
            u.tile = 0;
            if (++u.unit < units) return;
            u.unit = 0;
            do ++u.b; while (cum[u.b + 1] == cum[u.b]);   // f < total: there is one
            u.ntile = static_cast<int>(cum[u.b + 1] - cum[u.b]);
            u.len = request_len(a, u.b);
        };
        auto page_of = [&](const Cursor& u) {   // this lane's token of the tile: its page or -1
            const int t = u.tile * kTile + lane;
            if (t >= u.len) return -1;
            const int p = a.page_table[u.b * a.table_stride + (t >> a.page_shift)];
            if (p >= 0 && p < a.pages) return p;
            atomicOr(a.status, kStatusBadArgument);
            return -1;
        };
        const int in_page = (1 << a.page_shift) - 1;
        auto issue = [&](const Cursor& u, int page, int stage) {
            const uint32_t base = ring + stage * S::kStageBytes;
            const int h = u.unit / a.row_tiles;
            const int t0 = u.tile * kTile;
            constexpr int kPerRow = D / 16, kPerStep = 32 / kPerRow;
            const int chunk = lane % kPerRow;
#pragma unroll
            for (int i = 0; i < kTile / kPerStep; ++i) {
                const int t = i * kPerStep + lane / kPerRow;
                const int p = __shfl_sync(0xFFFFFFFFu, page, t);
                const int64_t row = ((static_cast<int64_t>(max(p, 0)) * a.kv_heads + h) << a.page_shift) +
                                    ((t0 + t) & in_page);
                const uint32_t dst = base + chunk_at<D>(t, chunk);
                const int64_t off = row * D + chunk * 16;
                cp_async16(dst, a.k + off, p < 0 ? 0 : 16);
                cp_async16(dst + kTile * D, a.v + off, p < 0 ? 0 : 16);
            }
            const int64_t row = ((static_cast<int64_t>(max(page, 0)) * a.kv_heads + h) << a.page_shift) +
                                ((t0 + lane) & in_page);
            const uint32_t sc = base + 2 * kTile * D + lane * 4;
            cp_async4(sc, a.k_scale + row, page < 0 ? 0 : 4);
            cp_async4(sc + kTile * 4, a.v_scale + row, page < 0 ? 0 : 4);
        };

        Cursor in = start(f0), at = in;
        int64_t fin = f0;
        int page = page_of(in);
#pragma unroll 1
        for (int s = 0; s < kStages; ++s) {
            if (fin < f1) {
                issue(in, page, s);
                if (++fin < f1) {
                    advance(in);
                    page = page_of(in);
                }
            }
            cp_commit();
        }

        uint32_t qa[D / 16][4];   // this unit's queries, as the first product's A operand
        float qscale[2] = {0.0f, 0.0f};
        int seen[2] = {0, 0}, seen_min = 0;
        State<D> st;
        int stage = 0, first_tile = 0;

        for (int64_t f = f0; f < f1; ++f) {
            const int h = at.unit / a.row_tiles, r0 = (at.unit - h * a.row_tiles) * kRows;
            if (f == f0 || at.tile == 0) {
                // ---- a new unit: its queries, normalised by a power of two
                first_tile = at.tile;
                const int len = at.len;
                seen_min = 0x7FFFFFFF;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = r0 + g + 8 * j;
                    const bool valid = r < a.rows;
                    int64_t token = 0;
                    int head = 0;
                    if (valid) row_place(a, at.b, h, r, &token, &head);
                    const uint16_t* src = a.q + token * a.q_ts + head * a.q_hs;
                    uint4 w[D / 32];
                    uint32_t top = 0;
#pragma unroll
                    for (int p = 0; p < S::kParts; ++p)
#pragma unroll
                        for (int i = 0; i < S::kDims / 8; ++i) {
                            const int k = p * (S::kDims / 8) + i;
                            w[k] = valid ? *reinterpret_cast<const uint4*>(src + p * S::kSpan + c * S::kDims + 8 * i)
                                         : make_uint4(0, 0, 0, 0);
                        }
                    float mul = 1.0f;
                    qscale[j] = a.scale_log2;
                    if constexpr (!kFp16) {
                        // BF16 queries: FP16 has more mantissa but less
                        // range, so a row is scaled by a power of two that
                        // brings its largest value to [1, 2).
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                top = max(top, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
                        }
                        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                        const int e = min(max(static_cast<int>(top >> 7), 1), 253);   // biased exponent
                        mul = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                        qscale[j] *= __uint_as_float(static_cast<uint32_t>(e) << 23);
                    }
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t v = x[i];
                            if constexpr (!kFp16)
                                v = f32x2_to_f16x2(__uint_as_float(v << 16) * mul,
                                                   __uint_as_float(v & 0xFFFF0000u) * mul);
                            // dims 8k + 2i, +1: MMA step 2k + i/2, k columns 2c.. (i even) or 2c + 8..
                            qa[2 * k + (i >> 1)][2 * (i & 1) + j] = v;
                        }
                    }
                    const int i = r / a.group;
                    seen[j] = !valid || !a.causal ? len : max(0, len - a.q_len + 1 + i);
                    if (valid) seen_min = min(seen_min, seen[j]);
                    st.m[j] = -INFINITY;
                    st.l[j] = 0.0f;
                }
                seen_min = __reduce_min_sync(0xFFFFFFFFu, seen_min);
                seen_min = min(seen_min, len);
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) st.acc[j][i] = 0.0f;
            }

            cp_wait<kStages - 1>();
            __syncwarp();
            const uint32_t kb = ring + stage * S::kStageBytes, vb = kb + kTile * D;
            const float* sk = reinterpret_cast<const float*>(smem + (kb - smem_addr(smem)) + 2 * kTile * D);
            const float* sv = sk + kTile;

            // ---- scores
            float s[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] = 0.0f;
            if constexpr (D == 64) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint4 x = lds128(kb + chunk_at<D>(8 * n + g, c));
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma16816(s[n], qa[i][0], qa[i][1], qa[i][2], qa[i][3], half2_of(w[i], 0),
                                 half2_of(w[i], 1));
                }
            } else {
#pragma unroll
                for (int p = 0; p < D / 64; ++p) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const uint4 x = lds128(kb + chunk_at<D>(8 * n + g, 8 * (p >> 1) + 2 * c + (p & 1)));
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma16816(s[n], qa[4 * p + i][0], qa[4 * p + i][1], qa[4 * p + i][2],
                                     qa[4 * p + i][3], half2_of(w[i], 0), half2_of(w[i], 1));
                    }
                }
            }

            // ---- softmax: lane holds tokens 8n + 2c, +1 of rows g (s[n][0..1]) and g + 8
            const int t0 = at.tile * kTile;
            const bool masked = t0 + kTile > seen_min;
            // this lane's token: log2 and reciprocal of the value's scale
            const float own_sv = sv[lane];
            const float safe_sv = own_sv < 0x1p-100f ? 0x1p-100f : own_sv;
            const float own_log = __log2f(safe_sv), own_rcp = __frcp_rn(safe_sv);
            float rsv[4][2];
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 k2 = *reinterpret_cast<const float2*>(sk + 8 * n + 2 * c);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tok = 8 * n + 2 * c + i;
                    const float lg = __shfl_sync(0xFFFFFFFFu, own_log, tok);
                    rsv[n][i] = __shfl_sync(0xFFFFFFFFu, own_rcp, tok);
                    const float kk = i == 0 ? k2.x : k2.y;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float y = fmaf(s[n][2 * j + i] * kk, qscale[j], lg);
                        if (masked && t0 + tok >= seen[j]) y = -INFINITY;
                        s[n][2 * j + i] = y;
                        top[j] = fmaxf(top[j], y);
                    }
                }
            }
            float base[2];
            bool grew = false;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                top[j] = fmaxf(top[j], __shfl_xor_sync(0xFFFFFFFFu, top[j], 1));
                top[j] = fmaxf(top[j], __shfl_xor_sync(0xFFFFFFFFu, top[j], 2));
                grew |= top[j] > st.m[j];
            }
            if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float m = fmaxf(st.m[j], top[j]);
                    const float f = m == -INFINITY ? 1.0f : ex2(st.m[j] - m);
                    st.m[j] = m;
                    st.l[j] *= f;
#pragma unroll
                    for (int k = 0; k < D / 8; ++k) {
                        st.acc[k][2 * j] *= f;
                        st.acc[k][2 * j + 1] *= f;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) base[j] = st.m[j] == -INFINITY ? 0.0f : st.m[j];
            uint32_t pw[4][2];
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float w0 = ex2(s[n][2 * j] - base[j]), w1 = ex2(s[n][2 * j + 1] - base[j]);
                    // a token that a row does not see adds nothing, whatever its scale holds
                    const int tok = t0 + 8 * n + 2 * c;
                    if (!masked || tok < seen[j]) st.l[j] += w0 * rsv[n][0];
                    if (!masked || tok + 1 < seen[j]) st.l[j] += w1 * rsv[n][1];
                    pw[n][j] = f32x2_to_f16x2(w0, w1);
                }

            // ---- values: tokens 2c, 2c+1, 2c+8, 2c+9 of each 16; dims of chunk g
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const int t = 16 * kk + 2 * c;
                const uint32_t a0 = pw[2 * kk][0], a1 = pw[2 * kk][1], a2 = pw[2 * kk + 1][0],
                               a3 = pw[2 * kk + 1][1];
                auto words = [&](int j0, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
                    const uint32_t lo = __byte_perm(x0, x1, 0x5140), hi = __byte_perm(x0, x1, 0x7362);
                    const uint32_t lp = __byte_perm(x2, x3, 0x5140), hp = __byte_perm(x2, x3, 0x7362);
                    mma16816(st.acc[j0], a0, a1, a2, a3, half2_of(lo, 0), half2_of(lp, 0));
                    mma16816(st.acc[j0 + 1], a0, a1, a2, a3, half2_of(lo, 1), half2_of(lp, 1));
                    mma16816(st.acc[j0 + 2], a0, a1, a2, a3, half2_of(hi, 0), half2_of(hp, 0));
                    mma16816(st.acc[j0 + 3], a0, a1, a2, a3, half2_of(hi, 1), half2_of(hp, 1));
                };
                if constexpr (D == 64) {
                    const int ch = g >> 1, part = (g & 1) * 8;
                    const uint2 x0 = lds64(vb + chunk_at<D>(t, ch) + part);
                    const uint2 x1 = lds64(vb + chunk_at<D>(t + 1, ch) + part);
                    const uint2 x2 = lds64(vb + chunk_at<D>(t + 8, ch) + part);
                    const uint2 x3 = lds64(vb + chunk_at<D>(t + 9, ch) + part);
                    words(0, x0.x, x1.x, x2.x, x3.x);
                    words(4, x0.y, x1.y, x2.y, x3.y);
                } else {
#pragma unroll
                    for (int p = 0; p < S::kParts; ++p) {
                        const uint4 x0 = lds128(vb + chunk_at<D>(t, 8 * p + g));
                        const uint4 x1 = lds128(vb + chunk_at<D>(t + 1, 8 * p + g));
                        const uint4 x2 = lds128(vb + chunk_at<D>(t + 8, 8 * p + g));
                        const uint4 x3 = lds128(vb + chunk_at<D>(t + 9, 8 * p + g));
                        words(16 * p, x0.x, x1.x, x2.x, x3.x);
                        words(16 * p + 4, x0.y, x1.y, x2.y, x3.y);
                        words(16 * p + 8, x0.z, x1.z, x2.z, x3.z);
                        words(16 * p + 12, x0.w, x1.w, x2.w, x3.w);
                    }
                }
            }

            // ---- refill the stage
            __syncwarp();
            if (fin < f1) {
                issue(in, page, stage);
                if (++fin < f1) {
                    advance(in);
                    page = page_of(in);
                }
            }
            cp_commit();
            stage = stage + 1 == kStages ? 0 : stage + 1;

            // ---- the unit's (or the run's) end
            const bool unit_end = at.tile + 1 == at.ntile;
            if (unit_end || f + 1 == f1) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    st.l[j] += __shfl_xor_sync(0xFFFFFFFFu, st.l[j], 1);
                    st.l[j] += __shfl_xor_sync(0xFFFFFFFFu, st.l[j], 2);
                }
                const bool whole = unit_end && first_tile == 0;
                // first piece of the run when its unit began before it, else the last one
                const bool is_head = !whole && first_tile != 0;
                float* stash = is_head ? head_stash : tail_stash;
                if (!whole && !is_head) {   // over the ring: nothing is in flight any more
                    cp_wait<0>();
                    __syncwarp();
                }
                if (!whole && lane == 0) {
                    piece_b[2 * warp + (is_head ? 0 : 1)] = at.b;
                    piece_unit[2 * warp + (is_head ? 0 : 1)] = at.unit;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int rr = g + 8 * j;
                    const bool valid = r0 + rr < a.rows;
                    int64_t token = 0;
                    int head = 0;
                    if (valid) row_place(a, at.b, h, r0 + rr, &token, &head);
                    float* row = stash + rr * S::kState;
                    if (!whole && c == 0) {
                        row[0] = st.m[j];
                        row[1] = st.l[j];
                    }
#pragma unroll
                    for (int p = 0; p < S::kParts; ++p) {
#pragma unroll
                        for (int k = 0; k < S::kDims / 4; ++k) {
                            // column 2c of n-tile i is dim c * kDims + i, column 2c + 1 dim + kDims / 2
                            const int half = k / (S::kDims / 8), i = (k % (S::kDims / 8)) * 4;
                            const int e = 2 * j + half, n = p * (S::kDims / 2) + i;
                            const float4 x = make_float4(st.acc[n][e], st.acc[n + 1][e],
                                                         st.acc[n + 2][e], st.acc[n + 3][e]);
                            const int d = p * S::kSpan + c * S::kDims + 4 * k;
                            if (!whole)
                                *reinterpret_cast<float4*>(row + 4 + d) = x;
                            else if (valid)
                                emit4<D, kFp16>(a, token, head, d, st.m[j], st.l[j], x);
                        }
                    }
                }
            }
            if (f + 1 < f1) advance(at);
        }
        cp_wait<0>();
    }
    __syncthreads();

    // ---- join the pieces of each unit, in warp (token) order
    for (int i = 0; i < 2 * kWarps;) {
        const int b = piece_b[i];
        if (b < 0) {
            ++i;
            continue;
        }
        const int unit = piece_unit[i];
        int end = i + 1;
        while (end < 2 * kWarps && (piece_b[end] < 0 || (piece_b[end] == b && piece_unit[end] == unit))) ++end;
        const int64_t ntile = cum[b + 1] - cum[b];
        const int64_t u0 = static_cast<int64_t>(cum[b]) * units + unit * ntile, u1 = u0 + ntile;
        const bool inside = u0 >= block0 && u1 <= block1;
        float* slot = a.slots + (2 * static_cast<int64_t>(blockIdx.x) + (u0 < block0 ? 0 : 1)) *
                                    (kRows * S::kState);
        const int h = unit / a.row_tiles, r0 = (unit - h * a.row_tiles) * kRows;
        const int rows = min(kRows, a.rows - r0);
        for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
            const int r = e / (D / 4), d = 4 * (e % (D / 4));
            float m = -INFINITY;
            for (int p = i; p < end; ++p) {
                if (piece_b[p] < 0) continue;
                const uint8_t* base = (p & 1) ? smem + (p >> 1) * S::kRingBytes
                                              : smem + kWarps * S::kRingBytes + (p >> 1) * S::kStashBytes;
                m = fmaxf(m, reinterpret_cast<const float*>(base)[r * S::kState]);
            }
            const float safe = m == -INFINITY ? 0.0f : m;
            float l = 0.0f;
            float4 x = make_float4(0, 0, 0, 0);
            for (int p = i; p < end; ++p) {
                if (piece_b[p] < 0) continue;
                const uint8_t* base = (p & 1) ? smem + (p >> 1) * S::kRingBytes
                                              : smem + kWarps * S::kRingBytes + (p >> 1) * S::kStashBytes;
                const float* row = reinterpret_cast<const float*>(base) + r * S::kState;
                const float w = ex2(row[0] - safe);
                const float4 y = *reinterpret_cast<const float4*>(row + 4 + d);
                l += w * row[1];
                x.x += w * y.x;
                x.y += w * y.y;
                x.z += w * y.z;
                x.w += w * y.w;
            }
            if (inside) {
                int64_t token;
                int head;
                row_place(a, b, h, r0 + r, &token, &head);
                emit4<D, kFp16>(a, token, head, d, m, l, x);
            } else {
                float* row = slot + r * S::kState;
                *reinterpret_cast<float4*>(row + 4 + d) = x;
                if (d == 0) {
                    row[0] = m;
                    row[1] = l;
                }
            }
        }
        i = end;
    }
}

// Joins the units that cross blocks: block x of the grid takes the unit that
// begins in block x's run of the split kernel and goes on past its end, warp
// y one of its rows.
template <int D, bool kFp16>
__global__ void __launch_bounds__(128)
attn_join_kernel(const AttnArgs a, int split_blocks) {
    constexpr int kState = Shape<D>::kState, kWarps = Shape<D>::kWarps;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t warp_sum[4];
    uint32_t* cum = reinterpret_cast<uint32_t*>(smem);
    pdl_wait();
    scan_tiles<128>(a, cum, warp_sum);
    const int units = a.kv_heads * a.row_tiles;
    const int64_t total = static_cast<int64_t>(cum[a.batch]) * units;
    const int64_t per_block = kWarps * tiles_per_warp(total, static_cast<int64_t>(split_blocks) * kWarps);
    const int64_t f0 = blockIdx.x * per_block, f1 = f0 + per_block;
    if (f1 >= total) return;
    const int b = find_request(cum, a.batch, units, f1);
    const int64_t ntile = cum[b + 1] - cum[b], before = static_cast<int64_t>(cum[b]) * units;
    const int unit = static_cast<int>((f1 - before) / ntile);
    const int64_t u0 = before + unit * ntile, u1 = u0 + ntile;
    if (u0 == f1 || u0 < f0) return;   // ends there, or began in an earlier block
    const int last = static_cast<int>((u1 - 1) / per_block);
    const int h = unit / a.row_tiles, r0 = (unit - h * a.row_tiles) * kRows;
    const int r = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r0 + r >= a.rows) return;
    int64_t token;
    int head;
    row_place(a, b, h, r0 + r, &token, &head);
    // slot 2x + 1 of the first block, then slot 2y of each later one
    auto state = [&](int blk) {
        return a.slots + ((2 * static_cast<int64_t>(blk) + (blk == static_cast<int>(blockIdx.x) ? 1 : 0)) * kRows + r) * kState;
    };
    float m = -INFINITY;
    for (int i = blockIdx.x + lane; i <= last; i += 32) m = fmaxf(m, state(i)[0]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float safe = m == -INFINITY ? 0.0f : m;
    for (int d = 4 * lane; d < D; d += 128) {
        float l = 0.0f;
        float4 x = make_float4(0, 0, 0, 0);
#pragma unroll 4
        for (int i = blockIdx.x; i <= last; ++i) {
            const float* row = state(i);
            const float w = ex2(row[0] - safe);
            const float4 y = *reinterpret_cast<const float4*>(row + 4 + d);
            l += w * row[1];
            x.x += w * y.x;
            x.y += w * y.y;
            x.z += w * y.z;
            x.w += w * y.w;
        }
        emit4<D, kFp16>(a, token, head, d, m, l, x);
    }
}

template <int D, bool kFp16>
cudaError_t run_split(const AttnArgs& a, int blocks, cudaStream_t s) {
    using S = Shape<D>;
    const size_t cum = sizeof(uint32_t) * (a.batch + 1);
    const size_t smem = S::kSmem + cum;
    cudaError_t e = cudaFuncSetAttribute(attn_split_kernel<D, kFp16>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         S::kSmem + static_cast<int>(sizeof(uint32_t)) * (kAttnMaxBatch + 1));
    if (e != cudaSuccess) return e;
    e = launch_kernel(attn_split_kernel<D, kFp16>, dim3(blocks), dim3(S::kWarps * 32), smem, s, a);
    if (e != cudaSuccess) return e;
    const dim3 grid(std::max(1, blocks - 1), (std::min(kRows, a.rows) + 3) / 4);
    return launch_kernel(attn_join_kernel<D, kFp16>, grid, dim3(128), cum, s, a, blocks);
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
    a.slots = reinterpret_cast<float*>(L.scratch);
    a.status = L.status;
    float* states = a.slots + attn_slot_floats(L.sm_count, D);
    if (L.prefix_len > 0) {
        // The prefix as one request that every query row of the batch asks.
        AttnArgs p = a;
        p.page_table = L.prefix_pages;
        p.max_len = static_cast<int>(L.prefix_len);
        p.batch = 1;
        p.q_len = L.batch * L.q_len;
        p.rows = p.q_len * p.group;
        p.row_tiles = (p.rows + kRows - 1) / kRows;
        p.states = states;
        const cudaError_t e = run_split<D, kFp16>(p, L.sm_count, s);
        if (e != cudaSuccess) return e;
        a.prefix = states;
    }
    a.page_table = L.page_table;
    a.table_stride = L.table_stride;
    a.max_len = static_cast<int>(L.max_len);
    a.kv_lens = L.kv_lens;
    a.batch = L.batch;
    a.q_len = L.q_len;
    a.rows = L.q_len * a.group;
    a.row_tiles = (a.rows + kRows - 1) / kRows;
    a.causal = true;
    return run_split<D, kFp16>(a, L.sm_count, s);
}

}  // namespace

int64_t attn_slot_floats(int sm_count, int head_dim) {
    return static_cast<int64_t>(2) * sm_count * kRows * (head_dim + 4);
}

int64_t attn_scratch_bytes(int batch, int q_len, int q_heads, int head_dim, int64_t prefix_len,
                           int sm_count) {
    int64_t n = attn_slot_floats(sm_count, head_dim);
    if (prefix_len > 0) n += static_cast<int64_t>(batch) * q_len * q_heads * (head_dim + 4);
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
