// k_norm.cu -- root-mean-square norm of rows, with the addition of a residual
// before it and E4M3 or 16-bit output, and its gradient.
//
//   s = x + r            (FP32; written rounded, as the new residual stream)
//   y = s rsqrt(mean(s^2) + eps) w
//   out: y rounded; or codes E4M3(y / scale) with scale = amax / 448 of the
//   row ([FP8-guide] §3.2's rule with the row as the tensor); or codes with
//   one given scale and the tensor's amax recorded for the next call.
// [FP8-guide] = "DeepGEMM实战：FP8矩阵乘法与JIT编译优化指南".
//
// The work is memory's: 2 bytes an element read (4 with a residual) and 1 to 4
// written, against some ten FP32 operations.  A block keeps a whole row in
// registers between its two reductions (sum of squares, maximum), so each
// element crosses memory once; blocks are persistent and have the next row's
// loads in flight while a row is reduced and written.  BF16 with a residual to
// codes, 16001 x 4096: 71.5 us, 0.95 of the rate of a copy; FP16 to codes of
// one scale, 6001 x 8192: 32.5 us, 0.67 (2 bytes read and 1 written an element
// leave the instructions as the bound: 65 % of the issue slots).
//
// Gradient, with u = s rsqrt(mean(s^2) + eps) and g = dy w:
//   dx = rsqrt(..) (g - u mean(g u)) + dsum,   dw = sum over rows of dy u
// dx belongs to x and to the residual alike.  A thread owns the same columns
// of every row of its block, so dw is summed in registers and leaves the
// block once; the blocks' sums are joined in order by a second kernel, so
// that results do not depend on timing.  BF16 with dsum and dw, 16384 x 4096:
// 82.9 us, 0.95.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "row_common.cuh"

namespace dg {
namespace {

// A sum of squares past FP32's range is taken again of elements times this:
// 32768 squares of 2^128 2^-80 hold, and one element at least was above 2^56.
constexpr float kDown = 0x1p-80f;

// A block's 1024 threads, or two blocks of 512 and more of fewer, at 64
// registers: a row in FP32 and the next row's loads at two vectors a thread
// (3000 x 16384 BF16 with residual, codes: 55.5 us, 0.91 of the rate of a
// copy; four vectors of 512 threads at 128 registers 90.7); at four, past
// 16384 columns, the row stays packed and is unpacked again for each pass, the
// next one on its way to L2 (1500 x 24576: 56.6 us, 0.67; held in FP32 70.6).
// Even so 64 registers are too few there: with a residual 84 bytes a thread are
// spilled to codes, 308 to 16-bit output (62.4 us, 0.70) and 332 to one scale
// (65.1, 0.58), without one 12, 144 and 120.
constexpr int kLimits[3] = {1024, 1024, 0};
constexpr int kPerSm[3] = {1024, 1024, 0};
static_assert(hold_widest_row(kLimits) && kLimits[0] <= kRowThreads && kLimits[1] <= kRowThreads, "launch bounds");

template <int NV, bool kFp16, int kOut, bool kNarrow, bool kResidual>
__global__ void __launch_bounds__(kRowThreads, 1) rmsnorm_kernel(const NormArgs a, int team_size) {
    __shared__ float2 buffer[2][kRowThreads / 32];
    pdl_wait();
    const uint16_t* const weight = behind_wait(a.weight);
    const RowTeam<kNarrow> team(team_size);
    RowReduce<kNarrow> reduce{buffer, team.size};
    const int vectors = a.cols >> 3;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    // The weight, packed, in registers where they reach; else it is read again
    // for every row.
    constexpr bool kKeep = NV == 2;
    constexpr bool kKeepWeight = NV == 2 && (kOut == kNormRows || (kOut == kNormTensor && !kResidual));
    uint4 x[NV], r[NV], w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        x[i] = r[i] = make_uint4(0, 0, 0, 0);
        const int at = team.at + i * team.size;
        if (kKeepWeight) w[i] = weight_if(a.weight != nullptr && at < vectors, weight, at);
    }
    // The next row's loads are in flight while a row is worked on: x and r; or,
    // without a residual, those of the next two rows (x, then r).
    auto load_row = [&](const uint16_t* row, uint4 (&to)[NV]) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            load_if(team.at + i * team.size < vectors, row + 8 * (team.at + i * team.size), to[i]);
    };
    float pre = 1.0f, by = 0.0f;
    if constexpr (kOut == kNormTensor) {
        const ByScale given = by_scale(*a.scale);
        pre = given.pre;
        by = given.inv;
    }
    float tensor_top = 0.0f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * team.rows;
    int64_t first = static_cast<int64_t>(blockIdx.x) * team.rows;   // the block's rows, together
    // The addresses of x, residual and codes are stepped, not multiplied out
    // again (all of them stepped took more registers than there are).
    const uint16_t* x_next = a.x + (first + team.row) * a.x_stride;
    const uint16_t* r_next = kResidual ? a.residual + (first + team.row) * a.residual_stride : nullptr;
    uint8_t* q_row = kOut != kNormHalf ? a.q + (first + team.row) * a.cols : nullptr;
    if (first + team.row < a.rows) {
        load_row(x_next, x);
        if constexpr (kResidual) load_row(r_next, r);
    }
    if (kKeep && !kResidual && first + team.row + step < a.rows) load_row(x_next += step * a.x_stride, r);
    auto forget_all = [&] {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            forget(x[i]);
            if constexpr (kResidual) forget(r[i]);
        }
    };
    for (; first < a.rows; first += step) {
        const int64_t row = first + team.row;
        const int end = row < a.rows ? vectors : 0;   // this thread's vectors lie below
        if (!kKeep && threadIdx.x == 0 && row + step < a.rows) {
            prefetch_row(x_next + step * a.x_stride, 2 * a.cols);
            if constexpr (kResidual) prefetch_row(r_next + step * a.residual_stride, 2 * a.cols);
        }
        auto value = [&](int i, pair (&to)[4]) {   // s
            unpack8<kFp16>(x[i], to);
            if constexpr (kResidual) {
                pair add[4];
                unpack8<kFp16>(r[i], add);
#pragma unroll
                for (int e = 0; e < 4; ++e) to[e] = pair_add(to[e], add[e]);
            }
        };
        pair v[kKeep ? NV : 1][4], squares = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            pair (&t)[4] = v[kKeep ? i : 0];
            value(i, t);
            if (a.sum != nullptr) store_if(at < end, a.sum + row * a.sum_stride + 8 * at, pack8<kFp16>(t));
#pragma unroll
            for (int e = 0; e < 4; ++e) squares = pair_fma(t[e], t[e], squares);
        }
        if constexpr (!kKeep) {
            forget_all();
        } else if constexpr (kResidual) {
            if (row + step < a.rows) {
                load_row(x_next += step * a.x_stride, x);
                load_row(r_next += step * a.residual_stride, r);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) x[i] = r[i];
            if (row + 2 * step < a.rows) load_row(x_next += step * a.x_stride, r);
        }
        float total = reduce.sum(pair_sum(squares)), down = 1.0f;
        // (a vote: rows of a warp differ, and the reduction takes all of it)
        const bool again = !(total <= 3.0e38f);
        if (kNarrow ? __any_sync(0xFFFFFFFFu, again) : again) {
            down = again ? kDown : 1.0f;
            squares = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if constexpr (!kKeep) value(i, v[0]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const pair t = pair_mul(v[kKeep ? i : 0][e], pair_of(down));
                    squares = pair_fma(t, t, squares);
                }
            }
            total = reduce.sum(pair_sum(squares));
            if constexpr (!kKeep) forget_all();
        }
        const float inv = rsqrtf(fmaf(total, inv_cols, a.eps * down * down)) * down;
        auto normed = [&](int i, pair (&t)[4]) {   // y in place of s
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = pair_mul(t[e], pair_of(inv));
            if (a.weight != nullptr) {
                const int at = team.at + i * team.size;
                pair f[4];
                unpack8<kFp16>(kKeepWeight ? w[i] : weight_if(at < vectors, kKeep ? weight : behind_wait(weight), at), f);
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = pair_mul(t[e], f[e]);
            }
        };
        auto emit = [&](int i, pair (&t)[4]) {
            const int at = team.at + i * team.size;
            if constexpr (kOut == kNormHalf) {
                store_if(at < end, a.y + row * a.y_stride + 8 * at, pack8<kFp16>(t));
            } else {
                if constexpr (kOut == kNormTensor) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[e] = pair_mul(t[e], pair_of(pre));
                }
                store_if(at < end, q_row + 8 * at, codes8(t, by));
            }
        };
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            pair (&t)[4] = v[kKeep ? i : 0];
            if constexpr (!kKeep) value(i, t);
            normed(i, t);
            if (kOut != kNormHalf) top = top8(t, top);   // (zeros past the row)
            if constexpr (!kKeep && kOut != kNormRows) emit(i, t);
        }
        if constexpr (kOut == kNormRows) {
            top = reduce.max1(top);
            const float scale = row_scale(top);
            by = row_factor(scale);
            if (team.at == 0 && end != 0) a.row_scale[row] = scale;
            if constexpr (!kKeep) {
                asm volatile("" : "+f"(by));   // (formed first: the pass behind it needs all registers)
                forget_all();
            }
        }
        if (kOut == kNormTensor && end != 0)   // (fmaxf would drop a NaN)
            tensor_top = __uint_as_float(max(__float_as_uint(tensor_top), __float_as_uint(top)));
        if constexpr (kKeep || kOut == kNormRows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                pair (&t)[4] = v[kKeep ? i : 0];
                if constexpr (!kKeep) {
                    value(i, t);
                    normed(i, t);
                }
                emit(i, t);
            }
        }
        if (!kKeep && row + step < a.rows) {
            load_row(x_next += step * a.x_stride, x);
            if constexpr (kResidual) load_row(r_next += step * a.residual_stride, r);
        }
        if (kOut != kNormHalf) q_row += step * a.cols;
    }
    if constexpr (kOut == kNormTensor) {
        // One atomic a block.
        uint32_t* tops = reinterpret_cast<uint32_t*>(buffer);
        const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(tensor_top));
        __syncthreads();
        if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = bits;
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t top = 0;
            for (unsigned i = 0; i < blockDim.x >> 5; ++i) top = max(top, tops[i]);
            if (top != 0) atomicMax(a.amax_bits, top);
            // The last block to arrive forms the next call's scale; the word
            // counts the arrivals until then (it is zeroed with the maximum).
            if (a.next_scale != nullptr) {
                __threadfence();
                if (atomicAdd(reinterpret_cast<uint32_t*>(a.next_scale), 1u) == gridDim.x - 1) {
                    __threadfence();
                    *a.next_scale = scale_of_amax(__uint_as_float(atomicOr(a.amax_bits, 0u)));
                }
            }
        }
    }
}

__global__ void zero_words_kernel(uint32_t* a, uint32_t* b) {
    pdl_launch_dependents();   // the norm's launch overlaps this one's; it waits for its end
    pdl_wait();
    *a = 0u;
    if (b != nullptr) *b = 0u;
}

// The next scale where no last block can write it: no rows, or the word is
// the scale that the rows read.
__global__ void next_scale_kernel(const float* amax, float* scale) {
    pdl_wait();
    *scale = scale_of_amax(*amax);
}

// The gradient's blocks: up to 512 threads at 128 registers (a row, the next
// row's loads, the weight and the columns' sums).  Rows of more than 8192
// columns are a cluster's of two or four blocks, each with its part of the
// columns (BF16 with dw: 4000 x 11008 81.5 us, 3000 x 16384 77.8, 1500 x 24576
// 71.4; four or eight vectors a thread of one block, with spills, 112.8, 104.8
// and 181.1).
constexpr int kGradThreads = 512, kGradPerSm = 512;
constexpr int kGradColumns = 16 * kGradThreads;   // of a block
constexpr int kGradRanks = kMaxRowElements / kGradColumns;   // at most, a cluster
static_assert(kGradRanks * kGradColumns == kMaxRowElements, "widest row");

// Sums over a cluster's threads (each warp's value to every block, in one
// buffer of two, taken in turn as RowReduce's).
struct ClusterReduce {
    float2 (*buffer)[kGradRanks * kGradThreads / 32];
    int ranks, rank;
    int turn = 0;

    __device__ __forceinline__ float2 sum2(float a, float b) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        float2* buf = buffer[turn];
        turn ^= 1;
        if (lane < ranks)
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};"
                         :: "r"(map_to_rank(buf + rank * warps + warp, static_cast<uint32_t>(lane))), "f"(a), "f"(b)
                         : "memory");
        cluster_sync_all_diverged();
        const int n = ranks * warps;   // at most 64
        const float2 zero = make_float2(0.0f, 0.0f);
        const float2 u = lane < n ? buf[lane] : zero, v = lane + 32 < n ? buf[lane + 32] : zero;
        a = u.x + v.x;
        b = u.y + v.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        return make_float2(a, b);
    }
};

// Columns' sums of a block: the teams of a warp and then the warps are added in
// order; one partial a block.
enum GradRows : int { kWideRows, kNarrowRows, kClusterRows };
template <bool kFp16, GradRows kRows>
__global__ void __launch_bounds__(kGradThreads, kGradPerSm / kGradThreads) rmsnorm_grad_kernel(const NormGradArgs whole, int team_size) {
    constexpr int NV = 2;
    constexpr bool kNarrow = kRows == kNarrowRows, kCluster = kRows == kClusterRows;
    using Reduce = std::conditional_t<kCluster, ClusterReduce, RowReduce<kNarrow>>;
    __shared__ float2 buffer[2][kCluster ? kGradRanks * kGradThreads / 32 : kRowThreads / 32];
    __shared__ float columns[kNarrow ? 4 : 1][256];   // four warps' sums
    // A cluster's block: the columns from `column` on.
    NormGradArgs a = whole;
    int vectors = a.cols >> 3, block = blockIdx.x, blocks = gridDim.x;
    const RowTeam<kNarrow> team(team_size);
    Reduce reduce{};
    reduce.buffer = buffer;
    if constexpr (kCluster) {
        const int ranks = team_size, rank = static_cast<int>(cluster_ctarank()), each = (vectors + ranks - 1) / ranks;
        const int column = 8 * each * rank;
        a.x += column;
        a.dy += column;
        a.dx += column;
        if (a.dsum != nullptr) a.dsum += column;
        if (a.weight != nullptr) a.weight += column;
        if (a.partials != nullptr) a.partials += column;
        vectors = min(each, vectors - each * rank);
        block /= ranks;
        blocks /= ranks;
        reduce.ranks = ranks;
        reduce.rank = rank;
        cluster_sync_all();   // every block has started: its shared memory may be written
    } else {
        reduce.size = team.size;
    }
    pdl_wait();
    const uint16_t* const weight = behind_wait(a.weight);
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    // The next row's x and dy are loaded ahead, and the packed weight stays in
    // registers.
    pair dw[NV][4];
    uint4 next_x[NV], next_d[NV], add[NV], w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = team.at + i * team.size;
        next_x[i] = next_d[i] = add[i] = make_uint4(0, 0, 0, 0);
        w[i] = weight_if(a.weight != nullptr && at < vectors, weight, at);
#pragma unroll
        for (int e = 0; e < 4; ++e) dw[i][e] = 0;
    }
    auto fetch = [&](const uint16_t* x_row, const uint16_t* d_row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            load_if(at < vectors, x_row + 8 * at, next_x[i]);
            load_if(at < vectors, d_row + 8 * at, next_d[i]);
        }
    };
    const int64_t step = static_cast<int64_t>(blocks) * team.rows;
    int64_t first = static_cast<int64_t>(block) * team.rows;
    const uint16_t* x_next = a.x + (first + team.row) * a.x_stride;
    const uint16_t* d_next = a.dy + (first + team.row) * a.dy_stride;
    if (first + team.row < a.rows) fetch(x_next, d_next);
    for (; first < a.rows; first += step) {
        const int64_t row = first + team.row;
        const int end = row < a.rows ? vectors : 0;
        uint4 x[NV], d[NV];
        const uint16_t* add_row = a.dsum + row * a.dsum_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            x[i] = next_x[i];
            d[i] = next_d[i];
            if (a.dsum != nullptr) load_if(at < end, add_row + 8 * at, add[i]);
        }
        x_next += step * a.x_stride;
        d_next += step * a.dy_stride;
        if (row + step < a.rows) fetch(x_next, d_next);
        const int64_t later = row + 2 * step;
        if (!kNarrow && threadIdx.x == 0) {
            if (later < a.rows) {
                prefetch_row(a.x + later * a.x_stride, 16 * vectors);
                prefetch_row(a.dy + later * a.dy_stride, 16 * vectors);
            }
            if (a.dsum != nullptr && row + step < a.rows) prefetch_row(a.dsum + (row + step) * a.dsum_stride, 16 * vectors);
        }
        // g = dy w
        auto g_of = [&](int i, const pair (&dy)[4], pair (&g)[4]) {
            if (a.weight != nullptr) {
                unpack8<kFp16>(w[i], g);
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = pair_mul(g[e], dy[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = dy[e];
            }
        };
        // sums of (s by)^2 and of (g g_by) (s by)
        auto sums = [&](float by, float g_by) {
            pair squares = 0, dot = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                pair v[4], dy[4], g[4];
                unpack8<kFp16>(x[i], v);
                unpack8<kFp16>(d[i], dy);
                g_of(i, dy, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (by != 1.0f) v[e] = pair_mul(v[e], pair_of(by));
                    if (g_by != 1.0f) g[e] = pair_mul(g[e], pair_of(g_by));
                    squares = pair_fma(v[e], v[e], squares);
                    dot = pair_fma(g[e], v[e], dot);
                }
            }
            const float2 both = reduce.sum2(pair_sum(squares), pair_sum(dot));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                forget(x[i]);
                forget(d[i]);
            }
            return both;
        };
        float2 both = sums(1.0f, 1.0f);
        float unit = rsqrtf(fmaf(both.x, inv_cols, a.eps));   // u = s unit
        float share = both.y * unit * inv_cols;               // mean(g u)
        // Out of FP32's range: once more, what left it scaled down.  |g| and |s|
        // are below 2^128 each, or s 2^64 where its squares hold: 32768 products
        // of the scaled ones do.  (A vote: rows of a warp differ, and the
        // reduction takes all of it.)
        const bool far_s = !(both.x <= 3.0e38f), far_g = !(fabsf(both.y) <= 3.0e38f);
        if (kNarrow ? __any_sync(0xFFFFFFFFu, far_s || far_g) : far_s || far_g) {
            const float down = far_s ? kDown : 1.0f, g_down = far_g ? kDown : 1.0f;
            both = sums(down, g_down);
            unit = rsqrtf(fmaf(both.x, inv_cols, a.eps * down * down));
            share = both.y * unit * inv_cols * (far_g ? 1.0f / kDown : 1.0f);
            unit *= down;
        }
        uint16_t* dx_row = a.dx + row * a.dx_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            if (kNarrow && end == 0) continue;   // dw: no row of this team's (zeros past a row)
            pair v[4], dy[4], g[4], more[4];
            unpack8<kFp16>(x[i], v);
            unpack8<kFp16>(d[i], dy);
            g_of(i, dy, g);
            unpack8<kFp16>(add[i], more);   // zeros without dsum
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const pair u = pair_mul(v[e], pair_of(unit));
                dw[i][e] = pair_fma(dy[e], u, dw[i][e]);
                g[e] = pair_fma(pair_fma(u, pair_of(-share), g[e]), pair_of(unit), more[e]);
            }
            store_if(at < end, dx_row + 8 * at, pack8<kFp16>(g));
        }
    }
    if (a.partials == nullptr) return;
    pdl_launch_dependents();   // the join's launch
    float* part = a.partials + static_cast<int64_t>(block) * a.cols;
    if constexpr (!kNarrow) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            if (at < vectors) store_sums(part + 8 * at, dw[i]);
        }
        return;
    }
    const int warp = kNarrow ? threadIdx.x >> 5 : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // narrow rows have two vectors a thread, 256 columns
        for (int o = team.size; o < 32; o *= 2)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dw[i][e] = pair_add(dw[i][e], __shfl_xor_sync(0xFFFFFFFFu, dw[i][e], o));
        const int at = team.at + i * team.size;
        if ((threadIdx.x & 31) < team.size && at < vectors) store_sums(columns[warp] + 8 * at, dw[i]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x)
        part[c] = columns[0][c] + columns[1][c] + columns[2][c] + columns[3][c];
}

// Columns' sums over parts: kLanes threads side by side take four columns each,
// the block's kThreads / kLanes runs of parts one under another.  (Pointers
// that may alias: the loads stay behind pdl_wait.)
template <int kLanes, int kThreads>
__global__ void __launch_bounds__(kThreads) join_columns_kernel(const float* partials, int parts, int cols,
                                                            float* out) {
    constexpr int kRuns = kThreads / kLanes, kColumns = 4 * kLanes;
    static_assert(kRuns % 8 == 0 && 8 * kColumns <= kThreads, "eight threads a column at the end");
    __shared__ float4 sums[kThreads];
    pdl_wait();
    const int lane = threadIdx.x % kLanes, run = threadIdx.x / kLanes;
    const int c = blockIdx.x * kColumns + 4 * lane;
    const int p0 = static_cast<int>(static_cast<int64_t>(parts) * run / kRuns);
    const int p1 = static_cast<int>(static_cast<int64_t>(parts) * (run + 1) / kRuns);
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < cols) {   // (a multiple of 8 columns in all)
#pragma unroll 4
        for (int p = p0; p < p1; ++p) {
            const float4 v = *reinterpret_cast<const float4*>(partials + static_cast<int64_t>(p) * cols + c);
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
        }
    }
    sums[threadIdx.x] = sum;
    __syncthreads();
    // eight threads a column add an eighth of its runs each, in their order,
    // and are added in theirs
    const int t = threadIdx.x >> 3, part = threadIdx.x & 7;
    if (t >= kColumns) return;   // whole warps
    const float* column = reinterpret_cast<const float*>(sums) + t + kColumns * (part * (kRuns / 8));
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < kRuns / 8; ++i) total += column[kColumns * i];
#pragma unroll
    for (int o = 1; o < 8; o *= 2) total += __shfl_down_sync(0xFFFFFFFFu, total, o, 8);
    const int at = static_cast<int>(blockIdx.x) * kColumns + t;
    if (part == 0 && at < cols) out[at] = total;
}

template <int NV, bool kFp16, bool kNarrow, bool kResidual>
cudaError_t run_norm_out(const NormArgs& a, int out, const RowPlan& p, cudaStream_t s) {
    const dim3 grid(p.blocks), block(p.threads);
    auto launch = [&](void (*kernel)(const NormArgs, int)) { return launch_kernel(kernel, grid, block, 0, s, a, p.team); };
    if (out == kNormRows) return launch(rmsnorm_kernel<NV, kFp16, kNormRows, kNarrow, kResidual>);
    if (out == kNormTensor) return launch(rmsnorm_kernel<NV, kFp16, kNormTensor, kNarrow, kResidual>);
    return launch(rmsnorm_kernel<NV, kFp16, kNormHalf, kNarrow, kResidual>);
}

template <int NV, bool kFp16, bool kNarrow>
cudaError_t run_norm_rows(const NormArgs& a, int out, const RowPlan& p, cudaStream_t s) {
    return a.residual != nullptr ? run_norm_out<NV, kFp16, kNarrow, true>(a, out, p, s)
                                 : run_norm_out<NV, kFp16, kNarrow, false>(a, out, p, s);
}

template <bool kFp16>
cudaError_t run_norm(const NormArgs& a, int out, const RowPlan& p, cudaStream_t s) {
    if (p.narrow) return run_norm_rows<2, kFp16, true>(a, out, p, s);
    if (p.each == 2) return run_norm_rows<2, kFp16, false>(a, out, p, s);
    return run_norm_rows<4, kFp16, false>(a, out, p, s);
}

// p.blocks: of rows, or clusters of `ranks` blocks.
struct GradPlan {
    RowPlan p;
    int ranks;
};
GradPlan grad_plan(int64_t rows, int cols, int sm_count) {
    constexpr int kLimits2[3] = {kGradThreads, 0, 0}, kPerSm2[3] = {kGradPerSm, 0, 0};
    if (cols <= kGradColumns) return {row_plan(rows, cols, sm_count, kLimits2, kPerSm2), 1};
    int ranks = 2;
    while (ranks * kGradColumns < cols) ranks *= 2;
    const int each = (cols / 8 + ranks - 1) / ranks;   // vectors of a block
    GradPlan g{{}, ranks};
    g.p.each = 2;
    g.p.team = g.p.threads = ((each + 1) / 2 + 31) / 32 * 32;
    const int64_t resident = std::max(1, sm_count * (kGradPerSm / g.p.threads) / ranks);
    g.p.blocks = static_cast<int>(std::min<int64_t>(rows, resident));
    return g;
}

// No more clusters than are resident at once (a GPC's last SMs may be too few
// for one; two clusters left over for a second round doubled the time).
template <bool kFp16>
cudaError_t fit_clusters(GradPlan* g) {
    constexpr int kDevices = 64, kSizes = kGradThreads / 32 + 1;
    static std::atomic<int> known[kDevices][kGradRanks + 1][kSizes];
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int>* const cell = dev < kDevices ? &known[dev][g->ranks][g->p.threads / 32] : nullptr;
    if (cell != nullptr) n = cell->load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(g->ranks);
        cfg.blockDim = dim3(g->p.threads);
        cudaLaunchAttribute ranks;
        ranks.id = cudaLaunchAttributeClusterDimension;
        ranks.val.clusterDim.x = static_cast<unsigned>(g->ranks);
        ranks.val.clusterDim.y = ranks.val.clusterDim.z = 1;
        cfg.attrs = &ranks;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, rmsnorm_grad_kernel<kFp16, kClusterRows>, &cfg);
        if (e != cudaSuccess) return e;
        n = std::max(n, 1);
        if (cell != nullptr) cell->store(n, std::memory_order_relaxed);
    }
    g->p.blocks = std::min(g->p.blocks, n);
    return cudaSuccess;
}

template <bool kFp16>
cudaError_t run_grad(const NormGradArgs& a, const GradPlan& g, cudaStream_t s) {
    const dim3 grid(g.p.blocks), block(g.p.threads);
    if (g.ranks > 1)
        return launch_clusters(rmsnorm_grad_kernel<kFp16, kClusterRows>, dim3(g.p.blocks * g.ranks), block, g.ranks, 0, s,
                               a, g.ranks);
    if (g.p.narrow) return launch_kernel(rmsnorm_grad_kernel<kFp16, kNarrowRows>, grid, block, 0, s, a, g.p.team);
    return launch_kernel(rmsnorm_grad_kernel<kFp16, kWideRows>, grid, block, 0, s, a, g.p.team);
}

}  // namespace

cudaError_t launch_join_columns(const float* partials, int parts, int cols, float* out, cudaStream_t s) {
    // 128 columns a block for wide sums (512 bytes of a part side by side); 32
    // for those that would leave SMs idle, with fewer threads where there is
    // little to add (the activation gradient of 63 x 2000 with dbias: 4.6 -> 3.7
    // us).
    if (cols >= 8192)
        return launch_kernel(join_columns_kernel<32, 1024>, dim3((cols + 127) / 128), dim3(1024), 0, s, partials, parts,
                             cols, out);
    if (parts > 256)
        return launch_kernel(join_columns_kernel<8, 1024>, dim3((cols + 31) / 32), dim3(1024), 0, s, partials, parts,
                             cols, out);
    return launch_kernel(join_columns_kernel<8, 256>, dim3((cols + 31) / 32), dim3(256), 0, s, partials, parts, cols,
                         out);
}

cudaError_t launch_rmsnorm(const NormArgs& args, int out, bool fp16, int sm_count, cudaStream_t s) {
    NormArgs a = args;
    float* after = nullptr;   // a next scale that only a further kernel can write
    if (out == kNormTensor) {
        if (a.rows == 0 || a.next_scale == a.scale) {
            after = a.next_scale;
            a.next_scale = nullptr;
        }
        const cudaError_t e = launch_kernel(zero_words_kernel, dim3(1), dim3(1), 0, s, a.amax_bits,
                                            reinterpret_cast<uint32_t*>(a.next_scale));
        if (e != cudaSuccess) return e;
    }
    if (a.rows > 0) {
        const RowPlan p = row_plan(a.rows, a.cols, sm_count, kLimits, kPerSm);
        const cudaError_t e = fp16 ? run_norm<true>(a, out, p, s) : run_norm<false>(a, out, p, s);
        if (e != cudaSuccess) return e;
    }
    if (after == nullptr) return cudaSuccess;
    return launch_kernel(next_scale_kernel, dim3(1), dim3(1), 0, s, reinterpret_cast<const float*>(a.amax_bits), after);
}

int64_t rmsnorm_grad_scratch_bytes(int64_t rows, int cols, int sm_count) {
    return static_cast<int64_t>(grad_plan(rows, cols, sm_count).p.blocks) * cols * 4;
}

cudaError_t launch_rmsnorm_grad(const NormGradArgs& a, bool fp16, float* dweight, int sm_count, cudaStream_t s) {
    GradPlan g = grad_plan(a.rows, a.cols, sm_count);
    if (g.ranks > 1 && a.rows > 0) {
        const cudaError_t e = fp16 ? fit_clusters<true>(&g) : fit_clusters<false>(&g);
        if (e != cudaSuccess) return e;
    }
    if (a.rows > 0) {
        const cudaError_t e = fp16 ? run_grad<true>(a, g, s) : run_grad<false>(a, g, s);
        if (e != cudaSuccess) return e;
    }
    return dweight == nullptr ? cudaSuccess : launch_join_columns(a.partials, g.p.blocks, a.cols, dweight, s);
}

}  // namespace dg
