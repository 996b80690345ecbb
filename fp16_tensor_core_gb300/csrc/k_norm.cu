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
// loads in flight while a row is reduced and written.
//
// Gradient, with u = s rsqrt(mean(s^2) + eps) and g = dy w:
//   dx = rsqrt(..) (g - u mean(g u)) + dsum,   dw = sum over rows of dy u
// dx belongs to x and to the residual alike.  A thread owns the same columns
// of every row of its block, so dw is summed in registers and leaves the
// block once; the blocks' sums are joined in order by a second kernel, so
// that results do not depend on timing.
#include <cuda_runtime.h>

#include <algorithm>

#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "row_common.cuh"

namespace dg {
namespace {

// A sum of squares past FP32's range is taken again of elements times this:
// 32768 squares of 2^128 2^-80 hold, and one element at least was above 2^56.
constexpr float kDown = 0x1p-80f;

// Threads of a block, and blocks an SM at least, by vectors a thread: the
// registers (64, 80, 128) hold a row and the next row's loads.
template <int NV>
constexpr int block_limit() { return NV == 4 ? 384 : 512; }
template <int NV>
constexpr int block_min() { return NV == 8 ? 1 : 2; }
constexpr int kLimits[3] = {512, 384, 512};
constexpr int kPerSm[3] = {1024, 768, 512};

template <int NV, bool kFp16, int kOut, bool kNarrow, bool kResidual>
__global__ void __launch_bounds__(block_limit<NV>(), block_min<NV>()) rmsnorm_kernel(const NormArgs a, int team_size) {
    __shared__ float2 buffer[2][kRowThreads / 32];
    pdl_wait();
    const uint16_t* const weight = behind_wait(a.weight);
    const RowTeam<kNarrow> team(team_size);
    RowReduce<kNarrow> reduce{buffer, team.size};
    const int vectors = a.cols >> 3;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    // The weight, packed, in registers where they reach; else it is read again
    // for every row.
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
    if (!kResidual && first + team.row + step < a.rows) load_row(x_next += step * a.x_stride, r);
    for (; first < a.rows; first += step) {
        const int64_t row = first + team.row;
        const int end = row < a.rows ? vectors : 0;   // this thread's vectors lie below
        pair v[NV][4], squares = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            unpack8<kFp16>(x[i], v[i]);
            if constexpr (kResidual) {
                pair add[4];
                unpack8<kFp16>(r[i], add);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = pair_add(v[i][e], add[e]);
            }
            if (a.sum != nullptr) store_if(at < end, a.sum + row * a.sum_stride + 8 * at, pack8<kFp16>(v[i]));
#pragma unroll
            for (int e = 0; e < 4; ++e) squares = pair_fma(v[i][e], v[i][e], squares);
        }
        if constexpr (kResidual) {
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
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const pair t = pair_mul(v[i][e], pair_of(down));
                    squares = pair_fma(t, t, squares);
                }
            total = reduce.sum(pair_sum(squares));
        }
        const float inv = rsqrtf(fmaf(total, inv_cols, a.eps * down * down)) * down;
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] = pair_mul(v[i][e], pair_of(inv));
            const int at = team.at + i * team.size;
            if (a.weight != nullptr) {
                pair f[4];
                unpack8<kFp16>(kKeepWeight ? w[i] : weight_if(at < vectors, weight, at), f);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = pair_mul(v[i][e], f[e]);
            }
            if (kOut != kNormHalf) top = top8(v[i], top);   // (zeros past the row)
        }
        if constexpr (kOut == kNormRows) {
            top = reduce.max1(top);
            by = row_factor(top);
            if (team.at == 0 && end != 0) a.row_scale[row] = row_scale(top);
        }
        if (kOut == kNormTensor && end != 0)   // (fmaxf would drop a NaN)
            tensor_top = __uint_as_float(max(__float_as_uint(tensor_top), __float_as_uint(top)));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            if constexpr (kOut == kNormHalf) {
                store_if(at < end, a.y + row * a.y_stride + 8 * at, pack8<kFp16>(v[i]));
            } else {
                if constexpr (kOut == kNormTensor) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[i][e] = pair_mul(v[i][e], pair_of(pre));
                }
                store_if(at < end, q_row + 8 * at, codes8(v[i], by));
            }
        }
        if (kOut != kNormHalf) q_row += step * a.cols;
    }
    if constexpr (kOut == kNormTensor) {
        // One atomic a block: a warp's each, on one address, took 5 us.
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

// The gradient's blocks: at most 128 registers a thread for the elements as
// they came, the columns' sums in FP32 and (two vectors a thread) the next
// row's loads.
constexpr int kGradLimits[3] = {512, 512, 512};
constexpr int kGradPerSm[3] = {512, 512, 512};

// Columns' sums of a block: the teams of a warp and then the warps are added in
// order; one partial a block.
template <int NV, bool kFp16, bool kNarrow>
__global__ void __launch_bounds__(kRowThreads, 1) rmsnorm_grad_kernel(const NormGradArgs a,
                                                                                         int team_size) {
    __shared__ float2 buffer[2][kRowThreads / 32];
    __shared__ float columns[kNarrow ? 4 : 1][256];   // four warps' sums
    pdl_wait();
    const uint16_t* const weight = behind_wait(a.weight);
    const RowTeam<kNarrow> team(team_size);
    RowReduce<kNarrow> reduce{buffer, team.size};
    const int vectors = a.cols >> 3;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    // Two vectors a thread: the next row's x and dy are loaded ahead, and the
    // packed weight stays in registers.
    constexpr bool kAhead = NV == 2;
    pair dw[NV][4];
    uint4 next_x[NV], next_d[NV], add[NV], w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = team.at + i * team.size;
        next_x[i] = next_d[i] = add[i] = make_uint4(0, 0, 0, 0);
        if (kAhead) w[i] = weight_if(a.weight != nullptr && at < vectors, weight, at);
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
    const int64_t step = static_cast<int64_t>(gridDim.x) * team.rows;
    int64_t first = static_cast<int64_t>(blockIdx.x) * team.rows;
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
        if (kAhead && row + step < a.rows) fetch(x_next, d_next);
        const int64_t later = row + (kAhead ? 2 : 1) * step;
        if (!kNarrow && threadIdx.x == 0) {
            if (later < a.rows) {
                prefetch_row(a.x + later * a.x_stride, 2 * a.cols);
                prefetch_row(a.dy + later * a.dy_stride, 2 * a.cols);
            }
            if (a.dsum != nullptr && row + step < a.rows) prefetch_row(a.dsum + (row + step) * a.dsum_stride, 2 * a.cols);
        }
        // g = dy w
        auto g_of = [&](int i, const pair (&dy)[4], pair (&g)[4]) {
            const int at = team.at + i * team.size;
            if (a.weight != nullptr) {
                unpack8<kFp16>(kAhead ? w[i] : weight_if(at < vectors, weight, at), g);
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = pair_mul(g[e], dy[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = dy[e];
            }
        };
        // sums of (s by)^2 and of g s by
        auto sums = [&](float by) {
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
        float down = 1.0f;
        float2 both = sums(1.0f);
        // Out of FP32's range: once more, scaled down.  (A vote: rows of a warp
        // differ, and the reduction takes all of it.)
        const bool again = !(both.x <= 3.0e38f);
        if (kNarrow ? __any_sync(0xFFFFFFFFu, again) : again) {
            down = again ? kDown : 1.0f;
            both = sums(down);
        }
        const float inv = rsqrtf(fmaf(both.x, inv_cols, a.eps * down * down));
        const float share = both.y * inv * inv_cols;   // mean(g u)
        const float unit = inv * down;                 // u = s unit
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
        if (!kAhead && row + step < a.rows) fetch(x_next, d_next);
    }
    if (a.partials == nullptr) return;
    pdl_launch_dependents();   // the join's launch
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * a.cols;
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
    if (p.each == 4) return run_norm_rows<4, kFp16, false>(a, out, p, s);
    return run_norm_rows<8, kFp16, false>(a, out, p, s);
}

RowPlan grad_plan(int64_t rows, int cols, int sm_count) {
    return row_plan(rows, cols, sm_count, kGradLimits, kGradPerSm);
}

template <bool kFp16>
cudaError_t run_grad(const NormGradArgs& a, const RowPlan& p, cudaStream_t s) {
    const dim3 grid(p.blocks), block(p.threads);
    if (p.narrow) return launch_kernel(rmsnorm_grad_kernel<2, kFp16, true>, grid, block, 0, s, a, p.team);
    if (p.each == 2) return launch_kernel(rmsnorm_grad_kernel<2, kFp16, false>, grid, block, 0, s, a, p.team);
    if (p.each == 4) return launch_kernel(rmsnorm_grad_kernel<4, kFp16, false>, grid, block, 0, s, a, p.team);
    return launch_kernel(rmsnorm_grad_kernel<8, kFp16, false>, grid, block, 0, s, a, p.team);
}

}  // namespace

cudaError_t launch_join_columns(const float* partials, int parts, int cols, float* out, cudaStream_t s) {
    // 128 columns a block for wide sums (110 parts of 22016: 2.2 times as fast
    // as 32); 32 for those that would leave SMs idle, with fewer threads where
    // there is little to add (63 parts of 2000: 0.8 us).
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
    return static_cast<int64_t>(grad_plan(rows, cols, sm_count).blocks) * cols * 4;
}

cudaError_t launch_rmsnorm_grad(const NormGradArgs& a, bool fp16, float* dweight, int sm_count, cudaStream_t s) {
    const RowPlan p = grad_plan(a.rows, a.cols, sm_count);
    if (a.rows > 0) {
        const cudaError_t e = fp16 ? run_grad<true>(a, p, s) : run_grad<false>(a, p, s);
        if (e != cudaSuccess) return e;
    }
    return dweight == nullptr ? cudaSuccess : launch_join_columns(a.partials, p.blocks, a.cols, dweight, s);
}

}  // namespace dg
