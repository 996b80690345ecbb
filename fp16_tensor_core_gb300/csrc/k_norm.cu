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

// A sum of squares past FP32's range is taken again of elements times this.
constexpr float kDown = 0x1p-64f;

// Threads of a block, and blocks an SM at least, by vectors a thread: the
// registers (64, 80, 128) hold a row and the next row's loads.
template <int NV>
constexpr int block_limit() { return NV == 4 ? 384 : 512; }
template <int NV>
constexpr int block_min() { return NV == 8 ? 1 : 2; }
constexpr int kLimits[3] = {512, 384, 512};
constexpr int kPerSm[3] = {1024, 768, 512};

// A vector of the weight: every block reads it for every row, from L1.
__device__ __forceinline__ uint4 weight_at(const uint16_t* weight, int at) {
    return __ldg(reinterpret_cast<const uint4*>(weight) + at);
}

template <int NV, bool kFp16, int kOut, bool kNarrow, bool kResidual>
__global__ void __launch_bounds__(block_limit<NV>(), block_min<NV>()) rmsnorm_kernel(const NormArgs a, int team_size) {
    __shared__ float2 buffer[2][kRowThreads / 32];
    pdl_wait();
    const RowTeam<kNarrow> team(team_size);
    RowReduce<kNarrow> reduce{buffer, team.size};
    const int vectors = a.cols >> 3;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    uint4 x[NV], r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = r[i] = make_uint4(0, 0, 0, 0);
    // The next row's loads are in flight while a row is worked on: x and r; or,
    // without a residual, those of the next two rows (x, then r).
    auto load_row = [&](const uint16_t* row, uint4 (&to)[NV]) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (team.at + i * team.size < vectors) to[i] = load_once(row + 8 * (team.at + i * team.size));
    };
    auto fetch = [&](int64_t row) {
        if (row >= a.rows) return;
        load_row(a.x + row * a.x_stride, x);
        if constexpr (kResidual) load_row(a.residual + row * a.residual_stride, r);
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
    fetch(first + team.row);
    if (!kResidual && first + team.row + step < a.rows) load_row(a.x + (first + team.row + step) * a.x_stride, r);
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
            if (a.sum != nullptr && at < end)
                *reinterpret_cast<uint4*>(a.sum + row * a.sum_stride + 8 * at) = pack8<kFp16>(v[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) squares = pair_fma(v[i][e], v[i][e], squares);
        }
        if constexpr (kResidual) {
            fetch(row + step);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) x[i] = r[i];
            if (row + 2 * step < a.rows) load_row(a.x + (row + 2 * step) * a.x_stride, r);
        }
        float total = reduce.sum(pair_sum(squares)), eps = a.eps;
        // (a vote: rows of a warp differ, and the reduction takes all of it)
        const bool again = !(total <= 3.0e38f);
        if (kNarrow ? __any_sync(0xFFFFFFFFu, again) : again) {
            const float down = again ? kDown : 1.0f;
            squares = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[i][e] = pair_mul(v[i][e], pair_of(down));
                    squares = pair_fma(v[i][e], v[i][e], squares);
                }
            total = reduce.sum(pair_sum(squares));
            eps = eps * down * down;
        }
        const float inv = rsqrtf(fmaf(total, inv_cols, eps));
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] = pair_mul(v[i][e], pair_of(inv));
            if (a.weight != nullptr && team.at + i * team.size < vectors) {
                pair f[4];
                unpack8<kFp16>(weight_at(a.weight, team.at + i * team.size), f);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = pair_mul(v[i][e], f[e]);
            }
            if (kOut != kNormHalf && team.at + i * team.size < end) top = top8(v[i], top);
        }
        if constexpr (kOut == kNormRows) {
            const float scale = row_scale(reduce.max1(top));
            by = __frcp_rn(scale);
            if (team.at == 0 && end != 0) a.row_scale[row] = scale;
        }
        if constexpr (kOut == kNormTensor)   // (fmaxf would drop a NaN)
            tensor_top = __uint_as_float(max(__float_as_uint(tensor_top), __float_as_uint(top)));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            if (at >= end) continue;
            if constexpr (kOut == kNormHalf) {
                *reinterpret_cast<uint4*>(a.y + row * a.y_stride + 8 * at) = pack8<kFp16>(v[i]);
            } else {
                if constexpr (kOut == kNormTensor) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[i][e] = pair_mul(v[i][e], pair_of(pre));
                }
                *reinterpret_cast<uint2*>(a.q + row * a.cols + 8 * at) = codes8(v[i], by);
            }
        }
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
    const RowTeam<kNarrow> team(team_size);
    RowReduce<kNarrow> reduce{buffer, team.size};
    const int vectors = a.cols >> 3;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    constexpr bool kAhead = NV == 2;
    pair dw[NV][4];
    uint4 next_x[NV], next_d[NV], next_add[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        next_x[i] = next_d[i] = next_add[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) dw[i][e] = 0;
    }
    auto fetch = [&](int64_t row) {
        if (row >= a.rows) return;
        const uint16_t* x_row = a.x + row * a.x_stride;
        const uint16_t* d_row = a.dy + row * a.dy_stride;
        const uint16_t* add_row = a.dsum + row * a.dsum_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            if (at >= vectors) continue;
            next_x[i] = load_once(x_row + 8 * at);
            next_d[i] = load_once(d_row + 8 * at);
            if (a.dsum != nullptr) next_add[i] = load_once(add_row + 8 * at);
        }
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * team.rows;
    int64_t first = static_cast<int64_t>(blockIdx.x) * team.rows;
    if (kAhead) fetch(first + team.row);
    for (; first < a.rows; first += step) {
        const int64_t row = first + team.row;
        const int end = row < a.rows ? vectors : 0;
        if (!kAhead) fetch(row);
        uint4 x[NV], d[NV], add[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = next_x[i];
            d[i] = next_d[i];
            add[i] = next_add[i];
        }
        if (kAhead) fetch(row + step);
        const int64_t later = row + (kAhead ? 2 : 1) * step;
        if (!kNarrow && threadIdx.x == 0 && later < a.rows) {
            prefetch_row(a.x + later * a.x_stride, 2 * a.cols);
            prefetch_row(a.dy + later * a.dy_stride, 2 * a.cols);
            if (a.dsum != nullptr) prefetch_row(a.dsum + later * a.dsum_stride, 2 * a.cols);
        }
        // dy, and g = dy w
        auto g_of = [&](int i, pair (&dy)[4], pair (&g)[4]) {
            unpack8<kFp16>(d[i], dy);
            const int at = team.at + i * team.size;
            if (a.weight != nullptr && at < vectors) {
                unpack8<kFp16>(weight_at(a.weight, at), g);
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = pair_mul(g[e], dy[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = dy[e];
            }
        };
        float down = 1.0f, eps = a.eps;
        float2 both;   // sums of (s down)^2 and of g s down
        bool again = false;   // out of FP32's range: once more, scaled down
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            down = again ? kDown : 1.0f;
            pair squares = 0, dot = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                pair v[4], dy[4], g[4];
                unpack8<kFp16>(x[i], v);
                g_of(i, dy, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = pair_mul(v[e], pair_of(down));
                    squares = pair_fma(v[e], v[e], squares);
                    dot = pair_fma(g[e], v[e], dot);
                }
            }
            both = reduce.sum2(pair_sum(squares), pair_sum(dot));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                forget(x[i]);
                forget(d[i]);
            }
            again = pass == 0 && !(both.x <= 3.0e38f);
            // (a vote: rows of a warp differ, and the reduction takes all of it)
            if (kNarrow ? !__any_sync(0xFFFFFFFFu, again) : !again) break;
        }
        eps = eps * down * down;
        const float inv = rsqrtf(fmaf(both.x, inv_cols, eps));
        const float share = both.y * inv * inv_cols;   // mean(g u)
        const float unit = inv * down;                 // u = s unit
        uint16_t* dx_row = a.dx + row * a.dx_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            if (at >= end) continue;
            pair v[4], dy[4], g[4], more[4];
            unpack8<kFp16>(x[i], v);
            g_of(i, dy, g);
            unpack8<kFp16>(add[i], more);   // zeros without dsum
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const pair u = pair_mul(v[e], pair_of(unit));
                dw[i][e] = pair_fma(dy[e], u, dw[i][e]);
                g[e] = pair_fma(pair_fma(u, pair_of(-share), g[e]), pair_of(unit), more[e]);
            }
            *reinterpret_cast<uint4*>(dx_row + 8 * at) = pack8<kFp16>(g);
        }
    }
    if (a.partials == nullptr) return;
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

// 32 warps take a run of parts each, 32 columns a block.
__global__ void __launch_bounds__(1024) join_columns_kernel(const float* __restrict__ partials, int parts, int cols,
                                                            float* __restrict__ out) {
    __shared__ float run[32][33];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const int p0 = static_cast<int>(static_cast<int64_t>(parts) * warp / 32);
    const int p1 = static_cast<int>(static_cast<int64_t>(parts) * (warp + 1) / 32);
    float sum = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int p = p0; p < p1; ++p) sum += partials[static_cast<int64_t>(p) * cols + c];
    }
    run[warp][lane] = sum;
    __syncthreads();
    // warp i adds column i's runs, as a tree in their order
    sum = run[lane][warp];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) sum += __shfl_down_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0 && static_cast<int>(blockIdx.x) * 32 + warp < cols) out[blockIdx.x * 32 + warp] = sum;
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
    return launch_kernel(join_columns_kernel, dim3((cols + 31) / 32), dim3(1024), 0, s, partials, parts, cols, out);
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
