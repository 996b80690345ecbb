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

template <int NV, bool kFp16, int kOut>
__global__ void __launch_bounds__(block_limit<NV>(), block_min<NV>()) rmsnorm_kernel(const NormArgs a, int team_size) {
    __shared__ float2 buffer[2][kRowThreads / 32];
    pdl_wait();
    const RowTeam team = row_team(team_size);
    RowReduce reduce{buffer, team.size};
    const int vectors = a.cols >> 3;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    uint4 x[NV], r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = r[i] = make_uint4(0, 0, 0, 0);
    auto fetch = [&](int64_t row) {
        if (row >= a.rows) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            if (at >= vectors) continue;
            x[i] = load_once(a.x + row * a.x_stride + 8 * at);
            if (a.residual != nullptr) r[i] = load_once(a.residual + row * a.residual_stride + 8 * at);
        }
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
    for (; first < a.rows; first += step) {
        const int64_t row = first + team.row;
        const int end = row < a.rows ? vectors : 0;   // this thread's vectors lie below
        pair v[NV][4], squares = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            unpack8<kFp16>(x[i], v[i]);
            if (a.residual != nullptr) {
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
        fetch(row + step);
        float total = reduce.sum(pair_sum(squares)), eps = a.eps;
        // (a vote: rows of a warp differ, and the reduction takes all of it)
        const bool again = !(total <= 3.0e38f);
        if (team.size < 32 ? __any_sync(0xFFFFFFFFu, again) : again) {
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
        const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(tensor_top));
        if ((threadIdx.x & 31) == 0 && bits != 0) atomicMax(a.amax_bits, bits);
        if (a.next_scale != nullptr) {
            // The last block to arrive forms the next call's scale; the word
            // counts the arrivals until then (it is zeroed with the maximum).
            __syncthreads();
            if (threadIdx.x == 0) {
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

// Columns' sums of a block: the teams of a warp and then the warps are added in
// order; one partial a block.
template <int NV>
constexpr int grad_limit() { return NV == 2 ? 384 : 512; }
template <int NV>
constexpr int grad_min() { return NV == 2 ? 2 : 1; }
constexpr int kGradLimits[3] = {384, 512, 512};
constexpr int kGradPerSm[3] = {768, 512, 512};

template <int NV, bool kFp16>
__global__ void __launch_bounds__(grad_limit<NV>(), grad_min<NV>()) rmsnorm_grad_kernel(const NormGradArgs a,
                                                                                         int team_size) {
    __shared__ float2 buffer[2][kRowThreads / 32];
    __shared__ float columns[4][256];   // narrow rows: four warps' sums
    pdl_wait();
    const RowTeam team = row_team(team_size);
    RowReduce reduce{buffer, team.size};
    const int vectors = a.cols >> 3;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    constexpr bool kAhead = NV == 2;   // the next row's loads in flight: registers
    pair dw[NV][4];
    uint4 x[NV], d[NV], next_d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        x[i] = next_d[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) dw[i][e] = 0;
    }
    auto fetch = [&](int64_t row) {
        if (row >= a.rows) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            if (at >= vectors) continue;
            x[i] = load_once(a.x + row * a.x_stride + 8 * at);
            next_d[i] = load_once(a.dy + row * a.dy_stride + 8 * at);
        }
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * team.rows;
    int64_t first = static_cast<int64_t>(blockIdx.x) * team.rows;
    if (kAhead) fetch(first + team.row);
    for (; first < a.rows; first += step) {
        const int64_t row = first + team.row;
        const int end = row < a.rows ? vectors : 0;
        if (!kAhead) fetch(row);
        pair v[NV][4];
        uint4 add[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            add[i] = make_uint4(0, 0, 0, 0);
            if (a.dsum != nullptr && at < end) add[i] = load_once(a.dsum + row * a.dsum_stride + 8 * at);
            unpack8<kFp16>(x[i], v[i]);
            d[i] = next_d[i];
        }
        if (kAhead) fetch(row + step);
        // dy, and g = dy w, formed where they are needed: registers
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
        float2 both;   // sums of s^2 and of g s
        auto sums = [&]() {
            pair squares = 0, dot = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                pair dy[4], g[4];
                g_of(i, dy, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    squares = pair_fma(v[i][e], v[i][e], squares);
                    dot = pair_fma(g[e], v[i][e], dot);
                }
            }
            both = reduce.sum2(pair_sum(squares), pair_sum(dot));
        };
        sums();
        float eps = a.eps, down = 1.0f;
        const bool again = !(both.x <= 3.0e38f);
        if (team.size < 32 ? __any_sync(0xFFFFFFFFu, again) : again) {
            down = again ? kDown : 1.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = pair_mul(v[i][e], pair_of(down));
            sums();
            eps = eps * down * down;
        }
        const float inv = rsqrtf(fmaf(both.x, inv_cols, eps));
        const float share = both.y * inv * inv_cols;   // mean(g u)
        const float out_by = inv * down;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            if (at >= end) continue;
            pair dy[4], g[4], more[4];
            g_of(i, dy, g);
            unpack8<kFp16>(add[i], more);   // zeros without dsum
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const pair u = pair_mul(v[i][e], pair_of(inv));
                dw[i][e] = pair_fma(dy[e], u, dw[i][e]);
                g[e] = pair_fma(pair_fma(u, pair_of(-share), g[e]), pair_of(out_by), more[e]);
            }
            *reinterpret_cast<uint4*>(a.dx + row * a.dx_stride + 8 * at) = pack8<kFp16>(g);
        }
    }
    if (a.partials == nullptr) return;
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * a.cols;
    if (team.size >= 32) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = team.at + i * team.size;
            if (at < vectors) store_sums(part + 8 * at, dw[i]);
        }
        return;
    }
    const int warp = threadIdx.x >> 5;
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

template <int NV, bool kFp16>
cudaError_t run_norm(const NormArgs& a, int out, const RowPlan& p, cudaStream_t s) {
    const dim3 grid(p.blocks), block(p.threads);
    if (out == kNormRows) return launch_kernel(rmsnorm_kernel<NV, kFp16, kNormRows>, grid, block, 0, s, a, p.team);
    if (out == kNormTensor) return launch_kernel(rmsnorm_kernel<NV, kFp16, kNormTensor>, grid, block, 0, s, a, p.team);
    return launch_kernel(rmsnorm_kernel<NV, kFp16, kNormHalf>, grid, block, 0, s, a, p.team);
}

template <int NV>
cudaError_t run_norm_type(const NormArgs& a, int out, bool fp16, const RowPlan& p, cudaStream_t s) {
    return fp16 ? run_norm<NV, true>(a, out, p, s) : run_norm<NV, false>(a, out, p, s);
}

RowPlan grad_plan(int64_t rows, int cols, int sm_count) {
    return row_plan(rows, cols, sm_count, kGradLimits, kGradPerSm);
}

template <int NV>
cudaError_t run_grad(const NormGradArgs& a, bool fp16, const RowPlan& p, cudaStream_t s) {
    const dim3 grid(p.blocks), block(p.threads);
    return fp16 ? launch_kernel(rmsnorm_grad_kernel<NV, true>, grid, block, 0, s, a, p.team)
                : launch_kernel(rmsnorm_grad_kernel<NV, false>, grid, block, 0, s, a, p.team);
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
        const cudaError_t e = p.each == 2   ? run_norm_type<2>(a, out, fp16, p, s)
                              : p.each == 4 ? run_norm_type<4>(a, out, fp16, p, s)
                                            : run_norm_type<8>(a, out, fp16, p, s);
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
        const cudaError_t e = p.each == 2   ? run_grad<2>(a, fp16, p, s)
                              : p.each == 4 ? run_grad<4>(a, fp16, p, s)
                                            : run_grad<8>(a, fp16, p, s);
        if (e != cudaSuccess) return e;
    }
    return dweight == nullptr ? cudaSuccess : launch_join_columns(a.partials, p.blocks, a.cols, dweight, s);
}

}  // namespace dg
