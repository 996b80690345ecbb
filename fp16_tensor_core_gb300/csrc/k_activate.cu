// k_activate.cu -- the activation between two products, gated or not, with
// E4M3 output and an 8-bit checkpoint of its input, and its gradient.
//
//   y = act(x)              or, gated, act(x[:, :n]) * x[:, n:]
//   out: y rounded; codes E4M3(y / scale) with scale = amax / 448 of the row;
//   x itself as codes, with a scale per row and half ([FP8-guide] §3.2's rule
//   with that as the tensor), which the backward pass reads in its place.
// [FP8-guide] = "DeepGEMM实战：FP8矩阵乘法与JIT编译优化指南".
//
// Gradient:  dx = dy act'(x)   or   (dy up act'(gate), dy act(gate)),
//            dbias = sum over rows of dx (before its rounding).
//
// Memory bounds both: 2 bytes an input element and 1 to 3 of output; the
// checkpoint halves what the backward pass reads of the input.  Forward, a
// block keeps a row in registers until the maxima of the row are known and
// has the next row's loads in flight.  Backward needs nothing of a row but
// its scales: a thread owns eight columns over a run of rows, so that dbias
// is summed in registers; the runs' sums are joined in order by a second
// kernel.
#include <cuda_runtime.h>

#include <algorithm>

#include "activation.cuh"
#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "row_common.cuh"

namespace dg {
namespace {

template <int NV, bool kFp16, bool kGated>
__global__ void __launch_bounds__(kRowThreads) activate_kernel(const ActArgs a) {
    __shared__ float2 buffer[2][kRowThreads / 32];
    pdl_wait();
    RowReduce reduce{buffer};
    constexpr int kHalves = kGated ? 2 : 1;
    const int vectors = a.cols >> 3, t = threadIdx.x, step = blockDim.x;
    uint4 x[kHalves][NV];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int i = 0; i < NV; ++i) x[h][i] = make_uint4(0, 0, 0, 0);
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (t + i * step < vectors)
                    x[h][i] = load_once(a.x + row * a.x_stride + static_cast<int64_t>(h) * a.cols + 8 * (t + i * step));
    };
    int64_t row = blockIdx.x;
    if (row < a.rows) fetch(row);
    for (; row < a.rows; row += gridDim.x) {
        if (a.x_q != nullptr) {
            uint32_t top[2] = {0, 0};
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float f[8];
                    unpack8<kFp16>(x[h][i], f);
                    top[h] = max(top[h], top8(f));
                }
            const uint2 both = reduce.max2(top[0], top[1]);
            const float scale[2] = {row_scale(both.x), row_scale(both.y)};
            if (t < kHalves) a.x_scale[row * kHalves + t] = scale[t];
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const float by = __frcp_rn(scale[h]);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (t + i * step >= vectors) continue;
                    float f[8];
                    unpack8<kFp16>(x[h][i], f);
                    *reinterpret_cast<uint2*>(a.x_q + (row * kHalves + h) * a.cols + 8 * (t + i * step)) =
                        codes8(f, by);
                }
            }
        }
        if (a.y == nullptr && a.q == nullptr) {
            if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
            continue;
        }
        float y[NV][8];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack8<kFp16>(x[0][i], y[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][e] = activation(a.act, y[i][e]);
            if constexpr (kGated) {
                float up[8];
                unpack8<kFp16>(x[kHalves - 1][i], up);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[i][e] *= up[e];
            }
            top = max(top, top8(y[i]));
        }
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
        if (a.y != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (t + i * step < vectors)
                    *reinterpret_cast<uint4*>(a.y + row * a.y_stride + 8 * (t + i * step)) = pack8<kFp16>(y[i]);
        }
        if (a.q != nullptr) {
            const float scale = row_scale(reduce.max1(top));
            const float by = __frcp_rn(scale);
            if (t == 0) a.q_scale[row] = scale;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (t + i * step < vectors)
                    *reinterpret_cast<uint2*>(a.q + row * a.cols + 8 * (t + i * step)) = codes8(y[i], by);
        }
    }
}

constexpr int kGradThreads = 128;   // 1024 columns a block

template <bool kFp16, bool kGated, bool kCodes>
__global__ void __launch_bounds__(kGradThreads) activate_grad_kernel(const ActGradArgs a) {
    pdl_wait();
    constexpr int kHalves = kGated ? 2 : 1;
    const int c = 8 * static_cast<int>(blockIdx.x * kGradThreads + threadIdx.x);
    if (c >= a.cols) return;
    const int64_t first = a.rows * blockIdx.y / gridDim.y, end = a.rows * (blockIdx.y + 1) / gridDim.y;
    const int64_t width = static_cast<int64_t>(kHalves) * a.cols;
    float sums[kHalves][8];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[h][e] = 0.0f;
#pragma unroll 2
    for (int64_t row = first; row < end; ++row) {
        float dy[8], x[kHalves][8];
        unpack8<kFp16>(load_once(a.dy + row * a.dy_stride + c), dy);
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            if constexpr (kCodes)
                decode8(load_once8(a.x_q + row * width + static_cast<int64_t>(h) * a.cols + c),
                        __ldg(a.x_scale + row * kHalves + h), x[h]);
            else
                unpack8<kFp16>(load_once(a.x + row * a.x_stride + static_cast<int64_t>(h) * a.cols + c), x[h]);
        }
        float dx[kHalves][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const ValueSlope f = activation_slope(a.act, x[0][e]);
            if constexpr (kGated) {
                dx[0][e] = dy[e] * x[kHalves - 1][e] * f.slope;
                dx[kHalves - 1][e] = dy[e] * f.value;
            } else {
                dx[0][e] = dy[e] * f.slope;
            }
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sums[h][e] += dx[h][e];
            *reinterpret_cast<uint4*>(a.dx + row * a.dx_stride + static_cast<int64_t>(h) * a.cols + c) =
                pack8<kFp16>(dx[h]);
        }
    }
    if (a.partials != nullptr) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            float4* dst = reinterpret_cast<float4*>(a.partials + blockIdx.y * width + static_cast<int64_t>(h) * a.cols + c);
            dst[0] = make_float4(sums[h][0], sums[h][1], sums[h][2], sums[h][3]);
            dst[1] = make_float4(sums[h][4], sums[h][5], sums[h][6], sums[h][7]);
        }
    }
}

// Vectors a thread: up to 2 of each half, more for wide rows.
int act_vectors_each(int vectors) {
    for (int each = 2; each < kRowVectors; each *= 2)
        if (row_threads(vectors, each) <= kRowThreads) return each;
    return kRowVectors;
}

template <int NV, bool kFp16>
cudaError_t run_act(const ActArgs& a, int sm_count, cudaStream_t s) {
    const int threads = row_threads(a.cols >> 3, NV);
    const int64_t blocks = std::min<int64_t>(a.rows, static_cast<int64_t>(sm_count) * std::max(1, 1024 / threads));
    const dim3 grid(static_cast<unsigned>(blocks)), block(threads);
    return a.gated ? launch_kernel(activate_kernel<NV, kFp16, true>, grid, block, 0, s, a)
                   : launch_kernel(activate_kernel<NV, kFp16, false>, grid, block, 0, s, a);
}

template <int NV>
cudaError_t run_act_type(const ActArgs& a, bool fp16, int sm_count, cudaStream_t s) {
    return fp16 ? run_act<NV, true>(a, sm_count, s) : run_act<NV, false>(a, sm_count, s);
}

// Runs of rows: enough blocks for 16 an SM over all column blocks, but no
// run without a row.
int act_grad_runs(int64_t rows, int cols, int sm_count) {
    const int64_t column_blocks = (cols / 8 + kGradThreads - 1) / kGradThreads;
    const int64_t runs = std::max<int64_t>(1, static_cast<int64_t>(sm_count) * 16 / column_blocks);
    return static_cast<int>(std::min(rows, runs));
}

template <bool kFp16, bool kGated>
cudaError_t run_act_grad(const ActGradArgs& a, int runs, cudaStream_t s) {
    const dim3 grid((a.cols / 8 + kGradThreads - 1) / kGradThreads, runs), block(kGradThreads);
    return a.x_q != nullptr ? launch_kernel(activate_grad_kernel<kFp16, kGated, true>, grid, block, 0, s, a)
                            : launch_kernel(activate_grad_kernel<kFp16, kGated, false>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_activate(const ActArgs& a, bool fp16, int sm_count, cudaStream_t s) {
    switch (act_vectors_each(a.cols >> 3)) {
        case 2: return run_act_type<2>(a, fp16, sm_count, s);
        case 4: return run_act_type<4>(a, fp16, sm_count, s);
        default: return run_act_type<8>(a, fp16, sm_count, s);
    }
}

int64_t activate_grad_scratch_bytes(int64_t rows, int cols, bool gated, int sm_count) {
    return static_cast<int64_t>(act_grad_runs(rows, cols, sm_count)) * cols * (gated ? 8 : 4);
}

cudaError_t launch_activate_grad(const ActGradArgs& a, bool fp16, float* dbias, int sm_count, cudaStream_t s) {
    const int runs = act_grad_runs(a.rows, a.cols, sm_count);
    if (runs > 0) {
        const cudaError_t e = fp16 ? (a.gated ? run_act_grad<true, true>(a, runs, s) : run_act_grad<true, false>(a, runs, s))
                                   : (a.gated ? run_act_grad<false, true>(a, runs, s) : run_act_grad<false, false>(a, runs, s));
        if (e != cudaSuccess) return e;
    }
    return dbias == nullptr ? cudaSuccess
                            : launch_join_columns(a.partials, runs, a.gated ? 2 * a.cols : a.cols, dbias, s);
}

}  // namespace dg
