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

template <int NV, bool kFp16, int kOut>
__global__ void __launch_bounds__(kRowThreads) rmsnorm_kernel(const NormArgs a) {
    __shared__ float2 buffer[2][kRowThreads / 32];
    pdl_wait();
    RowReduce reduce{buffer};
    const int vectors = a.cols >> 3, t = threadIdx.x, step = blockDim.x;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    uint4 w[NV], x[NV], r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        w[i] = x[i] = r[i] = make_uint4(0, 0, 0, 0);
        if (a.weight != nullptr && t + i * step < vectors)
            w[i] = __ldg(reinterpret_cast<const uint4*>(a.weight) + t + i * step);
    }
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (t + i * step >= vectors) continue;
            x[i] = load_once(a.x + row * a.x_stride + 8 * (t + i * step));
            if (a.residual != nullptr) r[i] = load_once(a.residual + row * a.residual_stride + 8 * (t + i * step));
        }
    };
    float pre = 1.0f, by = 0.0f;
    if constexpr (kOut == kNormTensor) {
        const ByScale given = by_scale(*a.scale);
        pre = given.pre;
        by = given.inv;
    }
    uint32_t tensor_top = 0;
    int64_t row = blockIdx.x;
    if (row < a.rows) fetch(row);
    for (; row < a.rows; row += gridDim.x) {
        float v[NV][8];
        float squares = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack8<kFp16>(x[i], v[i]);
            if (a.residual != nullptr) {
                float add[8];
                unpack8<kFp16>(r[i], add);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] += add[e];
            }
            if (a.sum != nullptr && t + i * step < vectors)
                *reinterpret_cast<uint4*>(a.sum + row * a.sum_stride + 8 * (t + i * step)) = pack8<kFp16>(v[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) squares = fmaf(v[i][e], v[i][e], squares);
        }
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
        squares = reduce.sum(squares);
        float eps = a.eps;
        if (!(squares <= 3.0e38f)) {   // the whole block
            squares = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[i][e] *= kDown;
                    squares = fmaf(v[i][e], v[i][e], squares);
                }
            squares = reduce.sum(squares);
            eps = eps * kDown * kDown;
        }
        const float inv = rsqrtf(fmaf(squares, inv_cols, eps));
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[8];
            unpack8<kFp16>(w[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * inv * (a.weight != nullptr ? f[e] : 1.0f);
            if (kOut != kNormHalf && t + i * step < vectors) top = max(top, top8(v[i]));
        }
        if constexpr (kOut == kNormRows) {
            const float scale = row_scale(reduce.max1(top));
            by = __frcp_rn(scale);
            if (t == 0) a.row_scale[row] = scale;
        }
        if constexpr (kOut == kNormTensor) tensor_top = max(tensor_top, top);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = t + i * step;
            if (at >= vectors) continue;
            if constexpr (kOut == kNormHalf) {
                *reinterpret_cast<uint4*>(a.y + row * a.y_stride + 8 * at) = pack8<kFp16>(v[i]);
            } else {
                if constexpr (kOut == kNormTensor) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] *= pre;
                }
                *reinterpret_cast<uint2*>(a.q + row * a.cols + 8 * at) = codes8(v[i], by);
            }
        }
    }
    if constexpr (kOut == kNormTensor) {
        tensor_top = reduce.max1(tensor_top);
        if (t == 0 && tensor_top != 0) atomicMax(a.amax_bits, tensor_top);
    }
}

// amax / 448 (1 for an all-zero tensor), when the blocks' maxima are in.
__global__ void next_scale_kernel(const float* amax, float* scale) {
    pdl_wait();
    const float a = *amax;
    *scale = a == 0.0f ? 1.0f : __fdiv_rn(a, 448.0f);
}

template <int NV, bool kFp16>
__global__ void __launch_bounds__(kRowThreads) rmsnorm_grad_kernel(const NormGradArgs a) {
    __shared__ float2 buffer[2][kRowThreads / 32];
    pdl_wait();
    RowReduce reduce{buffer};
    const int vectors = a.cols >> 3, t = threadIdx.x, step = blockDim.x;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    uint4 w[NV];
    float dw[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        w[i] = make_uint4(0, 0, 0, 0);
        if (a.weight != nullptr && t + i * step < vectors)
            w[i] = __ldg(reinterpret_cast<const uint4*>(a.weight) + t + i * step);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
    }
    uint4 x[NV], d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = d[i] = make_uint4(0, 0, 0, 0);
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (t + i * step >= vectors) continue;
            x[i] = load_once(a.x + row * a.x_stride + 8 * (t + i * step));
            d[i] = load_once(a.dy + row * a.dy_stride + 8 * (t + i * step));
        }
    };
    int64_t row = blockIdx.x;
    if (row < a.rows) fetch(row);
    for (; row < a.rows; row += gridDim.x) {
        float v[NV][8], dy[NV][8];
        float squares = 0.0f, dot = 0.0f;
        // g = dy w, formed where it is needed: registers
        auto g_of = [&](int i, float (&g)[8]) {
            if (a.weight != nullptr) unpack8<kFp16>(w[i], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = a.weight != nullptr ? g[e] * dy[i][e] : dy[i][e];
        };
        auto sums = [&]() {
            squares = dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float g[8];
                g_of(i, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    squares = fmaf(v[i][e], v[i][e], squares);
                    dot = fmaf(g[e], v[i][e], dot);
                }
            }
            const float2 both = reduce.sum2(squares, dot);
            squares = both.x;
            dot = both.y;
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack8<kFp16>(x[i], v[i]);
            unpack8<kFp16>(d[i], dy[i]);
        }
        uint4 add[NV];
        if (a.dsum != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (t + i * step < vectors) add[i] = load_once(a.dsum + row * a.dsum_stride + 8 * (t + i * step));
        }
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
        sums();
        float eps = a.eps, down = 1.0f;
        if (!(squares <= 3.0e38f)) {   // the whole block
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] *= kDown;
            sums();
            eps = eps * kDown * kDown;
            down = kDown;
        }
        const float inv = rsqrtf(fmaf(squares, inv_cols, eps));
        const float share = dot * inv * inv_cols;   // mean(g u)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (t + i * step >= vectors) continue;
            float g[8], out[8];
            g_of(i, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float u = v[i][e] * inv;
                dw[i][e] = fmaf(dy[i][e], u, dw[i][e]);
                out[e] = fmaf(-u, share, g[e]) * inv * down;
            }
            if (a.dsum != nullptr) {
                float extra[8];
                unpack8<kFp16>(add[i], extra);
#pragma unroll
                for (int e = 0; e < 8; ++e) out[e] += extra[e];
            }
            *reinterpret_cast<uint4*>(a.dx + row * a.dx_stride + 8 * (t + i * step)) = pack8<kFp16>(out);
        }
    }
    if (a.partials != nullptr) {
        float* part = a.partials + static_cast<int64_t>(blockIdx.x) * a.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (t + i * step >= vectors) continue;
            float4* dst = reinterpret_cast<float4*>(part + 8 * (t + i * step));
            dst[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            dst[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

// Eight warps take an eighth of the parts each, 32 columns a block.
__global__ void __launch_bounds__(256) join_columns_kernel(const float* __restrict__ partials, int parts, int cols,
                                                           float* __restrict__ out) {
    __shared__ float run[8][32];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const int p0 = static_cast<int>(static_cast<int64_t>(parts) * warp / 8);
    const int p1 = static_cast<int>(static_cast<int64_t>(parts) * (warp + 1) / 8);
    float sum = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int p = p0; p < p1; ++p) sum += partials[static_cast<int64_t>(p) * cols + c];
    }
    run[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < cols) {
        for (int i = 1; i < 8; ++i) sum += run[i][lane];
        out[c] = sum;
    }
}

// Vectors a thread: 2, fewer for narrow rows, more for wide ones.
int vectors_each(int vectors) {
    for (int each = 2; each < kRowVectors; each *= 2)
        if (row_threads(vectors, each) <= kRowThreads) return each;
    return kRowVectors;
}

template <int NV, bool kFp16>
cudaError_t run_norm(const NormArgs& a, int out, int sm_count, cudaStream_t s) {
    const int threads = row_threads(a.cols >> 3, NV);
    const int64_t blocks = std::min<int64_t>(a.rows, static_cast<int64_t>(sm_count) * std::max(1, 1024 / threads));
    const dim3 grid(static_cast<unsigned>(blocks)), block(threads);
    if (out == kNormRows) return launch_kernel(rmsnorm_kernel<NV, kFp16, kNormRows>, grid, block, 0, s, a);
    if (out == kNormTensor) return launch_kernel(rmsnorm_kernel<NV, kFp16, kNormTensor>, grid, block, 0, s, a);
    return launch_kernel(rmsnorm_kernel<NV, kFp16, kNormHalf>, grid, block, 0, s, a);
}

template <int NV>
cudaError_t run_norm_type(const NormArgs& a, int out, bool fp16, int sm_count, cudaStream_t s) {
    return fp16 ? run_norm<NV, true>(a, out, sm_count, s) : run_norm<NV, false>(a, out, sm_count, s);
}

int grad_blocks(int64_t rows, int cols, int sm_count) {
    const int threads = row_threads(cols >> 3, vectors_each(cols >> 3));
    return static_cast<int>(std::min<int64_t>(rows, static_cast<int64_t>(sm_count) * std::max(1, 1024 / threads)));
}

template <int NV>
cudaError_t run_grad(const NormGradArgs& a, bool fp16, int blocks, cudaStream_t s) {
    const dim3 grid(blocks), block(row_threads(a.cols >> 3, NV));
    return fp16 ? launch_kernel(rmsnorm_grad_kernel<NV, true>, grid, block, 0, s, a)
                : launch_kernel(rmsnorm_grad_kernel<NV, false>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_join_columns(const float* partials, int parts, int cols, float* out, cudaStream_t s) {
    return launch_kernel(join_columns_kernel, dim3((cols + 31) / 32), dim3(256), 0, s, partials, parts, cols, out);
}

cudaError_t launch_rmsnorm(const NormArgs& a, int out, bool fp16, float* next_scale, int sm_count, cudaStream_t s) {
    if (out == kNormTensor) {
        const cudaError_t e = launch_zero_word(a.amax_bits, s);
        if (e != cudaSuccess) return e;
    }
    if (a.rows > 0) {
        cudaError_t e;
        switch (vectors_each(a.cols >> 3)) {
            case 2: e = run_norm_type<2>(a, out, fp16, sm_count, s); break;
            case 4: e = run_norm_type<4>(a, out, fp16, sm_count, s); break;
            default: e = run_norm_type<8>(a, out, fp16, sm_count, s); break;
        }
        if (e != cudaSuccess) return e;
    }
    if (next_scale == nullptr) return cudaSuccess;
    return launch_kernel(next_scale_kernel, dim3(1), dim3(1), 0, s, reinterpret_cast<const float*>(a.amax_bits),
                         next_scale);
}

int64_t rmsnorm_grad_scratch_bytes(int64_t rows, int cols, int sm_count) {
    return static_cast<int64_t>(grad_blocks(rows, cols, sm_count)) * cols * 4;
}

cudaError_t launch_rmsnorm_grad(const NormGradArgs& a, bool fp16, float* dweight, int sm_count, cudaStream_t s) {
    const int blocks = grad_blocks(a.rows, a.cols, sm_count);
    if (blocks > 0) {
        cudaError_t e;
        switch (vectors_each(a.cols >> 3)) {
            case 2: e = run_grad<2>(a, fp16, blocks, s); break;
            case 4: e = run_grad<4>(a, fp16, blocks, s); break;
            default: e = run_grad<8>(a, fp16, blocks, s); break;
        }
        if (e != cudaSuccess) return e;
    }
    return dweight == nullptr ? cudaSuccess : launch_join_columns(a.partials, blocks, a.cols, dweight, s);
}

}  // namespace dg
