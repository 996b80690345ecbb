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
// block keeps a row in registers until the maxima of the row are known.
// Backward needs nothing of a row but its scales: a thread owns eight columns
// of every so-many-th row, so that dbias is summed in registers; the blocks'
// sums are joined in order by a second kernel.  The blocks of a column take
// the rows in turn, so that the grid moves through memory as one band (each
// on a run of rows of its own: 5 % more time).
// Gated, 8192 x 11008 BF16: codes and checkpoint 103.2 us, 0.90 of the rate of
// a copy; gradient from the checkpoint 119.4 us, 0.89 (122.5 with dbias), from
// the input 134.0 us, 0.99 (142.2).
#include <cuda_runtime.h>

#include <algorithm>

#include "activation.cuh"
#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "row_common.cuh"

namespace dg {
namespace {

// Threads of a block, and blocks an SM at least, by vectors (of each half) a
// thread: the registers (64, 80, 128) hold a row's packed input and FP32 output,
// but for gated rows of more than 12288 columns: eight vectors of both halves
// and their output are all of 128 registers, and 308 bytes a thread are spilled
// (4096 x 14336 to codes 53.9 us, 0.80, with checkpoint 74.7, 0.81; 2048 x 28672
// 57.5 and 84.8, 0.75 and 0.71).
template <int NV>
constexpr int block_limit() { return NV == 4 ? 384 : 512; }
template <int NV>
constexpr int block_min() { return NV == 8 ? 1 : 2; }
// Codes wait for a row's maximum: smaller blocks, and more of them to an SM,
// keep it busy meanwhile (4000 x 8192 BF16 ungated to codes 23.6 -> 20.8 us,
// with checkpoint 30.7 -> 26.6; without codes 22.6 -> 23.0).
constexpr int kLimits[3] = {512, 384, 512}, kCodeLimits[3] = {256, 384, 512};
constexpr int kPerSm[3] = {1024, 768, 512};
constexpr bool within_bounds(const int (&limits)[3]) {
    return limits[0] <= block_limit<2>() && limits[1] <= block_limit<4>() && limits[2] <= block_limit<8>();
}
static_assert(hold_widest_row(kLimits) && within_bounds(kLimits), "launch bounds");
static_assert(hold_widest_row(kCodeLimits) && within_bounds(kCodeLimits), "launch bounds");

template <int NV, bool kFp16, bool kGated, bool kNarrow>
__global__ void __launch_bounds__(block_limit<NV>(), block_min<NV>()) activate_kernel(const ActArgs a, int team_size) {
    __shared__ float2 buffer[2][kRowThreads / 32];
    pdl_wait();
    constexpr int kHalves = kGated ? 2 : 1;
    const RowTeam<kNarrow> team(team_size);
    RowReduce<kNarrow> reduce{buffer, team.size};
    const int vectors = a.cols >> 3;
    uint4 x[kHalves][NV];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int i = 0; i < NV; ++i) x[h][i] = make_uint4(0, 0, 0, 0);
    const int64_t step = static_cast<int64_t>(gridDim.x) * team.rows;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * team.rows; first < a.rows; first += step) {
        const int64_t row = first + team.row;
        const int end = row < a.rows ? vectors : 0;   // this thread's vectors lie below
        const uint16_t* x_row = a.x + row * a.x_stride;
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int at = team.at + i * team.size;
                load_if(at < end, x_row + h * a.cols + 8 * at, x[h][i]);
            }
        if (!kNarrow && threadIdx.x == 0 && row + step < a.rows)
            prefetch_row(a.x + (row + step) * a.x_stride, 2 * kHalves * a.cols);
        if (a.x_q != nullptr) {
            float top[2] = {0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    pair f[4];
                    unpack8<kFp16>(x[h][i], f);
                    top[h] = top8(f, top[h]);
                }
            const float2 both = reduce.max2(top[0], top[1]);
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int i = 0; i < NV; ++i) forget(x[h][i]);
            const float scales[2] = {row_scale(both.x), row_scale(both.y)};
            if (team.at == 0 && end != 0) {
#pragma unroll
                for (int h = 0; h < kHalves; ++h) a.x_scale[row * kHalves + h] = scales[h];
            }
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const float by = row_factor(scales[h]);
                uint8_t* q_row = a.x_q + (row * kHalves + h) * a.cols;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int at = team.at + i * team.size;
                    pair f[4];
                    unpack8<kFp16>(x[h][i], f);
                    store_if(at < end, q_row + 8 * at, codes8(f, by));
                }
            }
        }
        if (a.y == nullptr && a.q == nullptr) continue;
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int i = 0; i < NV; ++i) forget(x[h][i]);
        pair y[NV][4];
        with_activation(a.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                unpack8<kFp16>(x[0][i], y[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[i][e] = activation(act.value, y[i][e]);
            }
        });
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (kGated) {
                pair up[4];
                unpack8<kFp16>(x[kHalves - 1][i], up);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[i][e] = pair_mul(y[i][e], up[e]);
            }
            top = top8(y[i], top);   // (zeros past the row; a team without one has its own maximum)
        }
        if (a.y != nullptr) {
            uint16_t* y_row = a.y + row * a.y_stride;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int at = team.at + i * team.size;
                store_if(at < end, y_row + 8 * at, pack8<kFp16>(y[i]));
            }
        }
        if (a.q != nullptr) {
            top = reduce.max1(top);
            const float scale = row_scale(top), by = row_factor(scale);
            if (team.at == 0 && end != 0) a.q_scale[row] = scale;
            uint8_t* q_row = a.q + row * a.cols;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int at = team.at + i * team.size;
                store_if(at < end, q_row + 8 * at, codes8(y[i], by));
            }
        }
    }
}

constexpr int kGradResident = 7;    // blocks an SM (with 8, 64 registers: 1 to 4 % more time; with 6: 4 to 5 %)
constexpr int kGradThreads = 128;
constexpr int kGradAcross = 32;     // threads side by side at most: a warp's 512 bytes of a row

// kJoin: the runs are the blocks of a cluster, which add up the columns' sums
// themselves (ranks of them; dbias in place of partials).
template <bool kFp16, bool kGated, bool kCodes, bool kJoin>
__global__ void __launch_bounds__(kGradThreads, kGradResident) activate_grad_kernel(const ActGradArgs a, int across,
                                                                                    int ranks) {
    __shared__ float4 columns[kGradThreads][4];   // the threads' sums
    pdl_wait();
    constexpr int kHalves = kGated ? 2 : 1;
    // `across` threads (a power of two) side by side, the others on other rows
    const int t = threadIdx.x, down = kGradThreads / across;
    const int run = kJoin ? static_cast<int>(cluster_ctarank()) : blockIdx.y, runs = kJoin ? ranks : gridDim.y;
    const int c = 8 * static_cast<int>((kJoin ? blockIdx.x / ranks : blockIdx.x) * across + (t & (across - 1)));
    const int64_t width = static_cast<int64_t>(kHalves) * a.cols;
    const int64_t step = static_cast<int64_t>(runs) * down;
    pair sums[kHalves][4];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[h][e] = 0;
    if (c < a.cols) {
        // The next row's loads are in flight while a row is worked on.  Codes
        // leave too few bytes in flight: the row after it is on its way to L2
        // (126.0 -> 120.8 us; reading the input itself, 143 -> 160).
        uint4 next_dy = make_uint4(0, 0, 0, 0), next_x[kHalves];
        uint2 next_q[kHalves];
        float next_scale[kHalves];
        auto fetch = [&](int64_t row) {
            next_dy = load_once(a.dy + row * a.dy_stride + c);
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                if constexpr (kCodes) {
                    next_q[h] = load_once8(a.x_q + row * width + static_cast<int64_t>(h) * a.cols + c);
                    next_scale[h] = ld_float(a.x_scale + row * kHalves + h);
                } else {
                    next_x[h] = load_once(a.x + row * a.x_stride + static_cast<int64_t>(h) * a.cols + c);
                }
            }
        };
        int64_t row = static_cast<int64_t>(run) * down + t / across;
        if (row < a.rows) fetch(row);
#pragma unroll 1
        for (; row < a.rows; row += step) {
            pair dy[4], x[kHalves][4];
            unpack8<kFp16>(next_dy, dy);
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                if constexpr (kCodes)
                    decode8(next_q[h], next_scale[h], x[h]);
                else
                    unpack8<kFp16>(next_x[h], x[h]);
            }
            if (row + step < a.rows) fetch(row + step);
            if constexpr (kCodes) {
                const int64_t later = row + 2 * step;
                if (later < a.rows) {
                    prefetch_line(a.dy + later * a.dy_stride + c);
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
                        prefetch_line(a.x_q + later * width + static_cast<int64_t>(h) * a.cols + c);
                }
            }
            pair dx[kHalves][4];
            with_activation(a.act, [&](auto act) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const ValueSlope f = activation_slope(act.value, x[0][e]);
                    if constexpr (kGated) {
                        dx[0][e] = pair_mul(pair_mul(dy[e], x[kHalves - 1][e]), f.slope);
                        dx[kHalves - 1][e] = pair_mul(dy[e], f.value);
                    } else {
                        dx[0][e] = pair_mul(dy[e], f.slope);
                    }
                }
            });
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sums[h][e] = pair_add(sums[h][e], dx[h][e]);
                __stcs(reinterpret_cast<uint4*>(a.dx + row * a.dx_stride + static_cast<int64_t>(h) * a.cols + c),
                       pack8<kFp16>(dx[h]));
            }
        }
    }
    if (!kJoin && a.partials == nullptr) return;
    if (!kJoin) pdl_launch_dependents();   // the join's launch
    float* part = a.partials + (kJoin ? 0 : run * width);
#pragma unroll
    for (int h = 0; h < kHalves; ++h) store_sums(reinterpret_cast<float*>(&columns[t][2 * h]), sums[h]);
    __syncthreads();
    // thread t of the first row adds up what lies below it, in order
    const bool mine = t < across && c < a.cols;
    auto add = [](float4& s, const float4& v) {
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    };
    if (mine) {
#pragma unroll
        for (int i = 0; i < 2 * kHalves; ++i) {
            float4 s = columns[t][i];
            for (int r = 1; r < down; ++r) add(s, columns[t + r * across][i]);
            if (kJoin)
                columns[t][i] = s;
            else
                *reinterpret_cast<float4*>(part + static_cast<int64_t>(i >> 1) * a.cols + c + 4 * (i & 1)) = s;
        }
    }
    if constexpr (kJoin) {
        cluster_sync_all_diverged();
        if (run == 0 && mine) {
#pragma unroll
            for (int i = 0; i < 2 * kHalves; ++i) {
                float4 s = columns[t][i];
                for (int r = 1; r < runs; ++r) {
                    float4 v;
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                                 : "r"(map_to_rank(&columns[t][i], static_cast<uint32_t>(r))));
                    add(s, v);
                }
                *reinterpret_cast<float4*>(part + static_cast<int64_t>(i >> 1) * a.cols + c + 4 * (i & 1)) = s;
            }
        }
        cluster_sync_all_diverged();   // no block leaves while another reads its sums
    }
}

template <int NV, bool kFp16, bool kNarrow>
cudaError_t run_act_rows(const ActArgs& a, const RowPlan& p, cudaStream_t s) {
    const dim3 grid(p.blocks), block(p.threads);
    return a.gated ? launch_kernel(activate_kernel<NV, kFp16, true, kNarrow>, grid, block, 0, s, a, p.team)
                   : launch_kernel(activate_kernel<NV, kFp16, false, kNarrow>, grid, block, 0, s, a, p.team);
}

template <bool kFp16>
cudaError_t run_act(const ActArgs& a, const RowPlan& p, cudaStream_t s) {
    if (p.narrow) return run_act_rows<2, kFp16, true>(a, p, s);
    if (p.each == 2) return run_act_rows<2, kFp16, false>(a, p, s);
    if (p.each == 4) return run_act_rows<4, kFp16, false>(a, p, s);
    return run_act_rows<8, kFp16, false>(a, p, s);
}

// The gradient's blocks: `across` threads side by side and the others below
// them, `columns` blocks of that width, `runs` of them on the rows in turn: as
// many blocks as are resident at once, but no more than have rows, and past
// 256 runs, which the join has to add up, none of fewer than eight rows a
// thread (100000 x 8, gated with dbias: 9.6 us, 11.2 without this; 4096 x 256:
// 6.9, 7.6; 22397 x 64: 8.6, 8.1).
struct ActGradPlan {
    int across, columns, runs, down;
};
ActGradPlan act_grad_plan(int64_t rows, int cols, int sm_count) {
    ActGradPlan p{1, 1, 1, 1};
    const int vectors = cols / 8;
    while (p.across < kGradAcross && p.across < vectors) p.across *= 2;
    p.columns = (vectors + p.across - 1) / p.across;
    p.down = kGradThreads / p.across;
    const int64_t runs = std::max<int64_t>(1, static_cast<int64_t>(sm_count) * kGradResident / p.columns);
    const int64_t few = std::max<int64_t>(256, rows / (8 * p.down));
    p.runs = static_cast<int>(std::min({(rows + p.down - 1) / p.down, runs, few}));
    return p;
}

// dbias of few rows: as many runs as a cluster has blocks, and no second
// kernel, while each thread has one row (11008 gated, 1 row: 4.6 -> 2.2 us, 16
// rows 5.3 -> 4.8) or, where the blocks are no more than the SMs, two: that
// takes 0.3 to 0.5 us more by itself (63 x 2000: 3.3 -> 3.6), but one launch
// less, which is what calls that are not replayed from a graph wait for (6.9
// -> 5.1 us a call).
constexpr int kJoinRanks = 8;
bool join_in_cluster(const ActGradPlan& p, int64_t rows, int sm_count) {
    return rows <= (p.columns * kJoinRanks <= sm_count ? 2 : 1) * kJoinRanks * p.down;
}

template <bool kFp16, bool kGated, bool kCodes>
cudaError_t run_act_grad_from(const ActGradArgs& a, float* dbias, const ActGradPlan& p, int sm_count, cudaStream_t s) {
    const dim3 block(kGradThreads);
    if (dbias != nullptr && join_in_cluster(p, a.rows, sm_count)) {
        int ranks = 1;
        while (ranks < kJoinRanks && ranks * p.down < a.rows) ranks *= 2;
        ActGradArgs b = a;
        b.partials = dbias;
        return launch_clusters(activate_grad_kernel<kFp16, kGated, kCodes, true>, dim3(p.columns * ranks), block, ranks, 0,
                               s, b, p.across, ranks);
    }
    const cudaError_t e = launch_kernel(activate_grad_kernel<kFp16, kGated, kCodes, false>, dim3(p.columns, p.runs), block,
                                        0, s, a, p.across, 1);
    if (e != cudaSuccess || dbias == nullptr) return e;
    return launch_join_columns(a.partials, p.runs, kGated ? 2 * a.cols : a.cols, dbias, s);
}

template <bool kFp16, bool kGated>
cudaError_t run_act_grad(const ActGradArgs& a, float* dbias, const ActGradPlan& p, int sm_count, cudaStream_t s) {
    return a.x_q != nullptr ? run_act_grad_from<kFp16, kGated, true>(a, dbias, p, sm_count, s)
                            : run_act_grad_from<kFp16, kGated, false>(a, dbias, p, sm_count, s);
}

}  // namespace

cudaError_t launch_activate(const ActArgs& a, bool fp16, int sm_count, cudaStream_t s) {
    const bool codes = a.q != nullptr || a.x_q != nullptr;
    const RowPlan p = row_plan(a.rows, a.cols, sm_count, codes ? kCodeLimits : kLimits, kPerSm);
    return fp16 ? run_act<true>(a, p, s) : run_act<false>(a, p, s);
}

int64_t activate_grad_scratch_bytes(int64_t rows, int cols, bool gated, int sm_count) {
    return static_cast<int64_t>(act_grad_plan(rows, cols, sm_count).runs) * cols * (gated ? 8 : 4);
}

cudaError_t launch_activate_grad(const ActGradArgs& a, bool fp16, float* dbias, int sm_count, cudaStream_t s) {
    const ActGradPlan p = act_grad_plan(a.rows, a.cols, sm_count);
    if (a.rows == 0)
        return dbias == nullptr ? cudaSuccess : launch_join_columns(nullptr, 0, a.gated ? 2 * a.cols : a.cols, dbias, s);
    if (fp16) return a.gated ? run_act_grad<true, true>(a, dbias, p, sm_count, s) : run_act_grad<true, false>(a, dbias, p, sm_count, s);
    return a.gated ? run_act_grad<false, true>(a, dbias, p, sm_count, s) : run_act_grad<false, false>(a, dbias, p, sm_count, s);
}

}  // namespace dg
