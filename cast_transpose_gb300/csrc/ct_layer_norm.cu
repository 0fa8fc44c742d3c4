// ct_layer_norm.cu -- the junction between two blocks whose norm is a layer
// norm: the branch's dropout, the residual sum and the norm, forward and
// backward.
#include "ct_device.cuh"
#include "ct_dropout.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"
#include "ct_vec.cuh"

#include <algorithm>

namespace ct {
namespace {

constexpr int kMaxRowThreads = 1024;

// Sums of a and b over the block, the same in every thread, in a fixed order.
__device__ __forceinline__ float2 block_sums(float a, float b, float2 (&slots)[32]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    a = dev::warp_sum(a);
    b = dev::warp_sum(b);
    __syncthreads();                    // of the sums before
    if (lane == 0) slots[warp] = make_float2(a, b);
    __syncthreads();
    const float2 v = lane < warps ? slots[lane] : make_float2(0.0f, 0.0f);
    return make_float2(dev::warp_sum(v.x), dev::warp_sum(v.y));
}

// Forward, a block per row, which its threads hold in registers.
template <typename T, typename R, int G, int PER>
__global__ void __launch_bounds__(kMaxRowThreads) layer_norm_row_kernel(const LayerNormArgs a) {
    __shared__ float2 slots[32];
    __shared__ unsigned block_max;
    const int tid = threadIdx.x, H = a.hidden;
    const int64_t row = blockIdx.x, at = row * H;
    auto cols = [&](int p) { return dev::Cols<G>(p * blockDim.x + tid, H); };
    dev::pdl_launch_dependents();
    if (tid == 0) block_max = 0;
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    float v[PER][8];
    float sum = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        dev::load_cols<G>(static_cast<const R*>(a.res) + at, cols(p), v[p]);
        if (a.u) {
            float u[8];
            dev::load_cols<G>(static_cast<const T*>(a.u) + at, cols(p), u);
            const Drops drops(a.drop);
            if (drops.some) drops.apply(drops.kept<G>(static_cast<uint32_t>(row), p * blockDim.x + tid), u);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[p][j] += u[j];
            dev::store_cols<G>(static_cast<R*>(a.res_out) + at, cols(p), v[p]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += v[p][j];       // 0 past the row's end
    }
    const float mean = block_sums(sum, 0.0f, slots).x / H;
    float squares = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[p][j] -= mean;
            if (cols(p).has(j)) squares = fmaf(v[p][j], v[p][j], squares);
        }
    const float rstd = rsqrtf(block_sums(squares, 0.0f, slots).x / H + a.eps);
    if (tid == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    const float scale = a.scale ? *a.scale : 0.0f;
    unsigned most = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        float w[8], b[8];
        load_param<T>(a.weight, a.param_f32, 0, a.weight_offset, cols(p), w);
        load_bias<T>(a.bias, a.param_f32, 0, cols(p), b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[p][j] = fmaf(v[p][j] * rstd, w[j], b[j]);
            if (cols(p).has(j)) most = max(most, __float_as_uint(v[p][j]) & 0x7FFFFFFFu);
        }
        if (a.scale)
            store_fp8<G>(static_cast<uint8_t*>(a.y) + at, cols(p), v[p], scale, a.fmt);
        else
            dev::store_cols<G>(static_cast<T*>(a.y) + at, cols(p), v[p]);
    }
    if (!a.scale) return;
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if ((tid & 31) == 0) atomicMax(&block_max, most);
    __syncthreads();
    if (tid == 0) {
        if (block_max) atomicMax(reinterpret_cast<unsigned*>(a.amax), block_max);
        if (row == 0) *a.scale_inv = __fdiv_rn(1.0f, scale);
    }
}

// Backward of a row.  With xh = (res_out - mean) rstd and g = dy a(w):
//   dres = dres_out + rstd (g - mean(g) - xh mean(g xh))     du = dropout(dres)
template <typename T, typename R, int G, int PER>
__global__ void __launch_bounds__(kMaxRowThreads) layer_norm_backward_row_kernel(const LayerNormBackwardArgs a) {
    __shared__ float2 slots[32];
    const int tid = threadIdx.x, H = a.hidden;
    const int64_t row = blockIdx.x, at = row * H;
    auto cols = [&](int p) { return dev::Cols<G>(p * blockDim.x + tid, H); };
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float g[PER][8], x[PER][8];
    float sum_g = 0.0f, sum_gx = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        float w[8];
        dev::load_cols<G>(static_cast<const T*>(a.dy) + at, cols(p), g[p]);
        dev::load_cols<G>(static_cast<const R*>(a.res_out) + at, cols(p), x[p]);
        load_param<T>(a.weight, a.param_f32, 0, a.weight_offset, cols(p), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {                      // dy is 0 past the row's end
            x[p][j] = (x[p][j] - mean) * rstd;
            g[p][j] *= w[j];
            sum_g += g[p][j];
            sum_gx = fmaf(g[p][j], x[p][j], sum_gx);
        }
    }
    const float2 sums = block_sums(sum_g, sum_gx, slots);
    const float level = sums.x / H, along = sums.y / H;
    const Drops drops(a.drop);
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        float d[8] = {};
        if (a.dres_out) dev::load_cols<G>(static_cast<const R*>(a.dres_out) + at, cols(p), d);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, g[p][j] - level - x[p][j] * along, d[j]);
        dev::store_cols<G>(static_cast<R*>(a.dres) + at, cols(p), d);
        if (!a.du) continue;
        if (drops.some) drops.apply(drops.kept<G>(static_cast<uint32_t>(row), p * blockDim.x + tid), d);
        dev::store_cols<G>(static_cast<T*>(a.du) + at, cols(p), d);
    }
}

// Column sums dw = sum dy xh and db = sum dy over the rows of a share (blockIdx.y
// of `shares`): 32 columns a block, a warp takes every 32nd row.
constexpr int kColumnWarps = 32;

template <typename T, typename R>
__global__ void __launch_bounds__(32 * kColumnWarps)
    layer_norm_columns_kernel(const LayerNormBackwardArgs a, int shares) {
    __shared__ float parts[2][kColumnWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, H = a.hidden;
    const int col = blockIdx.x * 32 + lane;
    const int64_t share = blockIdx.y, begin = a.rows * share / shares, end = a.rows * (share + 1) / shares;
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    float w = 0.0f, b = 0.0f;
    if (col < H)
        for (int64_t r = begin + warp; r < end; r += kColumnWarps) {
            const float dy = dev::to_f32(static_cast<const T*>(a.dy)[r * H + col]);
            const float x = dev::to_f32(static_cast<const R*>(a.res_out)[r * H + col]);
            w = fmaf(dy, (x - a.mean[r]) * a.rstd[r], w);
            b += dy;
        }
    parts[0][warp][lane] = w;
    parts[1][warp][lane] = b;
    __syncthreads();
    if (warp >= 2 || col >= H) return;
    float sum = 0.0f;
    for (int i = 0; i < kColumnWarps; ++i) sum += parts[warp][i][lane];
    if (shares > 1) {
        a.workspace[(int64_t(warp) * shares + share) * H + col] = sum;
    } else {
        void* out = warp == 0 ? a.dweight : a.dbias;
        if (out) set_param<T>(out, a.param_f32, col, sum);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) layer_norm_join_kernel(const LayerNormBackwardArgs a, int shares) {
    const int col = blockIdx.x * blockDim.x + threadIdx.x, H = a.hidden;
    void* out = blockIdx.y == 0 ? a.dweight : a.dbias;
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if ((a.noop && *a.noop != 0.0f) || !out || col >= H) return;
    float sum = 0.0f;
    for (int i = 0; i < shares; ++i) sum += a.workspace[(int64_t(blockIdx.y) * shares + i) * H + col];
    set_param<T>(out, a.param_f32, col, sum);
}

// Threads of a block that holds a row of `hidden` columns, PER groups of eight each.
int row_threads(int hidden, int per) { return (hidden + 256 * per - 1) / (256 * per) * 32; }
int row_per(int hidden) { return hidden <= 8192 ? 1 : hidden <= 16384 ? 2 : 4; }

int column_shares(int64_t rows, int64_t hidden) {
    const int64_t blocks = (hidden + 31) / 32;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((rows + 127) / 128, 600 / std::max<int64_t>(blocks, 1))));
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, int dtype, int res_dtype, cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 && all_aligned(a.u, a.res, a.weight, a.bias, a.res_out, a.y);
    const int per = row_per(a.hidden);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        auto* kernel = per == 1 ? (vec ? layer_norm_row_kernel<T, R, 8, 1> : layer_norm_row_kernel<T, R, 1, 1>)
                     : per == 2 ? (vec ? layer_norm_row_kernel<T, R, 8, 2> : layer_norm_row_kernel<T, R, 1, 2>)
                                : (vec ? layer_norm_row_kernel<T, R, 8, 4> : layer_norm_row_kernel<T, R, 1, 4>);
        return launch_pdl(kernel, dim3(static_cast<unsigned>(a.rows)), dim3(row_threads(a.hidden, per)), 0,
                          stream, a);
    });
}

size_t layer_norm_backward_workspace(int64_t rows, int64_t hidden) {
    const int shares = column_shares(rows, hidden);
    return shares > 1 ? size_t(shares) * 2 * hidden * sizeof(float) : 0;
}

cudaError_t launch_layer_norm_backward(const LayerNormBackwardArgs& a, int dtype, int res_dtype,
                                       cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 &&
                     all_aligned(a.dy, a.dres_out, a.res_out, a.weight, a.dres, a.du);
    const int per = row_per(a.hidden);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        auto* kernel = per == 1 ? (vec ? layer_norm_backward_row_kernel<T, R, 8, 1> : layer_norm_backward_row_kernel<T, R, 1, 1>)
                     : per == 2 ? (vec ? layer_norm_backward_row_kernel<T, R, 8, 2> : layer_norm_backward_row_kernel<T, R, 1, 2>)
                                : (vec ? layer_norm_backward_row_kernel<T, R, 8, 4> : layer_norm_backward_row_kernel<T, R, 1, 4>);
        cudaError_t e = cudaSuccess;
        if (a.rows > 0)
            e = launch_pdl(kernel, dim3(static_cast<unsigned>(a.rows)), dim3(row_threads(a.hidden, per)), 0, stream, a);
        if (e != cudaSuccess || (!a.dweight && !a.dbias)) return e;
        const int shares = column_shares(a.rows, a.hidden);
        e = launch_pdl(layer_norm_columns_kernel<T, R>, dim3((a.hidden + 31) / 32, shares), dim3(32 * kColumnWarps), 0,
                       stream, a, shares);
        if (e != cudaSuccess || shares == 1) return e;
        return launch_pdl(layer_norm_join_kernel<T>, dim3((a.hidden + 255) / 256, 2), dim3(256), 0, stream, a, shares);
    });
}

}  // namespace ct
