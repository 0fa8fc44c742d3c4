// ct_norm.cu -- the junction between two blocks: norm, gate, residual sum and
// norm, forward and backward.
#include "ct_device.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"

#include <type_traits>

namespace ct {
namespace {

// a(w) = offset + w, or 1 without a weight.  Parameters are of the
// activations' type T or fp32, decided per launch (a uniform branch).
template <typename T, bool VEC>
__device__ __forceinline__ void load_param(const void* p, int f32, float offset,
                                           const dev::Cols<VEC>& c, float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 1.0f;
        return;
    }
    if (f32)
        dev::load_cols<VEC>(static_cast<const float*>(p), c, f);
    else
        dev::load_cols<VEC>(static_cast<const T*>(p), c, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += offset;
}

template <typename T>
__device__ __forceinline__ const void* gate_row(const void* gate, int f32, int64_t row,
                                                int64_t rows_per_gate, int hidden) {
    if (!gate) return nullptr;
    const int64_t at = row / rows_per_gate * hidden;
    return f32 ? static_cast<const void*>(static_cast<const float*>(gate) + at)
               : static_cast<const void*>(static_cast<const T*>(gate) + at);
}

// Eight FP8 codes of y * scale.
template <bool VEC>
__device__ __forceinline__ void store_fp8(uint8_t* row, const dev::Cols<VEC>& c,
                                          const float (&y)[8], float scale, int fmt) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float lo = __fmul_rn(y[2 * j], scale), hi = __fmul_rn(y[2 * j + 1], scale);
        h[j] = fmt == 0 ? dev::cvt_fp8x2<0>(lo, hi) : dev::cvt_fp8x2<1>(lo, hi);
    }
    if constexpr (VEC) {
        if (c.any())
            *reinterpret_cast<uint2*>(row + c.first) =
                make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.has(j)) row[c.at(j)] = static_cast<uint8_t>(h[j >> 1] >> (8 * (j & 1)));
    }
}

// One block per row; the row of u, then of res_out, stays in registers.
template <typename T, typename R, bool VEC, int PER>
__global__ void __launch_bounds__(1024) block_norm_kernel(NormArgs a) {
    __shared__ float slots[2][32];
    __shared__ unsigned amax_bits;
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int tid = threadIdx.x, nt = blockDim.x, H = a.hidden;
    const int64_t row = blockIdx.x, at = row * H;
    if (tid == 0) amax_bits = 0;
    float v[PER][8];
    float rstd = 1.0f;
    if (a.u) {
        float sum = 0.0f;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            dev::load_cols<VEC>(static_cast<const T*>(a.u) + at, dev::Cols<VEC>(p * nt + tid, nt, H),
                                v[p]);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(v[p][j], v[p][j], sum);
        }
        if (a.post) {
            sum = dev::block_sum(sum, slots[0]);
            rstd = rsqrtf(sum / H + a.eps);
            if (tid == 0 && a.rstd_post) a.rstd_post[row] = rstd;
        }
    }
    const void* gate = gate_row<T>(a.gate, a.param_f32, row, a.rows_per_gate, H);
    float sum = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const dev::Cols<VEC> c(p * nt + tid, nt, H);
        float r[8];
        dev::load_cols<VEC>(static_cast<const R*>(a.res) + at, c, r);
        if (a.u) {
            float w[8], g[8];
            if (a.post)
                load_param<T>(a.w_post, a.param_f32, a.weight_offset, c, w);
            else
                load_param<T>(nullptr, 0, 0.0f, c, w);
            load_param<T>(gate, a.param_f32, 0.0f, c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[p][j] = a.residual_scale * r[j] + a.branch_scale * g[j] * (v[p][j] * rstd * w[j]);
            dev::store_cols<VEC>(static_cast<R*>(a.res_out) + at, c, v[p]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[p][j] = r[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.has(j)) sum = fmaf(v[p][j], v[p][j], sum);
    }
    if (!a.pre) return;
    sum = dev::block_sum(sum, slots[1]);
    rstd = rsqrtf(sum / H + a.eps);
    if (tid == 0 && a.rstd_pre) a.rstd_pre[row] = rstd;
    const float scale = a.scale ? *a.scale : 0.0f;
    unsigned most = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const dev::Cols<VEC> c(p * nt + tid, nt, H);
        float w[8];
        load_param<T>(a.w_pre, a.param_f32, a.weight_offset, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[p][j] *= rstd * w[j];
            if (c.has(j)) most = max(most, __float_as_uint(v[p][j]) & 0x7FFFFFFFu);
        }
        if (a.scale)
            store_fp8<VEC>(static_cast<uint8_t*>(a.y) + at, c, v[p], scale, a.fmt);
        else
            dev::store_cols<VEC>(static_cast<T*>(a.y) + at, c, v[p]);
    }
    if (!a.scale) return;
    __syncthreads();
    atomicMax(&amax_bits, most);
    __syncthreads();
    if (tid == 0) {
        atomicMax(reinterpret_cast<unsigned*>(a.amax), amax_bits);
        if (row == 0) *a.scale_inv = __fdiv_rn(1.0f, scale);
    }
}

// Backward, per row: du and dres.  The workspace keeps each row's
// mean(G xh) for the column sums.
template <typename T, typename R, bool VEC, int PER>
__global__ void __launch_bounds__(1024) block_norm_backward_kernel(NormBackwardArgs a) {
    __shared__ float slots[2][32];
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int tid = threadIdx.x, nt = blockDim.x, H = a.hidden;
    const int64_t row = blockIdx.x, at = row * H;
    float d[PER][8], back[PER][8], hat[PER][8];
    float rstd = 0.0f, mean = 0.0f;
    if (a.pre) {
        rstd = a.rstd_pre[row];
        float sum = 0.0f;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const dev::Cols<VEC> c(p * nt + tid, nt, H);
            float w[8];
            dev::load_cols<VEC>(static_cast<const T*>(a.dy) + at, c, back[p]);
            dev::load_cols<VEC>(static_cast<const R*>(a.res_out) + at, c, hat[p]);
            load_param<T>(a.w_pre, a.param_f32, a.weight_offset, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                back[p][j] *= w[j];
                hat[p][j] *= rstd;
                sum = fmaf(back[p][j], hat[p][j], sum);
            }
        }
        mean = dev::block_sum(sum, slots[0]) / H;
        if (tid == 0) a.workspace[row] = mean;
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const dev::Cols<VEC> c(p * nt + tid, nt, H);
        if (a.dres_out) {
            dev::load_cols<VEC>(static_cast<const R*>(a.dres_out) + at, c, d[p]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[p][j] = 0.0f;
        }
        if (a.pre) {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[p][j] += rstd * (back[p][j] - hat[p][j] * mean);
        }
        float dr[8];
        const float beta = a.u ? a.residual_scale : 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) dr[j] = beta * d[p][j];
        dev::store_cols<VEC>(static_cast<R*>(a.dres) + at, c, dr);
    }
    if (!a.u) return;
    const void* gate = gate_row<T>(a.gate, a.param_f32, row, a.rows_per_gate, H);
    rstd = a.post ? a.rstd_post[row] : 1.0f;
    float sum = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const dev::Cols<VEC> c(p * nt + tid, nt, H);
        float w[8], g[8];
        load_param<T>(gate, a.param_f32, 0.0f, c, g);
        load_param<T>(a.post ? a.w_post : nullptr, a.param_f32, a.weight_offset, c, w);
        if (a.post) {
            dev::load_cols<VEC>(static_cast<const T*>(a.u) + at, c, hat[p]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) hat[p][j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            back[p][j] = a.branch_scale * g[j] * d[p][j] * w[j];
            hat[p][j] *= rstd;
            sum = fmaf(back[p][j], hat[p][j], sum);
        }
    }
    mean = a.post ? dev::block_sum(sum, slots[1]) / H : 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const dev::Cols<VEC> c(p * nt + tid, nt, H);
#pragma unroll
        for (int j = 0; j < 8; ++j) back[p][j] = rstd * (back[p][j] - hat[p][j] * mean);
        dev::store_cols<VEC>(static_cast<T*>(a.du) + at, c, back[p]);
    }
}

template <typename T>
__device__ __forceinline__ float param(const void* p, int f32, int64_t i) {
    return f32 ? static_cast<const float*>(p)[i] : dev::to_f32(static_cast<const T*>(p)[i]);
}
template <typename T>
__device__ __forceinline__ void set_param(void* p, int f32, int64_t i, float v) {
    if (f32)
        static_cast<float*>(p)[i] = v;
    else
        dev::from_f32(static_cast<T*>(p)[i], v);
}

// Column sums: one thread per column walks down the rows.
template <typename T, typename R>
__global__ void block_norm_columns_kernel(NormBackwardArgs a) {
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int col = blockIdx.x * blockDim.x + threadIdx.x, H = a.hidden;
    if (col >= H) return;
    const float a_pre = a.pre && a.w_pre ? param<T>(a.w_pre, a.param_f32, col) + a.weight_offset : 1.0f;
    const float a_post = a.post && a.w_post ? param<T>(a.w_post, a.param_f32, col) + a.weight_offset : 1.0f;
    float dw_pre = 0.0f, dw_post = 0.0f, dgate = 0.0f;
    for (int64_t row = 0; row < a.rows; ++row) {
        const int64_t i = row * H + col;
        float d = a.dres_out ? dev::to_f32(static_cast<const R*>(a.dres_out)[i]) : 0.0f;
        if (a.pre) {
            const float rstd = a.rstd_pre[row];
            const float dy = dev::to_f32(static_cast<const T*>(a.dy)[i]);
            const float hat = dev::to_f32(static_cast<const R*>(a.res_out)[i]) * rstd;
            dw_pre += dy * hat;
            d += rstd * (dy * a_pre - hat * a.workspace[row]);
        }
        if (!a.u) continue;
        const float hat = dev::to_f32(static_cast<const T*>(a.u)[i]) * (a.post ? a.rstd_post[row] : 1.0f);
        const int64_t group = a.gate ? row / a.rows_per_gate : 0;
        const float g = a.gate ? param<T>(a.gate, a.param_f32, group * H + col) : 1.0f;
        d *= a.branch_scale;
        dw_post += g * d * hat;
        dgate += d * hat * a_post;
        if (a.dgate && (row + 1 == a.rows || (row + 1) % a.rows_per_gate == 0)) {
            set_param<T>(a.dgate, a.param_f32, group * H + col, dgate);
            dgate = 0.0f;
        }
    }
    if (a.dw_pre) set_param<T>(a.dw_pre, a.param_f32, col, dw_pre);
    if (a.dw_post) set_param<T>(a.dw_post, a.param_f32, col, dw_post);
}

// T, R, vectors and columns per thread of a launch.
template <typename F>
cudaError_t by_types(int dtype, int res_dtype, F&& f) {
    if (dtype == 0)
        return res_dtype == 0 ? f(__nv_bfloat16{}, __nv_bfloat16{}) : f(__nv_bfloat16{}, float{});
    if (dtype == 1) return res_dtype == 1 ? f(__half{}, __half{}) : f(__half{}, float{});
    return f(float{}, float{});
}

template <typename... P>
bool all_aligned(P... p) {
    return ((reinterpret_cast<uintptr_t>(p) % 16 == 0) && ...);
}

template <typename F>
cudaError_t by_columns(int hidden, F&& f) {
    const int vectors = (hidden + 7) / 8;
    auto threads = [&](int per) { return ((vectors + per - 1) / per + 31) / 32 * 32; };
    if (vectors <= 1024) return f(std::integral_constant<int, 1>{}, threads(1));
    if (vectors <= 2048) return f(std::integral_constant<int, 2>{}, threads(2));
    return f(std::integral_constant<int, 4>{}, threads(4));
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, int dtype, int res_dtype, cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 && all_aligned(a.u, a.res, a.w_post, a.w_pre, a.gate,
                                                      a.res_out, a.y);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        return by_columns(a.hidden, [&](auto per, int threads) {
            constexpr int PER = decltype(per)::value;
            auto* kernel = vec ? block_norm_kernel<T, R, true, PER>
                               : block_norm_kernel<T, R, false, PER>;
            return launch_pdl(kernel, dim3(static_cast<unsigned>(a.rows)), dim3(threads), 0, stream,
                              a);
        });
    });
}

size_t norm_backward_workspace(int64_t rows, int64_t) {
    return (static_cast<size_t>(rows) * sizeof(float) + 15) / 16 * 16;
}

cudaError_t launch_block_norm_backward(const NormBackwardArgs& a, int dtype, int res_dtype,
                                       cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 &&
                     all_aligned(a.dy, a.dres_out, a.u, a.res_out, a.w_post, a.w_pre, a.gate, a.du,
                                 a.dres);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        if (a.rows > 0) {
            const cudaError_t e = by_columns(a.hidden, [&](auto per, int threads) {
                constexpr int PER = decltype(per)::value;
                auto* kernel = vec ? block_norm_backward_kernel<T, R, true, PER>
                                   : block_norm_backward_kernel<T, R, false, PER>;
                return launch_pdl(kernel, dim3(static_cast<unsigned>(a.rows)), dim3(threads), 0,
                                  stream, a);
            });
            if (e != cudaSuccess) return e;
        }
        if (!a.dw_pre && !a.dw_post && !a.dgate) return cudaSuccess;
        return launch_pdl(block_norm_columns_kernel<T, R>, dim3((a.hidden + 127) / 128), dim3(128), 0,
                          stream, a);
    });
}

}  // namespace ct
