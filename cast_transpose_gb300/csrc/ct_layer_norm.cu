// ct_layer_norm.cu -- the junction between two blocks whose norm is a layer
// norm: the branch's dropout, the residual sum and the norm, forward and
// backward.
#include "ct_device.cuh"
#include "ct_dropout.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"
#include "ct_vec.cuh"

#include <algorithm>
#include <atomic>

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
            if (drops.some) drops.apply<G>(static_cast<uint32_t>(row), p * blockDim.x + tid, u);
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
        if (drops.some) drops.apply<G>(static_cast<uint32_t>(row), p * blockDim.x + tid, d);
        dev::store_cols<G>(static_cast<T*>(a.du) + at, cols(p), d);
    }
}

// ---- many rows -----------------------------------------------------------------
// A block takes every gridDim.x-th row, a thread two groups of eight columns.
// Rows arrive in a ring of shared-memory stages by asynchronous copies that are
// issued stages ahead.  With G = 8 a thread copies what it will read itself, so
// that no barrier is needed for it; with G = 1 a row is copied as the aligned
// 16-byte blocks that cover it.
constexpr int kRingPer = 2;                     // groups of eight columns per thread
constexpr int kRingThreads = 768;               // at most, with 80 registers each
constexpr int kRingStages = 4;                  // at most
constexpr int kRingSmem = 226 * 1024;           // of an SM's blocks together

__host__ __device__ constexpr uint32_t align16(uint32_t v) { return (v + 15) & ~15u; }
// Bytes of a tensor's row in a stage.
template <int G>
__host__ __device__ constexpr uint32_t slot_bytes(int threads, int hidden, int size) {
    return G == 8 ? uint32_t(threads) * kRingPer * 8 * size : align16(uint32_t(hidden) * size) + 32;
}

template <typename T, int G>
struct Staged {
    const T* base;          // the tensor, null: left out
    int64_t rows;
    int H;

    __device__ __forceinline__ void fetch(uint8_t* stage, int64_t row) const {
        if (!base) return;
        const int tid = threadIdx.x, n = blockDim.x;
        if constexpr (G == 8) {
#pragma unroll
            for (int p = 0; p < kRingPer; ++p) {
                const dev::Cols<8> c(p * n + tid, H);
                const uint8_t* from = reinterpret_cast<const uint8_t*>(base + row * H + (c.any() ? c.first : 0));
#pragma unroll
                for (int w = 0; w < int(sizeof(T) / 2); ++w)
                    dev::cp_async16(stage + ((p * int(sizeof(T) / 2) + w) * n + tid) * 16, from + 16 * w, 16);
            }
        } else {
            const uintptr_t from = reinterpret_cast<uintptr_t>(base + row * H), first = from & ~uintptr_t(15);
            const uintptr_t begin = reinterpret_cast<uintptr_t>(base), end = begin + rows * H * sizeof(T);
            const int blocks = static_cast<int>((from - first + H * sizeof(T) + 15) / 16);
            for (int i = tid; i < blocks; i += n) {
                const uintptr_t at = first + 16 * uintptr_t(i);
                if (at >= begin) {
                    dev::cp_async16(stage + 16 * i, reinterpret_cast<const void*>(at),
                                    static_cast<int>(min(uintptr_t(16), end - at)));
                } else {        // the tensor begins inside these 16 bytes
                    T* to = reinterpret_cast<T*>(stage + (begin - at));
                    for (int j = 0; j < int((at + 16 - begin) / sizeof(T)) && j < rows * H; ++j) to[j] = base[j];
                }
            }
        }
    }
    // The thread's group p of the row in a stage.
    __device__ __forceinline__ V8 get(const uint8_t* stage, int64_t row, int p) const {
        const int tid = threadIdx.x, n = blockDim.x;
        float f[8];
        if constexpr (G == 8) {
            dev::Raw8<T> r;
#pragma unroll
            for (int w = 0; w < int(sizeof(T) / 2); ++w)
                r.v[w] = *reinterpret_cast<const uint4*>(stage + ((p * int(sizeof(T) / 2) + w) * n + tid) * 16);
            dev::unpack8(r, f);
        } else {
            const dev::Cols<1> c(p * n + tid, H);
            const T* at = reinterpret_cast<const T*>(stage + (reinterpret_cast<uintptr_t>(base + row * H) & 15));
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = dev::to_f32(at[c.has(j) ? c.at(j) : 0]);
        }
        return pairs(f);
    }
};

// Columns of the thread's group that lie past the row's end are 0 from here on,
// where there may be some beside others; a group that is past it as a whole adds
// nothing by on().
template <int G>
__device__ __forceinline__ void cut(const dev::Cols<G>& c, V8& v) {
    if constexpr (G == 8) return;
    float f[8];
    floats(v, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = c.has(j) ? f[j] : 0.0f;
    v = pairs(f);
}

template <int G>
__device__ __forceinline__ void drop(const Drops& drops, int64_t row, int item, V8& v) {
    float f[8];
    floats(v, f);
    drops.apply<G>(static_cast<uint32_t>(row), item, f);
    v = pairs(f);
}
// s / n, rounded to nearest but for rare last bits, given r = 1 / n.
__device__ __forceinline__ float divided(float s, float n, float r) {
    const float q = s * r;
    return fmaf(fmaf(-q, n, s), r, q);
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Waits for the thread's copies but those of the last `ahead` stages.
__device__ __forceinline__ void wait_stages(int ahead) {
    if (ahead == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (ahead == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
}
__device__ __forceinline__ void commit_stage() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Forward.  The mean and the squares about it need one exchange: a warp leaves the
// sum of its columns and the squares about its own mean, from which everyone gets
//   M2 = sum over warps of M2_w + n_w (mean_w - mean)^2
// without the cancellation of a difference of squares.
template <typename T, typename R, int G>
__global__ void __launch_bounds__(kRingThreads, 1) layer_norm_kernel(const LayerNormArgs a, int stages) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 slots[2][32];
    __shared__ unsigned block_max;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, H = a.hidden;
    auto cols = [&](int p) { return dev::Cols<G>(p * blockDim.x + tid, H); };
    if (tid == 0) block_max = 0;
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const Staged<R, G> res{static_cast<const R*>(a.res), a.rows, H};
    const Staged<T, G> u{static_cast<const T*>(a.u), a.rows, H};
    const uint32_t second = slot_bytes<G>(blockDim.x, H, sizeof(R));
    const uint32_t stage_bytes = second + (a.u ? slot_bytes<G>(blockDim.x, H, sizeof(T)) : 0);
    auto fetch = [&](int64_t row, int to) {
        if (row < a.rows) {
            res.fetch(smem + to * stage_bytes, row);
            u.fetch(smem + to * stage_bytes + second, row);
        }
        commit_stage();
    };
    for (int i = 0; i + 1 < stages; ++i) fetch(blockIdx.x + int64_t(i) * gridDim.x, i);
    const Drops drops(a.drop);
    const float scale = a.scale ? *a.scale : 0.0f;
    V8 w[kRingPer], b[kRingPer];
#pragma unroll
    for (int p = 0; p < kRingPer; ++p) {
        float f[8];
        load_param<T>(a.weight, a.param_f32, 0, a.weight_offset, cols(p), f);
        w[p] = pairs(f);
        load_bias<T>(a.bias, a.param_f32, 0, cols(p), f);
        b[p] = pairs(f);
    }
    // columns of warp `of`, as many as its groups have inside the row
    auto columns_of = [&](int of) {
        int n = 0;
#pragma unroll
        for (int p = 0; p < kRingPer; ++p) n += max(0, min(256, H - 256 * (p * warps + of)));
        return static_cast<float>(n);
    };
    const float own_columns = columns_of(warp), lane_columns = lane < warps ? columns_of(lane) : 1.0f;
    const float per_own = 1.0f / own_columns, per_lane = 1.0f / lane_columns, per_column = 1.0f / H;
    unsigned most = 0;
    int stage = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t at = row * H;
        wait_stages(stages - 2);
        if (G != 8) __syncthreads();
        const uint8_t* here = smem + stage * stage_bytes;
        V8 v[kRingPer];
        float sum_w = 0.0f, squares_w = 0.0f;
        if (a.u) {
            V8 x[kRingPer];
#pragma unroll
            for (int p = 0; p < kRingPer; ++p) x[p] = u.get(here + second, row, p);
            if (drops.some) {
#pragma unroll
                for (int p = 0; p < kRingPer; ++p) drop<G>(drops, row, p * blockDim.x + tid, x[p]);
            }
#pragma unroll
            for (int p = 0; p < kRingPer; ++p) {
                v[p] = res.get(here, row, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[p].p[j] = add2(v[p].p[j], x[p].p[j]);
                store_v8<G>(static_cast<R*>(a.res_out) + at, cols(p), v[p]);
            }
        } else {
#pragma unroll
            for (int p = 0; p < kRingPer; ++p) v[p] = res.get(here, row, p);
        }
#pragma unroll
        for (int p = 0; p < kRingPer; ++p) {
            cut<G>(cols(p), v[p]);
            const float part = lanes_sum(add2(add2(v[p].p[0], v[p].p[1]), add2(v[p].p[2], v[p].p[3])));
            sum_w += on(cols(p)) ? part : 0.0f;
        }
        // the stage before this one is free
        fetch(row + int64_t(stages - 1) * gridDim.x, stage == 0 ? stages - 1 : stage - 1);
        if (++stage == stages) stage = 0;
        sum_w = dev::warp_sum(sum_w);
        const float mean_w = divided(sum_w, own_columns, per_own);
        const uint64_t away = pair(-mean_w, -mean_w);
#pragma unroll
        for (int p = 0; p < kRingPer; ++p) {
            V8 d;
            uint64_t part = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) d.p[j] = add2(v[p].p[j], away);
            cut<G>(cols(p), d);
#pragma unroll
            for (int j = 0; j < 4; ++j) part = fma2(d.p[j], d.p[j], part);
            squares_w += on(cols(p)) ? lanes_sum(part) : 0.0f;
        }
        squares_w = dev::warp_sum(squares_w);
        if (lane == 0) slots[turn][warp] = make_float2(sum_w, squares_w);
        __syncthreads();
        const float2 other = lane < warps ? slots[turn][lane] : make_float2(0.0f, 0.0f);
        turn ^= 1;
        const float mean = dev::warp_sum(other.x) / H;
        const float apart = lane < warps ? divided(other.x, lane_columns, per_lane) - mean : 0.0f;
        const float squares = dev::warp_sum(fmaf(lane_columns * apart, apart, other.y));
        const float rstd = rsqrtf(fmaf(squares, per_column, a.eps));
        if (tid == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        const uint64_t mean2 = pair(-mean, -mean), rstd2 = pair(rstd, rstd);
#pragma unroll
        for (int p = 0; p < kRingPer; ++p) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[p].p[j] = fma2(mul2(add2(v[p].p[j], mean2), rstd2), w[p].p[j], b[p].p[j]);
            if (!a.scale) {
                store_v8<G>(static_cast<T*>(a.y) + at, cols(p), v[p]);
                continue;
            }
            float f[8];
            floats(v[p], f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (cols(p).has(j)) most = max(most, __float_as_uint(f[j]) & 0x7FFFFFFFu);
            store_fp8<G>(static_cast<uint8_t*>(a.y) + at, cols(p), f, scale, a.fmt);
        }
    }
    dev::pdl_launch_dependents();
    if (!a.scale) return;
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) atomicMax(&block_max, most);
    __syncthreads();
    if (tid == 0) {
        if (block_max) atomicMax(reinterpret_cast<unsigned*>(a.amax), block_max);
        if (blockIdx.x == 0) *a.scale_inv = __fdiv_rn(1.0f, scale);
    }
}

// Backward.  The two sums of a row are exchanged together; the column sums dw = sum
// dy xh and db = sum dy of the block's rows stay in registers, dy and res_out are
// read from the stage a second time instead.
template <typename T, typename R, int G>
__global__ void __launch_bounds__(kRingThreads, 1)
    layer_norm_backward_kernel(const LayerNormBackwardArgs a, int stages) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 slots[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, H = a.hidden;
    auto cols = [&](int p) { return dev::Cols<G>(p * blockDim.x + tid, H); };
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const Staged<R, G> res{static_cast<const R*>(a.res_out), a.rows, H};
    const Staged<R, G> down{static_cast<const R*>(a.dres_out), a.rows, H};
    const Staged<T, G> dy{static_cast<const T*>(a.dy), a.rows, H};
    const uint32_t second = slot_bytes<G>(blockDim.x, H, sizeof(R));
    const uint32_t third = second + slot_bytes<G>(blockDim.x, H, sizeof(T));
    const uint32_t stage_bytes = third + (a.dres_out ? second : 0);
    auto fetch = [&](int64_t row, int to) {
        if (row < a.rows) {
            res.fetch(smem + to * stage_bytes, row);
            dy.fetch(smem + to * stage_bytes + second, row);
            down.fetch(smem + to * stage_bytes + third, row);
        }
        commit_stage();
    };
    for (int i = 0; i + 1 < stages; ++i) fetch(blockIdx.x + int64_t(i) * gridDim.x, i);
    const Drops drops(a.drop);
    V8 w[kRingPer], dw[kRingPer] = {}, db[kRingPer] = {};
#pragma unroll
    for (int p = 0; p < kRingPer; ++p) {
        float f[8];
        load_param<T>(a.weight, a.param_f32, 0, a.weight_offset, cols(p), f);
        w[p] = pairs(f);
    }
    const float per_column = 1.0f / H;
    float mean = 0.0f, rstd = 0.0f;
    if (blockIdx.x < a.rows) {
        mean = a.mean[blockIdx.x];
        rstd = a.rstd[blockIdx.x];
    }
    int stage = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t at = row * H;
        const int64_t next = min(row + gridDim.x, a.rows - 1);
        const float next_mean = a.mean[next], next_rstd = a.rstd[next];
        wait_stages(stages - 2);
        if (G != 8) __syncthreads();
        const uint8_t* here = smem + stage * stage_bytes;
        fetch(row + int64_t(stages - 1) * gridDim.x, stage == 0 ? stages - 1 : stage - 1);
        if (++stage == stages) stage = 0;
        const uint64_t mean2 = pair(-mean, -mean), rstd2 = pair(rstd, rstd);
        float one = 0.0f, two = 0.0f;
#pragma unroll
        for (int p = 0; p < kRingPer; ++p) {
            const V8 x = res.get(here, row, p);
            V8 g = dy.get(here + second, row, p);
            uint64_t sum_g = 0, sum_gx = 0;
            cut<G>(cols(p), g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t hat = mul2(add2(x.p[j], mean2), rstd2), gw = mul2(g.p[j], w[p].p[j]);
                dw[p].p[j] = fma2(g.p[j], hat, dw[p].p[j]);
                db[p].p[j] = add2(db[p].p[j], g.p[j]);
                sum_g = add2(sum_g, gw);
                sum_gx = fma2(gw, hat, sum_gx);
            }
            one += on(cols(p)) ? lanes_sum(sum_g) : 0.0f;
            two += on(cols(p)) ? lanes_sum(sum_gx) : 0.0f;
        }
        one = dev::warp_sum(one);
        two = dev::warp_sum(two);
        if (lane == 0) slots[turn][warp] = make_float2(one, two);
        __syncthreads();
        const float2 other = lane < warps ? slots[turn][lane] : make_float2(0.0f, 0.0f);
        turn ^= 1;
        const float level = -dev::warp_sum(other.x) * per_column, along = -dev::warp_sum(other.y) * per_column;
        const uint64_t level2 = pair(level, level), along2 = pair(along, along);
#pragma unroll
        for (int p = 0; p < kRingPer; ++p) {
            const V8 x = res.get(here, row, p), g = dy.get(here + second, row, p);
            V8 d = {};
            if (a.dres_out) d = down.get(here + third, row, p);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t hat = mul2(add2(x.p[j], mean2), rstd2);
                d.p[j] = fma2(rstd2, fma2(hat, along2, fma2(g.p[j], w[p].p[j], level2)), d.p[j]);
            }
            store_v8<G>(static_cast<R*>(a.dres) + at, cols(p), d);
            if (!a.du) continue;
            if (drops.some) drop<G>(drops, row, p * blockDim.x + tid, d);
            store_v8<G>(static_cast<T*>(a.du) + at, cols(p), d);
        }
        mean = next_mean;
        rstd = next_rstd;
    }
    dev::pdl_launch_dependents();
    if (!a.dweight && !a.dbias) return;
    float* sums = a.workspace + 2 * int64_t(blockIdx.x) * H;
#pragma unroll
    for (int p = 0; p < kRingPer; ++p) {
        store_v8<G>(sums, cols(p), dw[p]);
        store_v8<G>(sums + H, cols(p), db[p]);
    }
}

// How a launch of many rows is divided.
struct RingShape {
    int threads, blocks, stages;        // blocks 0: the rows do not fit
    size_t smem;
};
// stage_bytes(threads): of one row.
template <typename F>
RingShape ring_shape(int64_t rows, int hidden, F&& stage_bytes) {
    RingShape s = {};
    s.threads = (hidden + 256 * kRingPer - 1) / (256 * kRingPer) * 32;
    if (s.threads > kRingThreads) return s;
    const uint32_t bytes = stage_bytes(s.threads);
    for (int per_sm = std::min(kRingThreads / s.threads, 24); per_sm > 0; --per_sm) {
        s.stages = std::min<int>(kRingStages, (kRingSmem / per_sm - 2048) / bytes);
        if (s.stages < 3 && !(per_sm == 1 && s.stages == 2)) continue;
        s.smem = size_t(s.stages) * bytes;
        s.blocks = static_cast<int>(std::min<int64_t>(rows, int64_t(sm_count()) * per_sm));
        return s;
    }
    return s;
}

// Launches a kernel of many rows; the first time on a device it is allowed its
// shared memory.
template <auto KERNEL, typename Args>
cudaError_t launch_ring(const RingShape& s, const Args& a, cudaStream_t stream) {
    static std::atomic<uint64_t> known{0};       // a bit per device
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if (e == cudaSuccess && !(known.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem - 2048);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e == cudaSuccess) known.fetch_or(bit, std::memory_order_release);
    }
    return e != cudaSuccess ? e : launch_pdl(KERNEL, dim3(s.blocks), dim3(s.threads), s.smem, stream, a, s.stages);
}

// ---- column sums -----------------------------------------------------------------
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
        a.workspace[(2 * share + warp) * H + col] = sum;
    } else {
        void* out = warp == 0 ? a.dweight : a.dbias;
        if (out) set_param<T>(out, a.param_f32, col, sum);
    }
}

// Joins the sums of `parts` blocks or shares, [part][2][H], in a fixed order: a warp
// takes every so many-th part of 32 columns, eight loads at a time.
constexpr int kJoinBatch = 8;

template <typename T>
__global__ void __launch_bounds__(1024) layer_norm_join_kernel(const LayerNormBackwardArgs a, int parts) {
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ways = blockDim.x >> 5, H = a.hidden;
    const int col = blockIdx.x * 32 + lane;
    void* out = blockIdx.y == 0 ? a.dweight : a.dbias;
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if ((a.noop && *a.noop != 0.0f) || !out) return;
    const float* from = a.workspace + int64_t(blockIdx.y) * H + min(col, H - 1);
    float sum = 0.0f;
    for (int i0 = warp; i0 < parts; i0 += ways * kJoinBatch) {
        float v[kJoinBatch];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) v[i] = from[2 * int64_t(min(i0 + i * ways, parts - 1)) * H];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) sum += i0 + i * ways < parts ? v[i] : 0.0f;
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || col >= H) return;
    for (int i = 1; i < ways; ++i) sum += sums[i][lane];
    set_param<T>(out, a.param_f32, col, sum);
}

// Threads of a block that holds a row of `hidden` columns, PER groups of eight each.
int row_threads(int hidden, int per) { return (hidden + 256 * per - 1) / (256 * per) * 32; }
int row_per(int hidden) { return hidden <= 8192 ? 1 : hidden <= 16384 ? 2 : 4; }

int column_shares(int64_t rows, int64_t hidden) {
    const int64_t blocks = (hidden + 31) / 32;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((rows + 127) / 128, 600 / std::max<int64_t>(blocks, 1))));
}

// Blocks of a launch of many rows, at most: the workspace has room for them.
int64_t most_blocks(int64_t rows, int64_t hidden) {
    const int threads = row_threads(static_cast<int>(hidden), kRingPer);
    if (threads < 1 || threads > kRingThreads || rows <= sm_count()) return 0;
    return std::min<int64_t>(rows, int64_t(sm_count()) * std::min(kRingThreads / threads, 24));
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, int dtype, int res_dtype, cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 && all_aligned(a.u, a.res, a.weight, a.bias, a.res_out, a.y);
    const int per = row_per(a.hidden);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        const RingShape s = ring_shape(a.rows, a.hidden, [&](int threads) {
            auto of = [&](int size) { return vec ? slot_bytes<8>(threads, a.hidden, size) : slot_bytes<1>(threads, a.hidden, size); };
            return of(sizeof(R)) + (a.u ? of(sizeof(T)) : 0);
        });
        if (s.blocks > 0 && a.rows > s.blocks)
            return vec ? launch_ring<layer_norm_kernel<T, R, 8>>(s, a, stream)
                       : launch_ring<layer_norm_kernel<T, R, 1>>(s, a, stream);
        auto* kernel = per == 1 ? (vec ? layer_norm_row_kernel<T, R, 8, 1> : layer_norm_row_kernel<T, R, 1, 1>)
                     : per == 2 ? (vec ? layer_norm_row_kernel<T, R, 8, 2> : layer_norm_row_kernel<T, R, 1, 2>)
                                : (vec ? layer_norm_row_kernel<T, R, 8, 4> : layer_norm_row_kernel<T, R, 1, 4>);
        return launch_pdl(kernel, dim3(static_cast<unsigned>(a.rows)), dim3(row_threads(a.hidden, per)), 0,
                          stream, a);
    });
}

size_t layer_norm_backward_workspace(int64_t rows, int64_t hidden) {
    const int shares = column_shares(rows, hidden);
    const int64_t parts = std::max<int64_t>(shares > 1 ? shares : 0, most_blocks(rows, hidden));
    return (size_t(parts) * 2 * hidden * sizeof(float) + 15) / 16 * 16;
}

cudaError_t launch_layer_norm_backward(const LayerNormBackwardArgs& a, int dtype, int res_dtype,
                                       cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 &&
                     all_aligned(a.dy, a.dres_out, a.res_out, a.weight, a.dres, a.du);
    const int per = row_per(a.hidden);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        const RingShape s = ring_shape(a.rows, a.hidden, [&](int threads) {
            auto of = [&](int size) { return vec ? slot_bytes<8>(threads, a.hidden, size) : slot_bytes<1>(threads, a.hidden, size); };
            return of(sizeof(R)) * (a.dres_out ? 2 : 1) + of(sizeof(T));
        });
        cudaError_t e = cudaSuccess;
        int parts;
        if (s.blocks > 0 && a.rows > s.blocks) {
            e = vec ? launch_ring<layer_norm_backward_kernel<T, R, 8>>(s, a, stream)
                    : launch_ring<layer_norm_backward_kernel<T, R, 1>>(s, a, stream);
            if (e != cudaSuccess || (!a.dweight && !a.dbias)) return e;
            parts = s.blocks;
        } else {
            auto* kernel = per == 1 ? (vec ? layer_norm_backward_row_kernel<T, R, 8, 1> : layer_norm_backward_row_kernel<T, R, 1, 1>)
                         : per == 2 ? (vec ? layer_norm_backward_row_kernel<T, R, 8, 2> : layer_norm_backward_row_kernel<T, R, 1, 2>)
                                    : (vec ? layer_norm_backward_row_kernel<T, R, 8, 4> : layer_norm_backward_row_kernel<T, R, 1, 4>);
            if (a.rows > 0)
                e = launch_pdl(kernel, dim3(static_cast<unsigned>(a.rows)), dim3(row_threads(a.hidden, per)), 0, stream, a);
            if (e != cudaSuccess || (!a.dweight && !a.dbias)) return e;
            parts = column_shares(a.rows, a.hidden);
            e = launch_pdl(layer_norm_columns_kernel<T, R>, dim3((a.hidden + 31) / 32, parts), dim3(32 * kColumnWarps), 0,
                           stream, a, parts);
            if (e != cudaSuccess || parts == 1) return e;
        }
        return launch_pdl(layer_norm_join_kernel<T>, dim3((a.hidden + 31) / 32, 2), dim3(parts > 256 ? 1024 : 256), 0,
                          stream, a, parts);
    });
}

}  // namespace ct
