// ct_norm.cu -- the junction between two blocks: norm, gate, residual sum and
// norm, forward and backward.
//
// Both passes are bound by HBM: forward reads u and res and writes res_out and
// y, backward reads dy, dres_out, u and res_out and writes du and dres, with a
// few operations per element.  Each row needs two sums over its columns, the
// second of which depends on the first, so what has to be avoided is memory
// standing still while a row waits for them.  The design, common to both:
//   - a cluster of blocks owns a contiguous run of rows, each of its blocks a
//     fixed slice of the columns, each thread eight fixed columns: parameters
//     stay in the thread's own shared memory, the backward pass's column sums
//     in its registers;
//   - rows arrive in a ring of shared-memory stages by bulk copies that one
//     thread issues rows ahead, so loads are in flight during every barrier;
//   - the first sum of row i+1 and the second sum of row i share one barrier.
// Rows shorter than kMaxSlice columns take one block; longer ones a cluster of
// 2, 4 or 8 that exchange partial sums through distributed shared memory.
// Few rows, odd sizes and unaligned buffers take the same kernels with plain
// loads in place of the ring.
#include "ct_device.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"

#include <algorithm>
#include <type_traits>

namespace ct {
namespace {

constexpr int kMaxThreads = 768;      // 80 registers a thread
constexpr int kMaxSlice = 8 * kMaxThreads;
constexpr int kMaxCluster = 8;
constexpr int kMaxStages = 4;
constexpr int kSmemPerSm = 227 * 1024;
constexpr int kSmemFixed = 8 * 1024;  // static shared memory and the system's, per block

// How a launch divides the work.
struct NormShape {
    int cluster;        // blocks per row
    int width;          // columns per block, a multiple of 8
    int stages;         // of the ring; 0: plain loads
    int clusters;       // runs of rows
};

// Bits as of the cast kernels' diagnostic word (ct_internal.h).
__device__ unsigned int g_norm_error;

// Rows [first, last) of run c out of `runs`.
__host__ __device__ __forceinline__ int64_t run_begin(int64_t rows, int64_t c, int64_t runs) {
    return rows * c / runs;
}
// The run that row r is in.
__device__ __forceinline__ int64_t run_of(int64_t rows, int64_t r, int64_t runs) {
    return ((r + 1) * runs - 1) / rows;
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

// Eight fp32 values of a thread in shared memory that no other thread reads:
// two planes of one float4 per thread, so that a warp's accesses are
// consecutive.
struct Own {
    float4* base;
    int threads;
    __device__ __forceinline__ void put(int slot, const float (&f)[8]) const {
        float4* p = base + 2 * slot * threads + threadIdx.x;
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[threads] = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ void get(int slot, float (&f)[8]) const {
        const float4* p = base + 2 * slot * threads + threadIdx.x;
        const float4 a = p[0], b = p[threads];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

// scale * (offset + w) of the thread's columns; scale without a weight.
template <typename T, bool VEC>
__device__ __forceinline__ void load_param(const void* p, int f32, int64_t at, float offset,
                                           float scale, const dev::Cols<VEC>& c, float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = scale;
        return;
    }
    if (f32)
        dev::load_cols<VEC>(static_cast<const float*>(p) + at, c, f);
    else
        dev::load_cols<VEC>(static_cast<const T*>(p) + at, c, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = scale * (offset + f[j]);
}

// Sums of a and b over the cluster's blocks, the same in every thread, in a
// fixed order; one barrier.  `slots` [2][kMaxCluster * warps]: a call writes
// the half that the call before it did not, which everyone has finished with
// once this call's barrier is passed.
struct RowSums {
    float2 (*slots)[kMaxCluster * kMaxThreads / 32];
    int cluster, rank, turn;

    __device__ __forceinline__ float2 operator()(float a, float b) {
        const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        a = dev::warp_sum(a);
        b = dev::warp_sum(b);
        float2* half = slots[turn];
        turn ^= 1;
        if (cluster == 1) {
            if (lane == 0) half[warp] = make_float2(a, b);
            __syncthreads();
        } else {
            if (lane < cluster) {
                uint32_t remote;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(remote)
                             : "r"(dev::smem_u32(half + rank * warps + warp)), "r"(lane));
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(a), "f"(b)
                             : "memory");
            }
            cluster_barrier();
        }
        a = b = 0.0f;
        for (int i = lane; i < cluster * warps; i += 32) {
            a += half[i].x;
            b += half[i].y;
        }
        return make_float2(dev::warp_sum(a), dev::warp_sum(b));
    }

    // Every block of the cluster has begun and set up its shared memory.
    static __device__ __forceinline__ void start(int cluster) {
        if (cluster == 1)
            __syncthreads();
        else
            cluster_barrier();
    }
    static __device__ __forceinline__ void cluster_barrier() {
        asm volatile("barrier.cluster.arrive.release;\n\t"
                     "barrier.cluster.wait.acquire;" ::: "memory");
    }
};

// The ring: stage s holds one row's slices of up to four tensors, one after
// the other.  Thread 0 issues the copies; everyone waits on full[s].
struct Ring {
    uint64_t* full;
    uint8_t* base;
    uint32_t stage_bytes;
    int stages;
    bool lost;          // a wait gave up: no more waiting, the error is reported

    __device__ __forceinline__ uint8_t* at(int stage) const { return base + stage * stage_bytes; }
    __device__ __forceinline__ void wait(int stage, uint32_t parity) {
        if (!lost && !dev::mbar_wait_bounded(full + stage, parity)) lost = true;
    }
    __device__ __forceinline__ void copy(int stage, uint32_t offset, const void* src,
                                         uint32_t bytes) const {
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
            ::"r"(dev::smem_u32(at(stage)) + offset), "l"(src), "r"(bytes),
            "r"(dev::smem_u32(full + stage)) : "memory");
    }
};

// A position in the ring.
struct Turn {
    int stage = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++stage == stages) {
            stage = 0;
            parity ^= 1;
        }
    }
};

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


// Forward.  Per row: sum u^2 -> rstd_post; res_out and sum res_out^2 ->
// rstd_pre; y.
template <typename T, typename R, bool VEC, bool RING>
__global__ void __launch_bounds__(kMaxThreads, 1) block_norm_kernel(const NormArgs a,
                                                                    const NormShape s) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 slots[2][kMaxCluster * kMaxThreads / 32];
    __shared__ __align__(8) uint64_t full[kMaxStages];
    __shared__ unsigned block_max;
    const int tid = threadIdx.x, H = a.hidden;
    const int rank = blockIdx.x % s.cluster, run = blockIdx.x / s.cluster;
    const int col0 = rank * s.width, W = min(s.width, H - col0);
    const dev::Cols<VEC> c(tid, blockDim.x, W);
    const int64_t begin = run_begin(a.rows, run, s.clusters), end = run_begin(a.rows, run + 1, s.clusters);
    const T* u = static_cast<const T*>(a.u) + col0;
    const R* res = static_cast<const R*>(a.res) + col0;
    const uint32_t u_at = s.width * sizeof(R);   // in a stage: res, then u
    Ring ring{full, smem, static_cast<uint32_t>(s.width * (sizeof(R) + sizeof(T))), s.stages, false};
    const Own own{reinterpret_cast<float4*>(smem + (RING ? s.stages * ring.stage_bytes : 0)),
                  static_cast<int>(blockDim.x)};
    enum { kPost, kPre, kGate };
    RowSums sums{slots, s.cluster, rank, 0};

    dev::pdl_launch_dependents();
    if (tid == 0) {
        block_max = 0;
        if constexpr (RING) {
            for (int i = 0; i < s.stages; ++i) dev::mbar_init(full + i, 1);
            dev::fence_barrier_init();
        }
    }
    RowSums::start(s.cluster);
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    auto fetch = [&](int64_t row, int stage) {
        dev::mbar_arrive_expect_tx(full + stage, W * (sizeof(R) + (a.u ? sizeof(T) : 0)));
        ring.copy(stage, 0, res + row * H, W * sizeof(R));
        if (a.u) ring.copy(stage, u_at, u + row * H, W * sizeof(T));
    };
    if constexpr (RING)
        if (tid == 0)
            for (int i = 0; i < s.stages && begin + i < end; ++i) fetch(begin + i, i);
    const float alpha = a.branch_scale, beta = a.residual_scale;
    int64_t gate_row = a.gate ? begin / a.rows_per_gate : 0;
    int64_t gate_end = a.gate ? (gate_row + 1) * a.rows_per_gate : a.rows;
    {
        float f[8];
        if (a.u) {
            load_param<T>(a.post ? a.w_post : nullptr, a.param_f32, col0,
                          a.post ? a.weight_offset : 0.0f, 1.0f, c, f);
            own.put(kPost, f);
            load_param<T>(a.gate, a.param_f32, gate_row * H + col0, 0.0f, alpha, c, f);
            own.put(kGate, f);
        }
        if (a.pre) {
            load_param<T>(a.w_pre, a.param_f32, col0, a.weight_offset, 1.0f, c, f);
            own.put(kPre, f);
        }
    }
    const float scale = a.scale ? *a.scale : 0.0f;
    const float per_column = 1.0f / H;
    unsigned most = 0;

    auto sum_u = [&](int64_t row, int stage) {
        float f[8], sum = 0.0f;
        dev::load_cols<VEC>(RING ? reinterpret_cast<const T*>(ring.at(stage) + u_at) : u + row * H, c, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
        return sum;
    };
    Turn now, ahead;
    if (RING) ring.wait(now.stage, now.parity);
    float rstd_u = 1.0f;
    if (a.post) {
        rstd_u = rsqrtf(sums(sum_u(begin, 0), 0.0f).x * per_column + a.eps);
        if (a.rstd_post && rank == 0 && tid == 0) a.rstd_post[begin] = rstd_u;
    }
    for (int64_t row = begin; row < end; ++row) {
        float v[8], sum_v = 0.0f, next_u = 0.0f;
        dev::load_cols<VEC>(RING ? reinterpret_cast<const R*>(ring.at(now.stage)) : res + row * H, c, v);
        if (a.u) {
            if (row == gate_end) {
                gate_end += a.rows_per_gate;
                float f[8];
                load_param<T>(a.gate, a.param_f32, ++gate_row * H + col0, 0.0f, alpha, c, f);
                own.put(kGate, f);
            }
            float x[8], w[8], g[8];
            dev::load_cols<VEC>(RING ? reinterpret_cast<const T*>(ring.at(now.stage) + u_at) : u + row * H,
                                c, x);
            own.get(kPost, w);
            own.get(kGate, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = beta * v[j] + g[j] * (x[j] * rstd_u * w[j]);
            dev::store_cols<VEC>(static_cast<R*>(a.res_out) + row * H + col0, c, v);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.has(j)) sum_v = fmaf(v[j], v[j], sum_v);
        ahead = now;
        ahead.next(s.stages);
        if (row + 1 < end) {
            if (RING) ring.wait(ahead.stage, ahead.parity);
            if (a.post) next_u = sum_u(row + 1, ahead.stage);
        }
        const float2 sum = sums(next_u, sum_v);
        // everyone has read this row's stage
        if constexpr (RING)
            if (tid == 0 && row + s.stages < end) fetch(row + s.stages, now.stage);
        now = ahead;
        if (a.post) {
            rstd_u = rsqrtf(sum.x * per_column + a.eps);
            if (a.rstd_post && rank == 0 && tid == 0 && row + 1 < end) a.rstd_post[row + 1] = rstd_u;
        }
        if (!a.pre) continue;
        const float rstd = rsqrtf(sum.y * per_column + a.eps);
        if (a.rstd_pre && rank == 0 && tid == 0) a.rstd_pre[row] = rstd;
        float w[8];
        own.get(kPre, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= rstd * w[j];
        if (a.scale) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c.has(j)) most = max(most, __float_as_uint(v[j]) & 0x7FFFFFFFu);
            store_fp8<VEC>(static_cast<uint8_t*>(a.y) + row * H + col0, c, v, scale, a.fmt);
        } else {
            dev::store_cols<VEC>(static_cast<T*>(a.y) + row * H + col0, c, v);
        }
    }
    if (a.scale && a.pre) {
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        if ((tid & 31) == 0) atomicMax(&block_max, most);
        __syncthreads();
        if (tid == 0) {
            if (block_max) atomicMax(reinterpret_cast<unsigned*>(a.amax), block_max);
            if (blockIdx.x == 0) *a.scale_inv = __fdiv_rn(1.0f, scale);
        }
    }
    if (RING && ring.lost && tid == 0) atomicOr(&g_norm_error, kErrWaitTimeout);
    // a block's shared memory stays until its peers have sent their last sums
    if (s.cluster > 1) RowSums::cluster_barrier();
}

// What the workspace holds for the backward pass, [clusters][H] each: partial
// column sums of dw_pre and dw_post, and those of dgate for the first and the
// last gate row of a run, where they belong to other runs too.
enum { kSumPre, kSumPost, kSumGateFirst, kSumGateLast, kSums };

// Backward.  With xh = res_out rstd_pre, G = dy a_pre, uh = u rstd_post:
//   D  = dres_out + rstd_pre (G - xh mean(G xh))      dres = beta D
//   P  = alpha gate D a_post                           du = rstd_post (P - uh mean(P uh))
//   dw_pre = sum dy xh,  dw_post = sum alpha gate D uh,  dgate = sum alpha D uh a_post
template <typename T, typename R, bool VEC, bool RING>
__global__ void __launch_bounds__(kMaxThreads, 1)
    block_norm_backward_kernel(const NormBackwardArgs a, const NormShape s) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 slots[2][kMaxCluster * kMaxThreads / 32];
    __shared__ __align__(8) uint64_t full[kMaxStages];
    const int tid = threadIdx.x, H = a.hidden;
    const int rank = blockIdx.x % s.cluster, run = blockIdx.x / s.cluster;
    const int col0 = rank * s.width, W = min(s.width, H - col0);
    const dev::Cols<VEC> c(tid, blockDim.x, W);
    const int64_t begin = run_begin(a.rows, run, s.clusters), end = run_begin(a.rows, run + 1, s.clusters);
    // in a stage: res_out, dres_out, dy, u
    const uint32_t dres_at = s.width * sizeof(R), dy_at = 2 * dres_at, u_at = dy_at + s.width * sizeof(T);
    Ring ring{full, smem, static_cast<uint32_t>(2 * s.width * (sizeof(R) + sizeof(T))), s.stages, false};
    const Own own{reinterpret_cast<float4*>(smem + (RING ? s.stages * ring.stage_bytes : 0)),
                  static_cast<int>(blockDim.x)};
    enum { kPost, kPre, kGate };
    RowSums sums{slots, s.cluster, rank, 0};
    const R* res_out = static_cast<const R*>(a.res_out) + col0;
    const R* dres_out = static_cast<const R*>(a.dres_out) + col0;
    const T* dy = static_cast<const T*>(a.dy) + col0;
    const T* u = static_cast<const T*>(a.u) + col0;

    dev::pdl_launch_dependents();
    if constexpr (RING) {
        if (tid == 0) {
            for (int i = 0; i < s.stages; ++i) dev::mbar_init(full + i, 1);
            dev::fence_barrier_init();
        }
    }
    RowSums::start(s.cluster);
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    auto fetch = [&](int64_t row, int stage) {
        const uint32_t rb = W * sizeof(R), tb = W * sizeof(T);
        const int64_t at = row * H;
        dev::mbar_arrive_expect_tx(full + stage, (a.pre ? rb + tb : 0) + (a.dres_out ? rb : 0) + (a.u ? tb : 0));
        if (a.pre) {
            ring.copy(stage, 0, res_out + at, rb);
            ring.copy(stage, dy_at, dy + at, tb);
        }
        if (a.dres_out) ring.copy(stage, dres_at, dres_out + at, rb);
        if (a.u) ring.copy(stage, u_at, u + at, tb);
    };
    if constexpr (RING)
        if (tid == 0)
            for (int i = 0; i < s.stages && begin + i < end; ++i) fetch(begin + i, i);
    const float alpha = a.branch_scale, beta = a.u ? a.residual_scale : 1.0f;
    const int64_t first_gate = a.gate ? begin / a.rows_per_gate : 0;
    int64_t gate_row = first_gate;
    int64_t gate_end = a.gate ? (gate_row + 1) * a.rows_per_gate : a.rows;
    {
        float f[8];
        if (a.u) {
            load_param<T>(a.post ? a.w_post : nullptr, a.param_f32, col0,
                          a.post ? a.weight_offset : 0.0f, 1.0f, c, f);
            own.put(kPost, f);
            load_param<T>(a.gate, a.param_f32, gate_row * H + col0, 0.0f, alpha, c, f);
            own.put(kGate, f);
        }
        if (a.pre) {
            load_param<T>(a.w_pre, a.param_f32, col0, a.weight_offset, 1.0f, c, f);
            own.put(kPre, f);
        }
    }
    const float per_column = 1.0f / H;
    float dw_pre[8] = {}, dw_post[8] = {}, dgate[8] = {};

    // sum of G xh over the row, and the row's part of dw_pre
    auto first_sum = [&](int64_t row, int stage, float rstd) {
        float g[8], x[8], w[8], sum = 0.0f;
        dev::load_cols<VEC>(RING ? reinterpret_cast<const T*>(ring.at(stage) + dy_at) : dy + row * H, c, g);
        dev::load_cols<VEC>(RING ? reinterpret_cast<const R*>(ring.at(stage)) : res_out + row * H, c, x);
        own.get(kPre, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float t = g[j] * (x[j] * rstd);
            dw_pre[j] += t;
            sum = fmaf(t, w[j], sum);
        }
        return sum;
    };
    // the gate row's sums: whole ones go to dgate, others to the workspace
    auto flush_gate = [&](bool to_the_end) {
        if (a.dgate) {
            const bool whole = gate_row * a.rows_per_gate >= begin && (to_the_end ? min(gate_end, a.rows) <= end : true);
            float* part = a.workspace + (int64_t(gate_row == first_gate ? kSumGateFirst : kSumGateLast) * s.clusters + run) * H + col0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!c.has(j)) continue;
                const float v = alpha * dgate[j];
                if (whole)
                    set_param<T>(a.dgate, a.param_f32, gate_row * H + col0 + c.at(j), v);
                else
                    part[c.at(j)] = v;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) dgate[j] = 0.0f;
    };

    Turn now, ahead;
    float rstd_x = a.pre ? a.rstd_pre[begin] : 0.0f, rstd_u = a.post ? a.rstd_post[begin] : 1.0f;
    if (RING) ring.wait(now.stage, now.parity);
    float mean_x = 0.0f;
    if (a.pre) mean_x = sums(first_sum(begin, 0, rstd_x), 0.0f).x * per_column;
    for (int64_t row = begin; row < end; ++row) {
        const bool more = row + 1 < end;
        const float next_x = a.pre && more ? a.rstd_pre[row + 1] : 0.0f;
        const float next_u = a.post && more ? a.rstd_post[row + 1] : 1.0f;
        float d[8], p[8], hat[8], sum_p = 0.0f, sum_x = 0.0f;
        if (a.dres_out) {
            dev::load_cols<VEC>(RING ? reinterpret_cast<const R*>(ring.at(now.stage) + dres_at)
                                     : dres_out + row * H, c, d);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = 0.0f;
        }
        if (a.pre) {
            float g[8], x[8], w[8];
            dev::load_cols<VEC>(RING ? reinterpret_cast<const T*>(ring.at(now.stage) + dy_at) : dy + row * H,
                                c, g);
            dev::load_cols<VEC>(RING ? reinterpret_cast<const R*>(ring.at(now.stage)) : res_out + row * H, c, x);
            own.get(kPre, w);
            const float back = rstd_x * rstd_x * mean_x;
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] += rstd_x * (g[j] * w[j]) - x[j] * back;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = beta * d[j];
        dev::store_cols<VEC>(static_cast<R*>(a.dres) + row * H + col0, c, p);
        if (a.u) {
            if (row == gate_end) {
                flush_gate(false);
                gate_end += a.rows_per_gate;
                float f[8];
                load_param<T>(a.gate, a.param_f32, ++gate_row * H + col0, 0.0f, alpha, c, f);
                own.put(kGate, f);
            }
            float w[8];
            dev::load_cols<VEC>(RING ? reinterpret_cast<const T*>(ring.at(now.stage) + u_at) : u + row * H,
                                c, hat);
            own.get(kPost, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                hat[j] *= rstd_u;
                dgate[j] = fmaf(d[j] * hat[j], w[j], dgate[j]);
            }
            own.get(kGate, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[j] *= d[j];
                dw_post[j] = fmaf(p[j], hat[j], dw_post[j]);
                p[j] *= w[j];
                sum_p = fmaf(p[j], hat[j], sum_p);
            }
        }
        ahead = now;
        ahead.next(s.stages);
        if (more) {
            if (RING) ring.wait(ahead.stage, ahead.parity);
            if (a.pre) sum_x = first_sum(row + 1, ahead.stage, next_x);
        }
        const float2 sum = sums(sum_x, sum_p);
        // everyone has read this row's stage
        if constexpr (RING)
            if (tid == 0 && row + s.stages < end) fetch(row + s.stages, now.stage);
        if (a.u) {
            const float mean = a.post ? sum.y * per_column : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = rstd_u * (p[j] - hat[j] * mean);
            dev::store_cols<VEC>(static_cast<T*>(a.du) + row * H + col0, c, p);
        }
        mean_x = sum.x * per_column;
        rstd_x = next_x;
        rstd_u = next_u;
        now = ahead;
    }
    flush_gate(true);
    float* part = a.workspace + int64_t(run) * H + col0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (!c.has(j)) continue;
        if (a.dw_pre) part[int64_t(kSumPre) * s.clusters * H + c.at(j)] = dw_pre[j];
        if (a.dw_post) part[int64_t(kSumPost) * s.clusters * H + c.at(j)] = dw_post[j];
    }
    if (RING && ring.lost && tid == 0) atomicOr(&g_norm_error, kErrWaitTimeout);
    if (s.cluster > 1) RowSums::cluster_barrier();
}

// Joins the runs' column sums, in run order.  blockIdx.y 0, 1: dw_pre, dw_post;
// from 2 on the gate rows that more than one run has rows of, by gate row
// (few of them, perhaps of many runs), else by the run they begin in.
constexpr int kJoinCols = 32, kJoinRuns = 8;

template <typename T>
__global__ void __launch_bounds__(kJoinCols * kJoinRuns)
    block_norm_join_kernel(const NormBackwardArgs a, int64_t runs, int by_gate_row) {
    __shared__ float parts[kJoinRuns][kJoinCols];
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int H = a.hidden, x = threadIdx.x % kJoinCols, y = threadIdx.x / kJoinCols;
    const int which = blockIdx.y;
    int64_t first = 0, last = runs - 1, at = 0;   // the runs to add up
    int col = blockIdx.x * kJoinCols + x;
    void* out = which == 0 ? a.dw_pre : which == 1 ? a.dw_post : a.dgate;
    bool gate_first_is_last = false;
    if (which >= 2) {
        int64_t gate_row;
        if (by_gate_row) {
            gate_row = which - 2;
            first = run_of(a.rows, gate_row * a.rows_per_gate, runs);
        } else {
            // a block of kJoinCols * kJoinRuns columns of the gate row that run
            // `which - 2` ends in, if it begins there
            col = blockIdx.x * (kJoinCols * kJoinRuns) + threadIdx.x;
            first = which - 2;
            gate_row = (run_begin(a.rows, first + 1, runs) - 1) / a.rows_per_gate;
            if (gate_row * a.rows_per_gate < run_begin(a.rows, first, runs)) return;
        }
        last = run_of(a.rows, min((gate_row + 1) * a.rows_per_gate, a.rows) - 1, runs);
        if (first == last) return;                // written by its run
        at = gate_row * H;
        gate_first_is_last = run_begin(a.rows, first, runs) / a.rows_per_gate != gate_row;
    }
    if (!out) return;
    // the sums of run r: a gate row is the last one of the first run unless it
    // is its first one too, and the first one of the others
    auto part = [&](int64_t r) {
        const int kind = which < 2 ? (which == 0 ? kSumPre : kSumPost)
                         : r == first && gate_first_is_last ? kSumGateLast : kSumGateFirst;
        return a.workspace[(int64_t(kind) * runs + r) * H + col];
    };
    float sum = 0.0f;
    if (which >= 2 && !by_gate_row) {
        if (col >= H) return;
        for (int64_t r = first; r <= last; ++r) sum += part(r);
        set_param<T>(out, a.param_f32, at + col, sum);
        return;
    }
    if (col < H) {
#pragma unroll 8
        for (int64_t r = first + y; r <= last; r += kJoinRuns) sum += part(r);
    }
    parts[y][x] = sum;
    __syncthreads();
    if (y == 0 && col < H) {
#pragma unroll
        for (int i = 1; i < kJoinRuns; ++i) sum += parts[i][x];
        set_param<T>(out, a.param_f32, at + col, sum);
    }
}

// The types of u and y, and of the residual stream.
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

int sm_count() {
    static const int count = [] {
        int device = 0, n = 0;
        if (cudaGetDevice(&device) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) {
            cudaGetLastError();
            return 152;
        }
        return n;
    }();
    return count;
}

int round_up(int v, int to) { return (v + to - 1) / to * to; }
int threads_of(int width) { return round_up((width + 7) / 8, 32); }

// Blocks of `width` columns that an SM's registers hold.
int blocks_per_sm(int width) { return kMaxThreads / threads_of(width); }

// The most runs of rows a launch makes: the workspace has room for them.
int64_t max_clusters(int64_t rows, int64_t hidden) {
    int cluster = 1;
    while (round_up(static_cast<int>((hidden + cluster - 1) / cluster), 8) > kMaxSlice) cluster *= 2;
    const int width = round_up(static_cast<int>((hidden + cluster - 1) / cluster), 8);
    return std::min<int64_t>(rows, int64_t(sm_count()) * blocks_per_sm(width) / cluster);
}

// column_bytes: of one column in a stage.  Picks the fewest blocks per row
// whose ring has two stages, then as many blocks per SM as the registers and
// then the ring allow.
NormShape shape_of(int64_t rows, int hidden, int column_bytes, bool vec, size_t* smem) {
    NormShape s = {};
    for (s.cluster = 1;; s.cluster *= 2) {
        s.width = round_up((hidden + s.cluster - 1) / s.cluster, 8);
        if (s.width > kMaxSlice) continue;
        if (s.cluster == kMaxCluster || !vec ||
            s.width * (2 * column_bytes + 12) + kSmemFixed <= kSmemPerSm)
            break;
    }
    const int threads = threads_of(s.width);
    const int own = 3 * 32 * threads;     // three parameters of eight columns
    int per_sm = blocks_per_sm(s.width);
    const int stage = s.width * column_bytes;
    auto stages = [&] { return (kSmemPerSm / per_sm - kSmemFixed - own) / std::max(stage, 1); };
    while (per_sm > 1 && vec && stages() < 2) --per_sm;
    s.clusters = static_cast<int>(std::min<int64_t>(rows, std::max(1, sm_count() * per_sm / s.cluster)));
    // the ring pays for itself once runs are longer than a row
    s.stages = vec && rows > s.clusters ? std::min(kMaxStages, stages()) : 0;
    if (s.stages < 2) s.stages = 0;
    *smem = size_t(own) + size_t(s.stages) * stage;
    return s;
}

template <typename Args>
cudaError_t launch_rows(void (*kernel)(const Args, const NormShape), const Args& a, const NormShape& s,
                        size_t smem, cudaStream_t stream) {
    if (smem > 40 * 1024) {   // 48 KB with the static part
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kSmemPerSm - kSmemFixed);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(s.clusters * s.cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads_of(s.width)));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(s.cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = s.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, s);
}

}  // namespace

cudaError_t read_norm_error(unsigned* value, bool clear) {
    const cudaError_t e = cudaMemcpyFromSymbol(value, g_norm_error, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_norm_error, &zero, sizeof(unsigned));
}

cudaError_t launch_block_norm(const NormArgs& a, int dtype, int res_dtype, cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 && all_aligned(a.u, a.res, a.w_post, a.w_pre, a.gate,
                                                      a.res_out, a.y);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        size_t smem;
        const NormShape s = shape_of(a.rows, a.hidden, sizeof(T) + sizeof(R), vec, &smem);
        auto* kernel = s.stages ? block_norm_kernel<T, R, true, true>
                       : vec    ? block_norm_kernel<T, R, true, false>
                                : block_norm_kernel<T, R, false, false>;
        return launch_rows(kernel, a, s, smem, stream);
    });
}

size_t norm_backward_workspace(int64_t rows, int64_t hidden) {
    return static_cast<size_t>(max_clusters(rows, hidden) * kSums * hidden) * sizeof(float) / 16 * 16 + 16;
}

cudaError_t launch_block_norm_backward(const NormBackwardArgs& a, int dtype, int res_dtype,
                                       cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 &&
                     all_aligned(a.dy, a.dres_out, a.u, a.res_out, a.w_post, a.w_pre, a.gate, a.du,
                                 a.dres);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        size_t smem;
        NormShape s = shape_of(a.rows, a.hidden, 2 * (sizeof(T) + sizeof(R)), vec, &smem);
        s.clusters = static_cast<int>(std::min<int64_t>(s.clusters, max_clusters(a.rows, a.hidden)));
        if (a.rows > 0) {
            auto* kernel = s.stages ? block_norm_backward_kernel<T, R, true, true>
                           : vec    ? block_norm_backward_kernel<T, R, true, false>
                                    : block_norm_backward_kernel<T, R, false, false>;
            const cudaError_t e = launch_rows(kernel, a, s, smem, stream);
            if (e != cudaSuccess) return e;
        }
        if (!a.dw_pre && !a.dw_post && !a.dgate) return cudaSuccess;
        const int64_t gates = a.dgate ? (a.rows + a.rows_per_gate - 1) / a.rows_per_gate : 0;
        const bool by_gate_row = gates <= s.clusters / 2;
        const int64_t joins = !a.dgate ? 0 : by_gate_row ? gates : s.clusters - 1;
        return launch_pdl(block_norm_join_kernel<T>,
                          dim3((a.hidden + kJoinCols - 1) / kJoinCols, static_cast<unsigned>(2 + joins)),
                          dim3(kJoinCols * kJoinRuns), 0, stream, a, int64_t(s.clusters),
                          by_gate_row ? 1 : 0);
    });
}

}  // namespace ct
