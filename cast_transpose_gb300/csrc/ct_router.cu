// ct_router.cu -- the router of a mixture-of-experts block: the choice of the
// experts, their weights, the counts per expert, the balance and z losses, and
// the gradient of the logits.
#include "ct_device.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"
#include "ct_vec.cuh"

#include <algorithm>

namespace ct {
namespace {

// A warp takes a token; its lane l holds the logits of the experts l, l + 32, ...
constexpr int kRouterWarps = 8;
constexpr int kRouterMaxBlocks = 304;
constexpr unsigned kAll = 0xFFFFFFFFu;

// Logits as numbers of the same order; equal values (0 and -0) get the same one.
// -inf, which is never chosen, and what lies past the last expert come lowest,
// a NaN highest.
constexpr unsigned kNever = 0x007FFFFFu;
__device__ __forceinline__ unsigned order_of(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const unsigned b = __float_as_uint(v + 0.0f);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float of_order(unsigned o) {
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

template <int N, typename T>
__device__ __forceinline__ void load_logits(const RouterArgs& a, int64_t t, float (&x)[N]) {
    const T* row = static_cast<const T*>(a.logits) + t * a.experts;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lane + 32 * i;
        x[i] = e < a.experts ? dev::to_f32(row[e]) : -INFINITY;
    }
}

// exp(x - top) in place of x; the sum of all.
template <int N>
__device__ __forceinline__ float exponentials(float (&x)[N], float top) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = expf(x[i] - top);
        sum += x[i];
    }
    return dev::warp_sum(sum);
}

// Per block of a launch: sums of the probabilities [E], counts [E + 1] (last:
// the tokens), the sum of squared logsumexps.
__device__ __forceinline__ float* block_probs(const RouterArgs& a, int64_t b) {
    return static_cast<float*>(a.workspace) + b * (2 * a.experts + 2);
}
__device__ __forceinline__ int* block_counts(const RouterArgs& a, int64_t b) {
    return reinterpret_cast<int*>(block_probs(a, b) + a.experts);
}

__device__ __forceinline__ void put_loss(const RouterArgs& a, float balance, float squares, int tokens) {
    if (!a.loss) return;
    const float n = static_cast<float>(tokens);
    *a.loss = tokens == 0 ? 0.0f
                          : a.balance * a.experts * (balance / (n * a.topk)) / n + a.z * (squares / n);
}

template <int N, typename T>
__global__ void __launch_bounds__(32 * kRouterWarps) router_kernel(const RouterArgs a) {
    extern __shared__ float smem[];
    float* probs = smem;                                                       // [warps][E]
    int* counts = reinterpret_cast<int*>(smem + kRouterWarps * a.experts);     // [E + 1]
    __shared__ float warp_squares[kRouterWarps], warp_balance[kRouterWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.experts, K = a.topk;
    dev::pdl_launch_dependents();
    for (int e = tid; e <= E; e += blockDim.x) counts[e] = 0;
    __syncthreads();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    float sums[N] = {};
    float squares = 0.0f;
    int tokens = 0;
    for (int64_t t = int64_t(blockIdx.x) * kRouterWarps + warp; t < a.tokens; t += int64_t(gridDim.x) * kRouterWarps) {
        float x[N];
        unsigned key[N];
        const bool counted = !a.mask || a.mask[t];
        int chosen[2] = {-1, -1};           // lane k: of slots k and k + 32
        float logit[2] = {};
        if (counted) {
            load_logits<N, T>(a, t, x);
#pragma unroll
            for (int i = 0; i < N; ++i) key[i] = lane + 32 * i < E ? order_of(x[i]) : 0;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) key[i] = 0;
        }
        float top = 0.0f;
        bool any = false;
        for (int k = 0; k < K; ++k) {
            unsigned best = key[0];
            int at = 0;
#pragma unroll
            for (int i = 1; i < N; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = i;
                }
            const unsigned most = __reduce_max_sync(kAll, best);
            if (most <= kNever) break;
            const int e = __reduce_min_sync(kAll, best == most ? unsigned(lane + 32 * at) : 0xFFFFu);
            if (k == 0) {
                top = of_order(most);
                any = true;
            }
            if (lane == (k & 31)) {
                chosen[k >> 5] = e;
                logit[k >> 5] = of_order(most);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (e == lane + 32 * i) key[i] = 0;
        }
        float sum = 1.0f;
        if (any) {
            sum = exponentials(x, top);
            const float lse = top + logf(sum);
            squares = fmaf(lse, lse, squares);
            ++tokens;
#pragma unroll
            for (int i = 0; i < N; ++i) sums[i] += x[i] / sum;
        }
        float part[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) part[i] = chosen[i] >= 0 ? expf(logit[i] - top) : 0.0f;
        if (a.normalize && any) sum = dev::warp_sum(part[0] + part[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = lane + 32 * i;
            if (k >= K) continue;
            a.idx[t * K + k] = chosen[i];
            a.weights[t * K + k] = part[i] / sum;
            if (chosen[i] >= 0) atomicAdd(counts + chosen[i], 1);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane + 32 * i < E) probs[warp * E + lane + 32 * i] = sums[i];
    if (lane == 0) {
        warp_squares[warp] = squares;
        atomicAdd(counts + E, tokens);
    }
    __syncthreads();
    const bool last = gridDim.x == 1;
    float balance = 0.0f;
    for (int e = tid; e <= E; e += blockDim.x) {
        const int count = counts[e];
        if (e < E) {
            float p = 0.0f;
            for (int w = 0; w < kRouterWarps; ++w) p += probs[w * E + e];
            balance = fmaf(static_cast<float>(count), p, balance);
            if (!last) block_probs(a, blockIdx.x)[e] = p;
        }
        if (last)
            a.counts[e] = count;
        else
            block_counts(a, blockIdx.x)[e] = count;
    }
    balance = dev::warp_sum(balance);
    if (lane == 0) warp_balance[warp] = balance;
    __syncthreads();
    if (tid != 0) return;
    float all = 0.0f, loss = 0.0f;
    for (int w = 0; w < kRouterWarps; ++w) {
        all += warp_squares[w];
        loss += warp_balance[w];
    }
    if (last)
        put_loss(a, loss, all, counts[E]);
    else
        reinterpret_cast<float*>(block_counts(a, blockIdx.x))[E + 1] = all;
}

// Joins the blocks' sums, in their order.
constexpr int kRouterJoinThreads = 1024;

__global__ void __launch_bounds__(kRouterJoinThreads) router_join_kernel(const RouterArgs a, int blocks) {
    __shared__ float warp_sums[2][32];
    __shared__ int all_tokens;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.experts;
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    float balance = 0.0f, squares = 0.0f;
    for (int e = tid; e <= E; e += blockDim.x) {
        float p = 0.0f;
        int count = 0;
        for (int b = 0; b < blocks; ++b) {
            count += block_counts(a, b)[e];
            if (e < E) p += block_probs(a, b)[e];
        }
        a.counts[e] = count;
        if (e < E) balance = fmaf(static_cast<float>(count), p, balance);
        else all_tokens = count;
    }
    for (int b = tid; b < blocks; b += blockDim.x)
        squares += reinterpret_cast<const float*>(block_counts(a, b))[E + 1];
    balance = dev::warp_sum(balance);
    squares = dev::warp_sum(squares);
    if (lane == 0) {
        warp_sums[0][warp] = balance;
        warp_sums[1][warp] = squares;
    }
    __syncthreads();
    if (tid >= 32) return;
    balance = dev::warp_sum(warp_sums[0][lane]);
    squares = dev::warp_sum(warp_sums[1][lane]);
    if (tid == 0) put_loss(a, balance, squares, all_tokens);
}

// With p = softmax(logits), A_e = c f_e + (its weight's gradient, where weights are
// probabilities), f_e = counts_e / (n K), c = dloss balance E / n:
//   dlogits_e = p_e (A_e - sum p A + 2 dloss z logsumexp / n)
// and, where weights are a softmax over the chosen experts, w_k (dw_k - sum w dw)
// at those.
template <int N, typename T>
__global__ void __launch_bounds__(32 * kRouterWarps) router_backward_kernel(const RouterArgs a) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.experts, K = a.topk;
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const float n = static_cast<float>(max(a.counts[E], 1)), dloss = a.dloss ? *a.dloss : 0.0f;
    const float z = 2.0f * a.z * dloss / n;
    float load[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lane + 32 * i;
        load[i] = e < E ? a.balance * dloss * E / n * (a.counts[e] / (n * K)) : 0.0f;
    }
    for (int64_t t = int64_t(blockIdx.x) * kRouterWarps + warp; t < a.tokens; t += int64_t(gridDim.x) * kRouterWarps) {
        T* out = static_cast<T*>(a.dlogits) + t * E;
        float x[N], g[N] = {}, each[N];
        float top = -INFINITY;
        bool nan = false;
        if (!a.mask || a.mask[t]) {
            load_logits<N, T>(a, t, x);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                top = fmaxf(top, x[i]);
                nan |= x[i] != x[i];
            }
        }
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        if (!__any_sync(kAll, top > -INFINITY || nan)) {      // not a token
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (lane + 32 * i < E) dev::from_f32(out[lane + 32 * i], 0.0f);
            continue;
        }
        int chosen[2];
        float dw[2], w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = lane + 32 * i;
            chosen[i] = k < K ? a.idx[t * K + k] : -1;
            if (chosen[i] >= E || !a.dweights) chosen[i] = -1;
            dw[i] = chosen[i] >= 0 ? a.dweights[t * K + k] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) each[i] = load[i];
        if (a.normalize) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = chosen[i] >= 0
                           ? expf(dev::to_f32(static_cast<const T*>(a.logits)[t * E + chosen[i]]) - top) : 0.0f;
            const float sum = dev::warp_sum(w[0] + w[1]);
            const float dot = dev::warp_sum(w[0] * dw[0] + w[1] * dw[1]) / sum;
#pragma unroll
            for (int i = 0; i < 2; ++i) dw[i] = w[i] / sum * (dw[i] - dot);
        }
        if (a.dweights)
            for (int k = 0; k < K; ++k) {
                const int e = __shfl_sync(kAll, k < 32 ? chosen[0] : chosen[1], k & 31);
                const float d = __shfl_sync(kAll, k < 32 ? dw[0] : dw[1], k & 31);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (e == lane + 32 * i) (a.normalize ? g : each)[i] += d;
            }
        const float sum = exponentials(x, top);
        const float lse = top + logf(sum);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] /= sum;
            dot = fmaf(x[i], each[i], dot);
        }
        dot = dev::warp_sum(dot);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 32 * i < E)
                dev::from_f32(out[lane + 32 * i], fmaf(x[i], each[i] - dot + z * lse, g[i]));
    }
}

int router_blocks(int64_t tokens) {
    return static_cast<int>(std::min<int64_t>(kRouterMaxBlocks, (tokens + kRouterWarps - 1) / kRouterWarps));
}

// The kernel for this many experts, K<N, T>::get(), N of them per lane.
template <template <int, typename> class K, typename F>
cudaError_t by_experts(int experts, int dtype, F&& f) {
    return by_types(dtype, dtype, [&](auto t, auto) {
        using T = decltype(t);
        return experts <= 32 ? f(K<1, T>::get()) : experts <= 64 ? f(K<2, T>::get())
             : experts <= 128 ? f(K<4, T>::get()) : experts <= 256 ? f(K<8, T>::get())
             : experts <= 512 ? f(K<16, T>::get()) : f(K<32, T>::get());
    });
}
template <int N, typename T>
struct Forward {
    static auto get() { return router_kernel<N, T>; }
};
template <int N, typename T>
struct Backward {
    static auto get() { return router_backward_kernel<N, T>; }
};

}  // namespace

size_t router_workspace(int64_t tokens, int topk, int experts) {
    const int blocks = router_blocks(tokens);
    return blocks > 1 ? size_t(blocks) * (2 * experts + 2) * 4 : 0;
}

cudaError_t launch_router(const RouterArgs& a, int dtype, cudaStream_t stream) {
    const int blocks = std::max(1, router_blocks(a.tokens));
    const size_t smem = (size_t(kRouterWarps) * a.experts + a.experts + 1) * 4;   // 36 KB at most
    const cudaError_t e = by_experts<Forward>(a.experts, dtype, [&](auto kernel) {
        return launch_pdl(kernel, dim3(blocks), dim3(32 * kRouterWarps), smem, stream, a);
    });
    if (e != cudaSuccess || blocks == 1) return e;
    return launch_pdl(router_join_kernel, dim3(1), dim3(kRouterJoinThreads), 0, stream, a, blocks);
}

cudaError_t launch_router_backward(const RouterArgs& a, int dtype, cudaStream_t stream) {
    const int64_t blocks = std::min<int64_t>((a.tokens + kRouterWarps - 1) / kRouterWarps, int64_t(sm_count()) * 8);
    return by_experts<Backward>(a.experts, dtype, [&](auto kernel) {
        return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(32 * kRouterWarps), 0, stream, a);
    });
}

}  // namespace ct
