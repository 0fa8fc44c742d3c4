// ct_router.cu -- the router of a mixture-of-experts block: the choice of the
// experts, their weights, the counts per expert, the balance and z losses, and
// the gradient of the logits.
//
// One pass over the logits: a warp holds a token's in registers, chooses, and adds
// its probabilities to sums that stay in registers too; blocks add theirs up through
// their cluster's shared memory, a second launch joins the clusters', all in a fixed
// order.  The logits are few bytes (16384 tokens of 256 fp32 17 MB, 2.6 us of HBM);
// what bounds it are instructions, some 610 a token: the choice of 8 among 256 takes a
// third of the time, 256 exponentials a tenth.  Measured, one GB300: that case 19.9 us
// with its join (18 of the launch alone, cold; instructions issue on 61% of the
// cycles, 80 registers leave 24 warps to an SM; 131072 tokens 94), a decoding step of 4
// tokens 3 us and the call; the gradient of the 16384 13.2 us (131072: 86), of 8191
// tokens of 64 bf16 logits 4.1 and the call.
#include "ct_device.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"
#include "ct_vec.cuh"

#include <algorithm>
#include <cfloat>
#include <cooperative_groups.h>

namespace ct {
namespace {

// A warp takes a token; its lane l holds the logits of the experts l, l + 32, ...
constexpr int kRouterWarps = 8;
constexpr int kRouterCluster = 4;
// Blocks of an SM, by their registers, and clusters on the GPU at a time with each.
// (16384 tokens of 1024 experts 43.7 us; with three blocks' clusters, of which most
// come after the first ones, 58; of 64 experts 13.4, and 14.3.)
constexpr int router_sm_blocks(int experts) {
    return experts <= 64 ? 6 : experts <= 128 ? 4 : experts <= 256 ? 3 : experts <= 512 ? 2 : 1;
}
constexpr int kRouterClusters = 36;
constexpr int kRouterOneCluster = 2;    // tokens per warp up to which one cluster takes them all
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

// What a warp reads of a token, without waiting for any of it: its logits and
// whether it counts.
template <int N, typename T>
struct Token {
    T v[N];
    uint8_t counted;

    __device__ __forceinline__ void load(const RouterArgs& a, int64_t t) {
        const T* row = static_cast<const T*>(a.logits) + t * a.experts;
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = row[min(lane + 32 * i, a.experts - 1)];
        counted = a.mask ? a.mask[t] : 1;
    }
    __device__ __forceinline__ void get(const RouterArgs& a, float (&x)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = (threadIdx.x & 31) + 32 * i < a.experts ? dev::to_f32(v[i]) : -INFINITY;
    }
};

// The largest of the lanes' values, a NaN if there is one.
__device__ __forceinline__ float lanes_max(float v) {
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// A lane's choice: slot i of the token gets the expert (-1: none) with this logit.
struct Choice {
    int slot, expert;
    float logit;
};

// What a warp needs to choose by.
struct Among {
    unsigned key[32];
    int expert[32];
};

// The K <= 32 largest logits x of a token, whose largest, `top`, is a number.  The
// K-th largest of the lanes' own largest is a bound that K logits reach at least,
// and few more do (with 8 of 256 some 10; equal ones, which leave together, lower
// it): those go to a lane each, which reads the logit again, and are ranked by
// comparing all with all.  False where more than 32 reach it: many equal ones.
template <int N, typename T>
__device__ __forceinline__ bool choose_few(const T* row, const float (&x)[N], float best, float top, int K,
                                           Among& among, Choice& mine) {
    const int lane = threadIdx.x & 31;
    float bound = top;
    for (int k = 1; k < K; ++k) {
        if (best == bound) best = -INFINITY;
        bound = lanes_max(best);
    }
    bound = fmaxf(bound, -FLT_MAX);         // -inf is not to be chosen
    unsigned reach = 0;                     // a bit for each of the lane's logits
#pragma unroll
    for (int i = 0; i < N; ++i) reach |= x[i] >= bound ? 1u << i : 0;
    int total = 0;
    while (const unsigned with = __ballot_sync(kAll, reach)) {
        const int at = total + __popc(with & ((1u << lane) - 1));
        if (reach && at < 32) among.expert[at] = lane + 32 * (__ffs(reach) - 1);
        reach &= reach - 1;
        total += __popc(with);
    }
    if (total > 32) return false;
    __syncwarp();
    const bool here = lane < total;
    mine.expert = here ? among.expert[lane] : -1;
    mine.logit = here ? dev::to_f32(row[mine.expert]) : -INFINITY;
    // A 16-bit logit leaves 13 bits of its order free, and there the expert decides
    // between equal ones.
    constexpr bool kRoom = sizeof(T) == 2;
    constexpr unsigned kFree = 0x1FFF;
    static_assert(kMaxExperts <= kFree + 1);
    unsigned key = order_of(mine.logit);
    if (kRoom) key = (key & ~kFree) | (kFree - mine.expert);
    key = here ? key : 0;
    among.key[lane] = key;
    __syncwarp();
    int before = 0;
#pragma unroll 1                            // some three rounds: unrolled 4% slower
    for (int j = 0; j < total; j += 4) {
        const uint4 other = *reinterpret_cast<const uint4*>(among.key + j);
        if (other.x > key) ++before;
        if (other.y > key) ++before;
        if (other.z > key) ++before;
        if (other.w > key) ++before;
    }
    // slots past the number of those that can be chosen get none
    if (!here) before = lane;
    // all ranks are there once, unless some are equal: those by their expert
    if (!kRoom && __reduce_add_sync(kAll, before) != 31 * 32 / 2)
        for (int j = 0; j < total; ++j) before += here && among.key[j] == key && among.expert[j] < mine.expert;
    __syncwarp();
    mine.slot = before;
    return true;
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

// Sums over a part of the tokens: the probabilities [E], counts [E + 1] (last: the
// tokens), the squared logsumexps.  In the workspace one for each cluster.
__host__ __device__ constexpr int sum_words(int experts) { return 2 * experts + 2; }

// A block's shared memory besides its warps' choices: its sums, and its warps'
// probabilities.  No launch needs more than a kernel may have unasked.
constexpr size_t router_smem(int experts) { return (size_t(kRouterWarps) * experts + sum_words(experts)) * 4; }
static_assert(router_smem(kMaxExperts) + kRouterWarps * sizeof(Among) + 256 <= 48 * 1024);

// Without a z loss squares past fp32, of a token whose logits are all the lowest
// number, do not matter.
__device__ __forceinline__ void put_loss(const RouterArgs& a, float balance, float squares, int tokens) {
    if (!a.loss) return;
    const float n = static_cast<float>(tokens);
    float loss = 0.0f;
    if (tokens > 0) loss = a.balance * a.experts * (balance / (n * a.topk)) / n;
    if (tokens > 0 && a.z != 0.0f) loss += a.z * (squares / n);
    *a.loss = loss;
}

// A cluster's blocks add up their sums through each other's shared memory, each
// some of the experts; a launch of one cluster goes on to the loss, else
// router_join_kernel does.
template <int N, typename T>
__global__ void __launch_bounds__(32 * kRouterWarps, router_sm_blocks(32 * N)) router_kernel(const RouterArgs a) {
    extern __shared__ float smem[];
    float* own = smem;                                                  // [sum_words]: of this block
    int* counts = reinterpret_cast<int*>(own + a.experts);
    float* probs = own + sum_words(a.experts);                          // [warps][E]
    __shared__ float warp_squares[kRouterWarps], warp_balance[kRouterWarps];
    __shared__ float block_balance;
    __shared__ __align__(16) Among among[kRouterWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.experts, K = a.topk;
    const auto cluster = cooperative_groups::this_cluster();
    const int blocks = cluster.num_blocks(), rank = cluster.block_rank();
    dev::pdl_launch_dependents();
    for (int e = tid; e <= E; e += blockDim.x) counts[e] = 0;
    __syncthreads();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    float sums[N] = {};
    float squares = 0.0f;
    int tokens = 0;
    const int64_t step = int64_t(gridDim.x) * kRouterWarps;
    constexpr bool kAhead = N <= 8;         // the next token's loads before this one's work: while registers last
    Token<N, T> next;
    int64_t t = int64_t(blockIdx.x) * kRouterWarps + warp;
    if (kAhead && t < a.tokens) next.load(a, t);
    for (; t < a.tokens; t += step) {
        float x[N];
        if (!kAhead) next.load(a, t);
        next.get(a, x);
        const bool counted = next.counted;
        if (kAhead && t + step < a.tokens) next.load(a, t + step);
        float best = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) best = max_nan(best, x[i]);
        float top = lanes_max(best);
        const bool any = counted && !(top == -INFINITY);
        Choice mine[2] = {{lane, -1, 0.0f}, {lane + 32, -1, 0.0f}};
        // (with a lane's one or two logits there is nothing to leave out first)
        const bool few = N >= 4 && K <= 32 && top == top;
        const T* row = static_cast<const T*>(a.logits) + t * E;
        if (any && !(few && choose_few<N>(row, x, best, top, K, among[warp], mine[0]))) {
            // one after the other
            unsigned key[N];
#pragma unroll
            for (int i = 0; i < N; ++i) key[i] = lane + 32 * i < E ? order_of(x[i]) : 0;
            for (int k = 0; k < K; ++k) {
                unsigned high = key[0];
#pragma unroll
                for (int i = 1; i < N; ++i) high = max(high, key[i]);
                const unsigned most = __reduce_max_sync(kAll, high);
                if (most <= kNever) break;
                unsigned low = 0xFFFFu;     // the lowest of the lane's experts with it
#pragma unroll
                for (int i = N - 1; i >= 0; --i) low = key[i] == most ? lane + 32 * i : low;
                const int e = __reduce_min_sync(kAll, low);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (k == mine[i].slot) {
                        mine[i].expert = e;
                        mine[i].logit = of_order(most);
                    }
#pragma unroll
                for (int i = 0; i < N; ++i) key[i] = e == lane + 32 * i ? 0 : key[i];
            }
        }
        float sum = 1.0f;
        if (any) {
            sum = exponentials(x, top);
            const float lse = top + logf(sum), one = 1.0f / sum;
            squares = fmaf(lse, lse, squares);
            ++tokens;
#pragma unroll
            for (int i = 0; i < N; ++i) sums[i] = fmaf(x[i], one, sums[i]);
        }
        float part[2] = {};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i == 1 && K <= 32) break;
            if (mine[i].expert >= 0 && mine[i].slot < K) part[i] = expf(mine[i].logit - top);
        }
        if (a.normalize && any) sum = dev::warp_sum(part[0] + part[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i == 1 && K <= 32) break;
            if (mine[i].slot >= K) continue;
            a.idx[t * K + mine[i].slot] = mine[i].expert;
            a.weights[t * K + mine[i].slot] = part[i] / sum;
            if (mine[i].expert >= 0) atomicAdd(counts + mine[i].expert, 1);     // integers: any order gives the same
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
    for (int e = tid; e < E; e += blockDim.x) {
        float p = 0.0f;
#pragma unroll
        for (int w = 0; w < kRouterWarps; ++w) p += probs[w * E + e];
        own[e] = p;
    }
    if (tid == 0) {
        float all = 0.0f;
        for (int w = 0; w < kRouterWarps; ++w) all += warp_squares[w];
        own[2 * E + 1] = all;
    }
    cluster.sync();
    // the cluster's sums of the experts rank, rank + blocks, ...
    const bool last = int(gridDim.x) == blocks;
    float* out = static_cast<float*>(a.workspace) + int64_t(blockIdx.x / blocks) * sum_words(E);
    float balance = 0.0f;
    for (int e = rank + blocks * tid; e <= E; e += blocks * blockDim.x) {
        float p = 0.0f;
        int count = 0;
#pragma unroll
        for (int b = 0; b < kRouterCluster; ++b) {
            if (b >= blocks) break;
            const float* other = cluster.map_shared_rank(own, b);
            count += reinterpret_cast<const int*>(other)[E + e];
            p += other[e < E ? e : 2 * E + 1];
        }
        if (e < E) balance = fmaf(static_cast<float>(count), p, balance);
        if (last) {
            a.counts[e] = count;
            if (e == E) {                   // the last one keeps them for the loss
                tokens = count;
                squares = p;
            }
        } else {
            out[e < E ? e : 2 * E + 1] = p;
            reinterpret_cast<int*>(out)[E + e] = count;
        }
    }
    if (last) {
        balance = dev::warp_sum(balance);
        if (lane == 0) warp_balance[warp] = balance;
        __syncthreads();
        if (tid == 0) {
            float all = 0.0f;
            for (int w = 0; w < kRouterWarps; ++w) all += warp_balance[w];
            block_balance = all;
        }
        cluster.sync();
        if (rank == E % blocks && tid == E / blocks % blockDim.x) {
            float all = 0.0f;
            for (int b = 0; b < blocks; ++b) all += *cluster.map_shared_rank(&block_balance, b);
            put_loss(a, all, squares, tokens);
        }
    }
    cluster.sync();      // before a block leaves that others read from
}

// Joins the clusters' sums in a fixed order, a cluster of blocks with some of the
// experts each (one SM alone would take 2 us to read 108 sums of 256 experts): a
// thread takes every `ways`-th of the sums for one expert, kJoinBatch loads at a time.
constexpr int kJoinThreads = 256, kJoinBlocks = 8, kJoinBatch = 8;

__global__ void __launch_bounds__(kJoinThreads) router_join_kernel(const RouterArgs a, int parts) {
    __shared__ float probs[kJoinThreads], warp_sums[kJoinThreads / 32], block_balance;
    __shared__ int counts[kJoinThreads];
    const auto cluster = cooperative_groups::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.experts, words = sum_words(E);
    const int columns = (E + kJoinBlocks) / kJoinBlocks, ways = kJoinThreads / columns;     // 1 (1024 experts) to 256
    const int x = tid % columns, y = tid / columns, e = blockIdx.x * columns + x;
    const float* sums = static_cast<const float*>(a.workspace);
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const bool here = e <= E && y < ways;
    float p = 0.0f;
    int count = 0;
    if (here)
        for (int b0 = y; b0 < parts; b0 += ways * kJoinBatch) {
            float q[kJoinBatch];
            int c[kJoinBatch];
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i) {
                const float* part = sums + min(b0 + i * ways, parts - 1) * words;
                q[i] = dev::load_now(part + (e < E ? e : 2 * E + 1));
                c[i] = dev::load_now(reinterpret_cast<const int*>(part) + E + e);
            }
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i) {
                const bool use = b0 + i * ways < parts;
                p += use ? q[i] : 0.0f;
                count += use ? c[i] : 0;
            }
        }
    probs[tid] = p;
    counts[tid] = count;
    __syncthreads();
    float balance = 0.0f;
    if (here && y == 0) {
        for (int w = 1; w < ways; ++w) {
            p += probs[w * columns + x];
            count += counts[w * columns + x];
        }
        a.counts[e] = count;
        if (e < E) balance = static_cast<float>(count) * p;
    }
    balance = dev::warp_sum(balance);
    if (lane == 0) warp_sums[warp] = balance;
    __syncthreads();
    if (tid == 0) {
        balance = 0.0f;
        for (int w = 0; w < kJoinThreads / 32; ++w) balance += warp_sums[w];
        block_balance = balance;
    }
    cluster.sync();
    if (here && y == 0 && e == E) {          // its count is the tokens', its sum the squares'
        balance = 0.0f;
        for (int b = 0; b < kJoinBlocks; ++b) balance += *cluster.map_shared_rank(&block_balance, b);
        put_loss(a, balance, p, count);
    }
    cluster.sync();      // before a block leaves that another reads from
}

// With p = softmax(logits), A_e = c f_e + (its weight's gradient, where weights are
// probabilities), f_e = counts_e / (n K), c = dloss balance E / n:
//   dlogits_e = p_e (A_e - sum p A + 2 dloss z logsumexp / n)
// and, where weights are a softmax over the chosen experts, w_k (dw_k - sum w dw)
// at those.
//
// The slots' gradients get to the lanes of their experts through shared memory: a
// lane of the K puts its own in the expert's place (K comparisons for each of a lane's
// experts instead: 16384 tokens of 256 21.1 us, so 14.4).
template <int N, typename T>
__global__ void __launch_bounds__(32 * kRouterWarps, router_sm_blocks(32 * N))
    router_backward_kernel(const RouterArgs a) {
    __shared__ int places[kRouterWarps][32 * N];        // zeros between tokens
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.experts, K = a.topk;
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const float n = static_cast<float>(max(a.counts[E], 1)), dloss = a.dloss ? *a.dloss : 0.0f;
    const float z = 2.0f * a.z * dloss / n;
    int* const place = places[warp];
    float load[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        place[lane + 32 * i] = 0;
        const int e = lane + 32 * i;
        load[i] = e < E ? a.balance * dloss * E / n * (a.counts[e] / (n * K)) : 0.0f;
    }
    for (int64_t t = int64_t(blockIdx.x) * kRouterWarps + warp; t < a.tokens; t += int64_t(gridDim.x) * kRouterWarps) {
        T* out = static_cast<T*>(a.dlogits) + t * E;
        Token<N, T> token;
        token.load(a, t);
        int chosen[2];
        float dw[2], w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = lane + 32 * i;
            const bool here = a.dweights && k < K;
            chosen[i] = here ? a.idx[t * K + k] : -1;
            dw[i] = here ? a.dweights[t * K + k] : 0.0f;
        }
        float x[N], g[N] = {}, each[N];
        token.get(a, x);
        float top = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) top = max_nan(top, x[i]);
        top = lanes_max(top);                    // with a NaN all of the token's gradients are
        if (!token.counted || top == -INFINITY) {             // padding
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (lane + 32 * i < E) dev::from_f32(out[lane + 32 * i], 0.0f);
            continue;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (chosen[i] < 0 || chosen[i] >= E) {
                chosen[i] = -1;
                dw[i] = 0.0f;
            }
#pragma unroll
        for (int i = 0; i < N; ++i) each[i] = load[i];
        if (a.normalize) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                w[i] = 0.0f;
                if (i == 1 && K <= 32) break;
                if (chosen[i] >= 0)
                    w[i] = expf(dev::to_f32(static_cast<const T*>(a.logits)[t * E + chosen[i]]) - top);
            }
            const float sum = dev::warp_sum(w[0] + w[1]);
            const float dot = dev::warp_sum(w[0] * dw[0] + w[1] * dw[1]) / sum;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i == 1 && K <= 32) break;
                dw[i] = w[i] / sum * (dw[i] - dot);
            }
        }
        const bool has = chosen[0] >= 0;
        bool one_by_one = K > 32;
        if (a.dweights && !one_by_one) {
            __syncwarp();
            if (has) place[chosen[0]] = lane;
            __syncwarp();
            one_by_one = __any_sync(kAll, has && place[chosen[0]] != lane);     // an expert twice
            if (has) place[chosen[0]] = one_by_one ? 0 : __float_as_int(dw[0]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float d = __int_as_float(place[lane + 32 * i]);
                if (a.normalize) g[i] = d;
                else each[i] += d;
            }
            __syncwarp();
            if (has) place[chosen[0]] = 0;
        }
        if (a.dweights && one_by_one)
            for (int k = 0; k < K; ++k) {
                const int e = __shfl_sync(kAll, k < 32 ? chosen[0] : chosen[1], k & 31);
                const float d = __shfl_sync(kAll, k < 32 ? dw[0] : dw[1], k & 31);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (e == lane + 32 * i) {
                        if (a.normalize) g[i] += d;
                        else each[i] += d;
                    }
            }
        const float sum = exponentials(x, top);
        const float lse = top + logf(sum), one = 1.0f / sum;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] *= one;
            dot = fmaf(x[i], each[i], dot);
        }
        dot = dev::warp_sum(dot);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 32 * i < E)
                dev::from_f32(out[lane + 32 * i], fmaf(x[i], each[i] - dot + z * lse, g[i]));
    }
}

// Blocks of a launch; up to kRouterCluster of them are one cluster.
int router_blocks(int64_t tokens, int experts) {
    const int64_t blocks = std::max<int64_t>(1, (tokens + kRouterWarps - 1) / kRouterWarps);
    if (blocks <= kRouterCluster) return static_cast<int>(blocks);
    if (blocks <= kRouterCluster * kRouterOneCluster) return kRouterCluster;
    return static_cast<int>(std::min<int64_t>(kRouterClusters * router_sm_blocks(experts),
                                              (blocks + kRouterCluster - 1) / kRouterCluster)) * kRouterCluster;
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

size_t router_workspace(int64_t tokens, int experts) {
    const int blocks = router_blocks(tokens, experts);
    return blocks > kRouterCluster ? size_t(blocks / kRouterCluster) * sum_words(experts) * 4 : 0;
}

cudaError_t launch_router(const RouterArgs& a, int dtype, cudaStream_t stream) {
    const int blocks = router_blocks(a.tokens, a.experts), parts = blocks / kRouterCluster;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(32 * kRouterWarps);
    cfg.dynamicSmemBytes = router_smem(a.experts);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = std::min(blocks, kRouterCluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = by_experts<Forward>(a.experts, dtype, [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, a); });
    if (e != cudaSuccess || parts <= 1) return e;
    cfg.gridDim = dim3(kJoinBlocks);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    attr[1].val.clusterDim.x = kJoinBlocks;
    return cudaLaunchKernelEx(&cfg, router_join_kernel, a, parts);
}

cudaError_t launch_router_backward(const RouterArgs& a, int dtype, cudaStream_t stream) {
    const int64_t blocks = std::min<int64_t>((a.tokens + kRouterWarps - 1) / kRouterWarps,
                                             int64_t(sm_count()) * router_sm_blocks(a.experts));
    return by_experts<Backward>(a.experts, dtype, [&](auto kernel) {
        return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(32 * kRouterWarps), 0, stream, a);
    });
}

}  // namespace ct
