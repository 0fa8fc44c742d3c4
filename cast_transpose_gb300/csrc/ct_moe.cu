// ct_moe.cu -- tokens sorted by expert and back: the stable counting sort of
// the router's choices, the row movement into expert order and back, and its
// gradients.
#include "ct_device.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"

#include <algorithm>
#include <atomic>
#include <cooperative_groups.h>

namespace ct {
namespace {

using dev::pdl_launch_dependents;
using dev::pdl_wait;

// ---- sort ------------------------------------------------------------------
// Stable counting sort of n slots by expert.  The slots are cut into one
// contiguous run per block and one per warp, so that the rank of a slot among
// its expert's is (slots of earlier blocks) + (of earlier warps) + (earlier in
// the warp's run): the first two are exclusive sums of counts, the third is
// counted on the way, 32 slots at a time, from the lanes with the same expert.
// Integers only; no order depends on atomics.  What it moves is small (12 bytes a slot); the
// time is latency, so blocks learn each other's counts in the cheapest way
// their number allows:
//   kOne      one block, up to kSortOneBlock slots
//   kCluster  one cluster of kSortCluster blocks, counts read from its other
//             blocks' shared memory: still one launch
//   kGrid     a first launch leaves every block's counts in the workspace
enum SortMode { kOne, kCluster, kGrid };
constexpr int kSortMaxThreads = 1024;
constexpr int kSortCluster = 8;
constexpr int kSortBatch = 4;         // groups of 32 slots loaded ahead of their counting

__device__ __forceinline__ int expert_of(const SortArgs& a, int64_t s) {
    const int64_t e = a.index64 ? static_cast<const int64_t*>(a.idx)[s]
                                : static_cast<const int32_t*>(a.idx)[s];
    return e >= 0 && e < a.experts ? static_cast<int>(e) : -1;
}

// The lanes with the same expert, from one ballot per bit of its number
// (__match_any_sync gives the same, but a warp of 32 different experts held
// the SM for some 50 cycles: a cluster's 32768 slots of 64 experts 12.8 us, so:
// 10.4).
__device__ __forceinline__ unsigned same_expert(int e, int bits) {
    const unsigned some = __ballot_sync(0xFFFFFFFFu, e >= 0);
    unsigned same = e >= 0 ? some : ~some;
    for (int i = 0; i < bits; ++i) {
        const bool bit = (e >> i) & 1;
        const unsigned set = __ballot_sync(0xFFFFFFFFu, bit);
        same &= bit ? set : ~set;
    }
    return same;
}

// Calls f(slot, expert, lanes of the same expert) for the slots [lo, hi) of a
// warp, 32 at a time in order; lanes past hi get expert -1.
template <typename F>
__device__ __forceinline__ void walk(const SortArgs& a, int64_t lo, int64_t hi, F&& f) {
    const int lane = threadIdx.x & 31;
    for (int64_t s0 = lo; s0 < hi; s0 += 32 * kSortBatch) {
        int e[kSortBatch];
#pragma unroll
        for (int i = 0; i < kSortBatch; ++i) {
            const int64_t s = s0 + 32 * i + lane;
            e[i] = s < hi ? expert_of(a, s) : -1;
        }
#pragma unroll
        for (int i = 0; i < kSortBatch; ++i) {
            if (s0 + 32 * i >= hi) break;
            f(s0 + 32 * i + lane, e[i], same_expert(e[i], a.expert_bits));
            __syncwarp();
        }
    }
}

// The run of this warp.
__device__ __forceinline__ void run_of(const SortArgs& a, int64_t& lo, int64_t& hi) {
    const int64_t warps = blockDim.x >> 5, runs = gridDim.x * warps;
    const int64_t len = ((a.n + runs - 1) / runs + 31) / 32 * 32;
    lo = min(a.n, len * (blockIdx.x * warps + (threadIdx.x >> 5)));
    hi = min(a.n, lo + len);
}

// hist[e][warp]: the slots of each warp's run by expert; a row is one entry
// longer than the warps, so that neither a warp's nor an expert's entries share
// a bank.
__device__ __forceinline__ int hist_row() { return static_cast<int>(blockDim.x >> 5) + 1; }

__device__ __forceinline__ void count_run(const SortArgs& a, int* hist, int64_t lo, int64_t hi) {
    const int row = hist_row();
    for (int i = threadIdx.x; i < row * a.experts; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    int* mine = hist + (threadIdx.x >> 5);
    walk(a, lo, hi, [&](int64_t, int e, unsigned same) {
        if (e >= 0 && int(threadIdx.x & 31) == __ffs(same) - 1) mine[e * row] += __popc(same);
    });
    __syncthreads();
}

// Makes hist[e][warp] the slots of earlier warps, and count[e] those of all
// the block's: a thread per expert in a small block, else a warp per expert
// and a lane per warp (16 slots of 64 experts in 4 warps: 3.5 us against 5.2;
// 1024 in 32: 7.5 against 6.5).
__device__ __forceinline__ void scan_warps(const SortArgs& a, int* hist, int* count) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, row = hist_row();
    if (warps <= 8) {
        for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
            int sum = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w)
                if (w < warps) {
                    const int c = hist[e * row + w];
                    hist[e * row + w] = sum;
                    sum += c;
                }
            count[e] = sum;
        }
        __syncthreads();
        return;
    }
    for (int e = threadIdx.x >> 5; e < a.experts; e += warps) {
        int* entry = hist + e * row + lane;
        const int c = lane < warps ? *entry : 0;
        int sum = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += up;
        }
        if (lane < warps) *entry = sum - c;
        if (lane == 31) count[e] = sum;
    }
    __syncthreads();
}

// Counts of every block's run, block_counts[block][E], for kGrid.
__global__ void __launch_bounds__(kSortMaxThreads) moe_count_kernel(SortArgs a, int* block_counts) {
    extern __shared__ int smem[];
    pdl_launch_dependents();
    pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    int64_t lo, hi;
    run_of(a, lo, hi);
    int* count = smem + hist_row() * a.experts;
    count_run(a, smem, lo, hi);
    scan_warps(a, smem, count);
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x)
        block_counts[int64_t(blockIdx.x) * a.experts + e] = count[e];
}

// Ints of dynamic shared memory: the warps' counts, then per expert the block's
// own count, the sums below, its first row (and the end).
__host__ __device__ constexpr int sort_ints(int warps, int experts) {
    return (warps + 5) * experts + 1;
}

template <SortMode MODE>
__global__ void __launch_bounds__(kSortMaxThreads)
    moe_sort_kernel(SortArgs a, const int* block_counts) {
    extern __shared__ int smem[];
    __shared__ int64_t warp_sums[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, E = a.experts;
    const int threads = blockDim.x, warps = threads >> 5, row_len = hist_row();
    const int b = blockIdx.x, blocks = gridDim.x;
    int* hist = smem;                   // [E][warps + 1]
    int* own = hist + row_len * E;      // [E]: slots of this block
    int* before = own + E;              // [E]: of earlier blocks
    int* total = before + E;            // [E]: of all blocks
    int* first = total + E;             // [E + 1]: first row
    pdl_launch_dependents();
    pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    int64_t lo, hi;
    run_of(a, lo, hi);
    count_run(a, hist, lo, hi);
    scan_warps(a, hist, own);
    if constexpr (MODE == kOne) {
        before = nullptr;
        total = own;
    } else if constexpr (MODE == kCluster) {
        const auto cluster = cooperative_groups::this_cluster();
        cluster.sync();
        for (int e = tid; e < E; e += threads) {
            int c[kSortCluster], earlier = 0, all = 0;
#pragma unroll
            for (int o = 0; o < kSortCluster; ++o) c[o] = cluster.map_shared_rank(own, o)[e];
#pragma unroll
            for (int o = 0; o < kSortCluster; ++o) {
                earlier += o < b ? c[o] : 0;
                all += c[o];
            }
            before[e] = earlier;
            total[e] = all;
        }
        // done with the other blocks' counts; waited for at the end, so that no
        // block leaves while another may still read its
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    } else {
        for (int e = tid; e < E; e += threads) before[e] = total[e] = 0;
        __syncthreads();
        // `parts` threads per expert, each over a share of the blocks
        const int parts = max(1, threads / E), share = (blocks + parts - 1) / parts;
        for (int i = tid; i < parts * E; i += threads) {
            const int e = i % E, o0 = i / E * share, o1 = min(blocks, o0 + share);
            int earlier = 0, all = 0;
#pragma unroll 16
            for (int o = o0; o < o1; ++o) {
                const int c = block_counts[int64_t(o) * E + e];
                all += c;
                earlier += o < b ? c : 0;
            }
            atomicAdd(&before[e], earlier);   // integers: any order gives the same
            atomicAdd(&total[e], all);
        }
    }
    __syncthreads();
    // first rows: the exclusive sum of the padded totals in expert order
    auto inclusive = [&](int64_t v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += up;
        }
        return v;
    };
    int64_t base = 0;
    for (int e0 = 0; e0 < E; e0 += threads) {
        const int e = e0 + tid;
        const int64_t padded = e < E ? (int64_t(total[e]) + a.align - 1) / a.align * a.align : 0;
        const int64_t sum = inclusive(padded);
        if (lane == 31) warp_sums[warp] = sum;
        __syncthreads();
        const int64_t sums = inclusive(lane < warps ? warp_sums[lane] : 0);
        const int64_t earlier = __shfl_sync(0xFFFFFFFFu, sums, warp > 0 ? warp - 1 : 0);
        if (e < E) first[e] = static_cast<int>(min(base + (warp > 0 ? earlier : 0) + sum - padded, a.rows));
        base += __shfl_sync(0xFFFFFFFFu, sums, 31);
        __syncthreads();
    }
    const int end = static_cast<int>(min(base, a.rows));
    if (tid == 0) first[E] = end;
    __syncthreads();
    walk(a, lo, hi, [&](int64_t s, int e, unsigned same) {
        int* mine = hist + e * row_len + warp;
        int64_t row = -1;
        if (e >= 0) {
            row = int64_t(first[e]) + *mine + (MODE == kOne ? 0 : before[e]) +
                  __popc(same & ((1u << lane) - 1));
            if (row >= a.rows) row = -1;
        }
        if (s < hi) a.row_of[s] = static_cast<int>(row);
        if (row >= 0) a.src[row] = static_cast<int>(s);
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) *mine += __popc(same);
    });
    if (b == 0) {
        for (int e = tid; e <= E; e += threads) a.offsets[e] = first[e];
        for (int e = tid; e < E; e += threads) a.counts[e] = total[e];
    }
    // padding rows: a warp per expert, then the rows after the last expert
    for (int e = b * warps + warp; e < E; e += blocks * warps)
        for (int64_t r = int64_t(first[e]) + total[e] + lane; r < first[e + 1]; r += 32) a.src[r] = -1;
    for (int64_t r = int64_t(end) + b * threads + tid; r < a.rows; r += int64_t(blocks) * threads)
        a.src[r] = -1;
    if constexpr (MODE == kCluster) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// ---- row movement ----------------------------------------------------------
// One block per token: its row is read once and written to its K places, or
// gathered from them, so that neither order's rows move twice; several slots'
// loads or stores of a thread are in flight at a time.  Bound by HBM; measured,
// bf16, of the measured copy rate: dispatch 8191x4x6144 75.7 us (515 MB, 1.0),
// combine 8192x8x4096 86.6 us (605 MB, 1.03), its gradient 8192x4x6144 142 us
// (918 MB, 0.95), dispatch's gradient 8192x4x6144 72.4 us (503 MB, 1.02).
constexpr int kMaxSlots = 64;         // K at most
constexpr int kMoveThreads = 256;

// The sorted row of each of token t's slots, -1 where dropped or out of range.
__device__ __forceinline__ void token_rows(const MoveArgs& a, int64_t t, int (&rows)[kMaxSlots]) {
    if (threadIdx.x < 32)
        for (int k = threadIdx.x; k < a.topk; k += 32) {
            const int r = a.row_of[t * a.topk + k];
            rows[k] = r >= 0 && r < a.rows ? r : -1;
        }
    __syncthreads();
}

// A launch that writes sorted rows has blocks for the padding rows before
// those of the tokens: each looks at kPadRows rows, a lane each, and clears the
// ones without a slot.
static_assert(kPadRows == 32, "a lane looks at a row");

template <typename W>
__device__ void clear_padding(const MoveArgs& a, int64_t words) {
    const int64_t row0 = int64_t(blockIdx.x) * kPadRows, row = row0 + (threadIdx.x & 31);
    bool empty = false;
    if (row < a.rows) {
        const int s = a.src[row];
        empty = s < 0 || s >= a.tokens * a.topk;
    }
    for (unsigned left = __ballot_sync(0xFFFFFFFFu, empty); left; left &= left - 1) {
        W* out = static_cast<W*>(a.sorted) + (row0 + __ffs(left) - 1) * words;
        for (int64_t c = threadIdx.x; c < words; c += blockDim.x) out[c] = W{};
    }
}

// What the first blocks of a dispatch ask to have in L2 while they wait for the
// kernel before, as a rule the sort, which leaves HBM idle for its 4 to 15 us:
// the rows of x that are moved first.  A hint: whatever is written to x
// meanwhile is written in L2 too.  A call with a noop flag does not ask.
//   8191x4x6144 with its sort: 89.3 us without, 85.3 with 24 MB, 85.8 with 48.
constexpr int64_t kPrefetchBytes = int64_t(24) << 20;
constexpr int kPrefetchBlocks = 608;

struct Prefetch {
    const uint8_t* from;
    int64_t bytes;          // a multiple of 16
    int blocks;
    static constexpr uint32_t kPiece = 4096;

    __device__ __forceinline__ void issue() const {
        if (blockIdx.x >= blocks) return;
        for (int64_t at = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * kPiece; at < bytes;
             at += int64_t(blocks) * blockDim.x * kPiece)
            dev::prefetch_l2_bulk(from + at, static_cast<uint32_t>(min(int64_t(kPiece), bytes - at)));
    }
};

// W: the word that rows are moved in.  kMoveWords loads of a thread are in
// flight at a time.
constexpr int kMoveWords = 4;

template <typename W>
__global__ void __launch_bounds__(kMoveThreads)
    moe_dispatch_kernel(MoveArgs a, int pad_blocks, Prefetch ahead) {
    __shared__ int rows[kMaxSlots];
    pdl_launch_dependents();
    ahead.issue();
    pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int words = static_cast<int>(a.hidden * a.elem_bytes / sizeof(W));
    if (blockIdx.x < pad_blocks) {
        clear_padding<W>(a, words);
        return;
    }
    const int64_t t = blockIdx.x - pad_blocks;
    token_rows(a, t, rows);
    const W* x = static_cast<const W*>(a.x) + t * words;
    for (int c0 = threadIdx.x; c0 < words; c0 += kMoveWords * blockDim.x) {
        W v[kMoveWords];
#pragma unroll
        for (int i = 0; i < kMoveWords; ++i) {
            const int c = c0 + i * blockDim.x;
            if (c < words) v[i] = __ldcs(x + c);
        }
        for (int k = 0; k < a.topk; ++k) {
            if (rows[k] < 0) continue;
            W* out = static_cast<W*>(a.sorted) + int64_t(rows[k]) * words;
#pragma unroll
            for (int i = 0; i < kMoveWords; ++i) {
                const int c = c0 + i * blockDim.x;
                if (c < words) __stcs(out + c, v[i]);
            }
        }
    }
}

// Slots handled together, so that their rows' loads are in flight at once.
constexpr int kSlotGroup = 4;

// Calls f(cols) for the block's threads' groups of eight columns.
template <int G, typename F>
__device__ __forceinline__ void each_cols(int H, F&& f) {
    for (int v = threadIdx.x;; v += blockDim.x) {
        const dev::Cols<G> cols(v, H);
        if (!cols.any()) break;      // later items begin later
        f(cols);
    }
}

template <typename T, int G>
__global__ void __launch_bounds__(kMoveThreads) moe_combine_kernel(MoveArgs a) {
    __shared__ int rows[kMaxSlots];
    pdl_launch_dependents();
    pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int64_t t = blockIdx.x;
    const T* ys = static_cast<const T*>(a.ys);
    const float* weights = a.weights ? a.weights + t * a.topk : nullptr;
    token_rows(a, t, rows);
    each_cols<G>(static_cast<int>(a.hidden), [&](const dev::Cols<G>& cols) {
        float sum[8] = {};
        for (int k0 = 0; k0 < a.topk; k0 += kSlotGroup) {
            float f[kSlotGroup][8], w[kSlotGroup];
#pragma unroll
            for (int i = 0; i < kSlotGroup; ++i) {
                const int r = k0 + i < a.topk ? rows[k0 + i] : -1;
                // a slot that is dropped takes no part, whatever its weight
                w[i] = r >= 0 ? (weights ? weights[k0 + i] : 1.0f) : 0.0f;
                if (r >= 0) {
                    dev::load_cols<G>(ys + r * a.hidden, cols, f[i]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[i][j] = 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < kSlotGroup; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] = fmaf(w[i], f[i][j], sum[j]);
        }
        dev::store_cols<G>(static_cast<T*>(a.out) + t * a.hidden, cols, sum);
    });
}

template <typename T, int G>
__global__ void __launch_bounds__(kMoveThreads) moe_combine_backward_kernel(MoveArgs a, int pad_blocks) {
    __shared__ int rows[kMaxSlots];
    __shared__ float4 slots[2][kMoveThreads / 32];
    static_assert(kSlotGroup == 4, "the sums of a group travel as a float4");
    pdl_launch_dependents();
    pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int H = static_cast<int>(a.hidden);
    if (blockIdx.x < pad_blocks) {
        if constexpr (G == 8)
            clear_padding<uint4>(a, a.hidden * sizeof(T) / 16);
        else
            clear_padding<T>(a, H);
        return;
    }
    const int64_t t = blockIdx.x - pad_blocks;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const T* dout = static_cast<const T*>(a.x) + t * a.hidden;
    const T* ys = static_cast<const T*>(a.ys);
    T* dys = static_cast<T*>(a.sorted);
    token_rows(a, t, rows);
    for (int k0 = 0; k0 < a.topk; k0 += kSlotGroup) {
        int r[kSlotGroup];
        float w[kSlotGroup], dot[kSlotGroup] = {};
#pragma unroll
        for (int i = 0; i < kSlotGroup; ++i) {
            r[i] = k0 + i < a.topk ? rows[k0 + i] : -1;
            w[i] = dys && r[i] >= 0 ? a.weights[t * a.topk + k0 + i] : 0.0f;
        }
        each_cols<G>(H, [&](const dev::Cols<G>& cols) {
            float g[8], f[kSlotGroup][8];
            dev::load_cols<G>(dout, cols, g);
            if (a.dweights) {
#pragma unroll
                for (int i = 0; i < kSlotGroup; ++i) {
                    if (r[i] >= 0) {
                        dev::load_cols<G>(ys + r[i] * a.hidden, cols, f[i]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[i][j] = 0.0f;
                    }
                }
#pragma unroll
                for (int i = 0; i < kSlotGroup; ++i)
                    if (r[i] >= 0) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) dot[i] = fmaf(g[j], f[i][j], dot[i]);
                    }
            }
            if (dys) {
#pragma unroll
                for (int i = 0; i < kSlotGroup; ++i) {
                    if (r[i] < 0) continue;
                    float d[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] = w[i] * g[j];
                    dev::store_cols<G>(dys + r[i] * a.hidden, cols, d);
                }
            }
        });
        if (!a.dweights) continue;
#pragma unroll
        for (int i = 0; i < kSlotGroup; ++i) dot[i] = dev::warp_sum(dot[i]);
        float4* half = slots[(k0 / kSlotGroup) & 1];
        if (lane == 0) half[warp] = make_float4(dot[0], dot[1], dot[2], dot[3]);
        __syncthreads();
        if (threadIdx.x < kSlotGroup && k0 + threadIdx.x < a.topk) {
            float sum = 0.0f;
            for (int i = 0; i < warps; ++i) sum += reinterpret_cast<const float*>(half + i)[threadIdx.x];
            a.dweights[t * a.topk + k0 + threadIdx.x] = sum;
        }
    }
}

// Whether rows and buffers allow accesses of `bytes`.
bool allow(const MoveArgs& a, int bytes) {
    auto ok = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    return a.hidden * a.elem_bytes % bytes == 0 && ok(a.x) && ok(a.ys) && ok(a.sorted) && ok(a.out);
}

bool vectors(const MoveArgs& a) { return a.hidden % 8 == 0 && allow(a, 16); }

// The kernel for the widest groups of columns that rows and buffers allow.
#define CT_BY_GROUP(kernel, T) \
    (vectors(a) ? kernel<T, 8> : allow(a, 2 * sizeof(T)) ? kernel<T, 2> : kernel<T, 1>)

int pad_blocks(const MoveArgs& a) { return static_cast<int>(a.sorted ? ct::pad_blocks(a.rows) : 0); }

// Threads of a block whose rows have `groups` words or groups of columns.
dim3 move_threads(int64_t groups, int per_thread) {
    const int64_t t = (groups + per_thread - 1) / per_thread;
    return dim3(static_cast<unsigned>(std::min<int64_t>(kMoveThreads, std::max<int64_t>(32, (t + 31) / 32 * 32))));
}

template <typename F>
cudaError_t by_type(int dtype, F&& f) {
    if (dtype == 0) return f(__nv_bfloat16{});
    if (dtype == 1) return f(__half{});
    return f(float{});
}

}  // namespace

// Measured, us (64 experts): 4096 slots in one block 9.3, in a cluster 6.7, in
// a grid 9.1; 16384: -, 8.0, 9.3; 32768: -, 10.4, 9.8; 65536: -, 15.6, 10.5.
constexpr int64_t kSortOneBlock = 1024, kSortClusterMost = 24576;
constexpr int64_t kSortBlockSlots = 1024, kSortMaxBlocks = 128;

static SortMode sort_mode(int64_t n) {
    return n <= kSortOneBlock ? kOne : n <= kSortClusterMost ? kCluster : kGrid;
}

static int grid_blocks(int64_t n) {
    return static_cast<int>(std::min(kSortMaxBlocks, (n + kSortBlockSlots - 1) / kSortBlockSlots));
}

// The most a sort's kernel ever asks for is allowed once per kernel and device:
// the limit belongs to the kernel, so one that followed each call's need could
// be lowered by another host thread between a call's setting and its launch.
static cudaError_t allow_sort_smem(const void* kernel, std::atomic<uint64_t>& allowed) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;   // beyond 64: every time
    if (allowed.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    constexpr int most = sizeof(int) * sort_ints(kSortMaxThreads / 32, kMaxExperts);
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

size_t sort_workspace(int64_t n, int experts) {
    if (sort_mode(n) != kGrid) return 0;
    return (sizeof(int) * grid_blocks(n) * size_t(experts) + 15) / 16 * 16;
}

cudaError_t launch_moe_sort(const SortArgs& a, void* workspace, cudaStream_t stream) {
    const SortMode mode = sort_mode(a.n);
    const int64_t most = std::max<int64_t>(a.n, a.experts);
    const int threads = mode != kOne ? kSortMaxThreads
                        : static_cast<int>(std::min<int64_t>(kSortMaxThreads, std::max<int64_t>(
                                                                 128, (most + 31) / 32 * 32)));
    const size_t smem = sizeof(int) * sort_ints(threads / 32, a.experts);
    static std::atomic<uint64_t> allowed[4];   // by mode, and the counting kernel's
    auto prepare = [&](auto* kernel, int which) {
        return smem <= 47 * 1024 ? cudaSuccess   // 48 KB with the static part
                                 : allow_sort_smem(reinterpret_cast<const void*>(kernel), allowed[which]);
    };
    cudaError_t e;
    if (mode == kOne) {
        e = prepare(moe_sort_kernel<kOne>, kOne);
        if (e != cudaSuccess) return e;
        return launch_pdl(moe_sort_kernel<kOne>, dim3(1), dim3(threads), smem, stream, a,
                          static_cast<const int*>(nullptr));
    }
    if (mode == kCluster) {
        e = prepare(moe_sort_kernel<kCluster>, kCluster);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kSortCluster);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = kSortCluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, moe_sort_kernel<kCluster>, a,
                                  static_cast<const int*>(nullptr));
    }
    e = prepare(moe_sort_kernel<kGrid>, kGrid);
    if (e == cudaSuccess) e = prepare(moe_count_kernel, 3);
    if (e != cudaSuccess) return e;
    const dim3 blocks(grid_blocks(a.n));
    int* block_counts = static_cast<int*>(workspace);
    e = launch_pdl(moe_count_kernel, blocks, dim3(threads), smem, stream, a, block_counts);
    if (e != cudaSuccess) return e;
    return launch_pdl(moe_sort_kernel<kGrid>, blocks, dim3(threads), smem, stream, a,
                      static_cast<const int*>(block_counts));
}

cudaError_t launch_moe_dispatch(const MoveArgs& a, cudaStream_t stream) {
    const int pad = pad_blocks(a);
    const int64_t bytes = a.tokens * a.hidden * a.elem_bytes;
    const Prefetch ahead = {static_cast<const uint8_t*>(a.x), std::min(bytes, kPrefetchBytes),
                            vectors(a) && !a.noop ? kPrefetchBlocks : 0};
    auto go = [&](auto w) {
        using W = decltype(w);
        return launch_pdl(moe_dispatch_kernel<W>, dim3(static_cast<unsigned>(a.tokens + pad)),
                          move_threads(a.hidden * a.elem_bytes / int64_t(sizeof(W)), 3), 0, stream, a, pad,
                          ahead);
    };
    if (vectors(a)) return go(uint4{});
    if (allow(a, 8)) return go(uint2{});
    return allow(a, 4) ? go(uint32_t{}) : go(uint16_t{});
}

cudaError_t launch_moe_combine(const MoveArgs& a, int dtype, cudaStream_t stream) {
    return by_type(dtype, [&](auto z) {
        using T = decltype(z);
        auto* kernel = CT_BY_GROUP(moe_combine_kernel, T);
        return launch_pdl(kernel, dim3(static_cast<unsigned>(a.tokens)),
                          move_threads((a.hidden + 7) / 8, 1), 0, stream, a);
    });
}

cudaError_t launch_moe_combine_backward(const MoveArgs& a, int dtype, cudaStream_t stream) {
    const int pad = pad_blocks(a);
    return by_type(dtype, [&](auto z) {
        using T = decltype(z);
        auto* kernel = CT_BY_GROUP(moe_combine_backward_kernel, T);
        return launch_pdl(kernel, dim3(static_cast<unsigned>(a.tokens + pad)),
                          move_threads((a.hidden + 7) / 8, 1), 0, stream, a, pad);
    });
}

}  // namespace ct
