// ct_moe.cu -- tokens sorted by expert and back: the stable counting sort of
// the router's choices, the row movement into expert order and back, and its
// gradients.
#include "ct_device.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"

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

__device__ __forceinline__ int expert_of(const SortArgs& a, int64_t s) {
    const int64_t e = a.index64 ? static_cast<const int64_t*>(a.idx)[s]
                                : static_cast<const int32_t*>(a.idx)[s];
    return e >= 0 && e < a.experts ? static_cast<int>(e) : -1;
}

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;

// One block: hist is [kSortWarps][E] in shared memory.
__global__ void __launch_bounds__(kSortThreads) moe_sort_kernel(SortArgs a) {
    extern __shared__ int smem[];
    int* hist = smem;
    int* first = smem + kSortWarps * a.experts;   // [E]: first row of the expert
    pdl_launch_dependents();
    pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, E = a.experts;
    const int64_t per_warp = ((a.n + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int64_t lo = per_warp * warp, hi = min(a.n, lo + per_warp);
    for (int i = tid; i < kSortWarps * E; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    int* mine = hist + warp * E;
    for (int64_t s0 = lo; s0 < hi; s0 += 32) {
        const int e = s0 + lane < hi ? expert_of(a, s0 + lane) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // counts per expert, padded, and their exclusive sum in expert order
    int64_t base = 0;
    for (int e0 = 0; e0 < E; e0 += kSortThreads) {
        const int e = e0 + tid;
        int count = 0;
        if (e < E)
            for (int w = 0; w < kSortWarps; ++w) {
                const int c = hist[w * E + e];
                hist[w * E + e] = count;
                count += c;
            }
        const int padded = static_cast<int>((int64_t(count) + a.align - 1) / a.align * a.align);
        int64_t sum = padded;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += up;
        }
        __shared__ int64_t warp_sums[kSortWarps];
        if (lane == 31) warp_sums[warp] = sum;
        __syncthreads();
        int64_t before = base, all = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            if (w < warp) before += warp_sums[w];
            all += warp_sums[w];
        }
        const int64_t begin = before + sum - padded;
        if (e < E) {
            first[e] = static_cast<int>(min(begin, a.rows));
            a.offsets[e] = first[e];
            a.counts[e] = count;
            // padding rows of this expert
            const int64_t end = min(begin + padded, a.rows);
            for (int64_t r = begin + count; r < end; ++r) a.src[r] = -1;
        }
        base += all;
        __syncthreads();
    }
    const int64_t end = min(base, a.rows);
    if (tid == 0) a.offsets[E] = static_cast<int>(end);
    for (int64_t r = end + tid; r < a.rows; r += kSortThreads) a.src[r] = -1;
    for (int64_t s0 = lo; s0 < hi; s0 += 32) {
        const int64_t s = s0 + lane;
        const int e = s < hi ? expert_of(a, s) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
        if (s < hi) {
            int64_t row = -1;
            if (e >= 0) {
                row = int64_t(first[e]) + mine[e] + __popc(same & ((1u << lane) - 1));
                if (row >= a.rows) row = -1;
            }
            a.row_of[s] = static_cast<int>(row);
            if (row >= 0) a.src[row] = static_cast<int>(s);
        }
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
}

// ---- row movement ----------------------------------------------------------
__device__ __forceinline__ int64_t row_at(const MoveArgs& a, int64_t slot) {
    const int r = a.row_of[slot];
    return r >= 0 && r < a.rows ? r : -1;
}

// W: the word that rows are moved in (their bytes are a multiple of it).
// Blocks 0 .. T-1 copy their token's row to its K places; the others look
// for padding rows, 32 rows to a block, and clear them.
constexpr int kMoveThreads = 256;
constexpr int kPadRows = 32;

template <typename W>
__device__ void clear_padding(const MoveArgs& a, int64_t block, int words) {
    const int64_t r0 = block * kPadRows;
    for (int i = 0; i < kPadRows && r0 + i < a.rows; ++i) {
        const int s = a.src[r0 + i];
        if (s >= 0 && s < a.tokens * a.topk) continue;
        W* row = static_cast<W*>(a.sorted) + (r0 + i) * words;
        for (int c = threadIdx.x; c < words; c += blockDim.x) row[c] = W{};
    }
}

template <typename W>
__global__ void __launch_bounds__(kMoveThreads) moe_dispatch_kernel(MoveArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int words = static_cast<int>(a.hidden * a.elem_bytes / sizeof(W));
    const int64_t t = blockIdx.x;
    if (t >= a.tokens) {
        clear_padding<W>(a, t - a.tokens, words);
        return;
    }
    const W* x = static_cast<const W*>(a.x) + t * words;
    W* out = static_cast<W*>(a.sorted);
    for (int c = threadIdx.x; c < words; c += kMoveThreads) {
        const W v = x[c];
        for (int k = 0; k < a.topk; ++k) {
            const int64_t r = row_at(a, t * a.topk + k);
            if (r >= 0) out[r * words + c] = v;
        }
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kMoveThreads) moe_combine_kernel(MoveArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int64_t t = blockIdx.x;
    const int H = static_cast<int>(a.hidden);
    const T* ys = static_cast<const T*>(a.ys);
    for (int v = threadIdx.x; v * 8 < H + 8 * kMoveThreads; v += kMoveThreads) {
        const dev::Cols<VEC> cols(v, kMoveThreads, H);
        if (!cols.any()) continue;
        float sum[8] = {};
        for (int k = 0; k < a.topk; ++k) {
            const int64_t r = row_at(a, t * a.topk + k);
            if (r < 0) continue;
            float f[8];
            dev::load_cols<VEC>(ys + r * a.hidden, cols, f);
            const float w = a.weights ? a.weights[t * a.topk + k] : 1.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] = fmaf(w, f[j], sum[j]);
        }
        dev::store_cols<VEC>(static_cast<T*>(a.out) + t * a.hidden, cols, sum);
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kMoveThreads) moe_combine_backward_kernel(MoveArgs a) {
    __shared__ float slots[2][kMoveThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int64_t t = blockIdx.x;
    const int H = static_cast<int>(a.hidden);
    if (t >= a.tokens) {
        clear_padding<T>(a, t - a.tokens, H);
        return;
    }
    const T* dout = static_cast<const T*>(a.x) + t * a.hidden;
    const T* ys = static_cast<const T*>(a.ys);
    T* dys = static_cast<T*>(a.sorted);
    for (int k = 0; k < a.topk; ++k) {
        const int64_t s = t * a.topk + k, r = row_at(a, s);
        float dot = 0.0f;
        if (r >= 0) {
            const float w = a.weights ? a.weights[s] : 1.0f;
            for (int v = threadIdx.x; v * 8 < H + 8 * kMoveThreads; v += kMoveThreads) {
                const dev::Cols<VEC> cols(v, kMoveThreads, H);
                if (!cols.any()) continue;
                float g[8], f[8];
                dev::load_cols<VEC>(dout, cols, g);
                if (a.dweights) {
                    dev::load_cols<VEC>(ys + r * a.hidden, cols, f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) dot = fmaf(g[j], f[j], dot);
                }
                if (dys) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[j] *= w;
                    dev::store_cols<VEC>(dys + r * a.hidden, cols, g);
                }
            }
        }
        if (a.dweights) {
            dot = dev::block_sum(dot, slots[k & 1]);
            if (threadIdx.x == 0) a.dweights[s] = dot;
        }
    }
}

// Rows whose bytes and buffers allow 16-byte vectors.
bool vectors(const MoveArgs& a) {
    auto ok = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    return a.hidden * a.elem_bytes % 16 == 0 && a.hidden % 8 == 0 && ok(a.x) && ok(a.ys) &&
           ok(a.sorted) && ok(a.out);
}

unsigned pad_blocks(const MoveArgs& a) {
    return static_cast<unsigned>(a.sorted ? (a.rows + kPadRows - 1) / kPadRows : 0);
}

template <typename F>
cudaError_t by_type(int dtype, F&& f) {
    if (dtype == 0) return f(__nv_bfloat16{});
    if (dtype == 1) return f(__half{});
    return f(float{});
}

}  // namespace

size_t sort_workspace(int64_t, int) { return 0; }

cudaError_t launch_moe_sort(const SortArgs& a, void*, cudaStream_t stream) {
    const size_t smem = sizeof(int) * (kSortWarps + 1) * a.experts;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            moe_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(moe_sort_kernel, dim3(1), dim3(kSortThreads), smem, stream, a);
}

cudaError_t launch_moe_dispatch(const MoveArgs& a, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.tokens) + pad_blocks(a));
    if (vectors(a))
        return launch_pdl(moe_dispatch_kernel<uint4>, grid, dim3(kMoveThreads), 0, stream, a);
    if (a.elem_bytes == 4)
        return launch_pdl(moe_dispatch_kernel<uint32_t>, grid, dim3(kMoveThreads), 0, stream, a);
    return launch_pdl(moe_dispatch_kernel<uint16_t>, grid, dim3(kMoveThreads), 0, stream, a);
}

cudaError_t launch_moe_combine(const MoveArgs& a, int dtype, cudaStream_t stream) {
    return by_type(dtype, [&](auto z) {
        using T = decltype(z);
        auto* kernel = vectors(a) ? moe_combine_kernel<T, true> : moe_combine_kernel<T, false>;
        return launch_pdl(kernel, dim3(static_cast<unsigned>(a.tokens)), dim3(kMoveThreads), 0,
                          stream, a);
    });
}

cudaError_t launch_moe_combine_backward(const MoveArgs& a, int dtype, cudaStream_t stream) {
    return by_type(dtype, [&](auto z) {
        using T = decltype(z);
        auto* kernel = vectors(a) ? moe_combine_backward_kernel<T, true>
                                  : moe_combine_backward_kernel<T, false>;
        return launch_pdl(kernel, dim3(static_cast<unsigned>(a.tokens) + pad_blocks(a)),
                          dim3(kMoveThreads), 0, stream, a);
    });
}

}  // namespace ct
