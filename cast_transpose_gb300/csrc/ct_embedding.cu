// ct_embedding.cu -- the embedding: rows of a table by token id, scaled, and
// the gradient of the table, the tokens sorted by id.
#include "ct_device.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"
#include "ct_vec.cuh"

#include <algorithm>

namespace ct {
namespace {

__device__ __forceinline__ int64_t id_of(const EmbeddingArgs& a, int64_t t) {
    return a.index64 ? static_cast<const int64_t*>(a.idx)[t] : static_cast<const int32_t*>(a.idx)[t];
}

constexpr int kEmbedThreads = 256;

// A block per token.
template <typename T, int G>
__global__ void __launch_bounds__(kEmbedThreads) embedding_kernel(const EmbeddingArgs a) {
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int H = static_cast<int>(a.hidden);
    const int64_t t = blockIdx.x, id = id_of(a, t);
    const bool inside = id >= 0 && id < a.vocab;
    const T* row = static_cast<const T*>(a.in) + (inside ? id : 0) * H;
    for (int vi = threadIdx.x; vi < (H + 255) / 256 * 32; vi += blockDim.x) {
        const dev::Cols<G> c(vi, H);
        float f[8] = {};
        if (inside) {
            dev::load_cols<G>(row, c, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= a.scale;
        }
        dev::store_cols<G>(static_cast<T*>(a.out) + t * H, c, f);
    }
}

// ---- sort --------------------------------------------------------------------
// A stable radix sort of the ids, the position of each along: passes of eight
// bits from the lowest, each of a count per block and digit, the sums of the
// counts, and the movement.  Ids outside the table get the number `vocab`, and
// so come last.
constexpr int kDigitBits = 8, kDigits = 1 << kDigitBits;
constexpr int kSortWarps = 8, kSortThreads = 32 * kSortWarps;
constexpr int kWarpKeys = 256, kBlockKeys = kWarpKeys * kSortWarps;

struct Sort {
    unsigned* key[2];     // [tokens], a pass reads one and writes the other
    int* pos[2];
    int* counts;          // [digits][blocks]
    int blocks;
};
int sort_blocks(int64_t tokens) { return static_cast<int>((tokens + kBlockKeys - 1) / kBlockKeys); }
int id_bits(int64_t vocab) {
    int bits = 1;
    while (bits < 31 && (int64_t(1) << bits) <= vocab) ++bits;
    return bits;
}
Sort sort_of(const EmbeddingArgs& a) {
    Sort s;
    const int64_t n = (a.tokens + 3) / 4 * 4;
    unsigned* w = static_cast<unsigned*>(a.workspace);
    for (int i = 0; i < 2; ++i) {
        s.key[i] = w + i * n;
        s.pos[i] = reinterpret_cast<int*>(w + (2 + i) * n);
    }
    s.counts = reinterpret_cast<int*>(w + 4 * n);
    s.blocks = sort_blocks(a.tokens);
    return s;
}

// Key i of pass `pass`, and its position.
__device__ __forceinline__ unsigned key_at(const EmbeddingArgs& a, const Sort& s, int pass, int64_t i) {
    if (pass > 0) return s.key[(pass - 1) & 1][i];
    const int64_t id = id_of(a, i);
    return static_cast<unsigned>(id >= 0 && id < a.vocab ? id : a.vocab);
}

// counts[digit][warp] of the block's keys.
__device__ __forceinline__ void count_keys(const EmbeddingArgs& a, const Sort& s, int pass,
                                           int (*counts)[kSortWarps + 1]) {
    for (int i = threadIdx.x; i < kDigits * (kSortWarps + 1); i += blockDim.x) counts[0][i] = 0;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = int64_t(blockIdx.x) * kBlockKeys + warp * kWarpKeys;
    for (int i = 0; i < kWarpKeys; i += 32) {
        const int64_t at = first + i + lane;
        if (at < a.tokens)
            atomicAdd(&counts[(key_at(a, s, pass, at) >> (kDigitBits * pass)) % kDigits][warp], 1);
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const EmbeddingArgs a, const Sort s, int pass) {
    __shared__ int counts[kDigits][kSortWarps + 1];
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    count_keys(a, s, pass, counts);
    for (int d = threadIdx.x; d < kDigits; d += blockDim.x) {
        int sum = 0;
        for (int w = 0; w < kSortWarps; ++w) sum += counts[d][w];
        s.counts[int64_t(d) * s.blocks + blockIdx.x] = sum;
    }
}

// Exclusive sums of the counts, in place.
__global__ void __launch_bounds__(1024) sort_scan_kernel(const EmbeddingArgs a, const Sort s) {
    __shared__ int warp_sums[32];
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n = int64_t(kDigits) * s.blocks;
    int base = 0;
    for (int64_t i0 = 0; i0 < n; i0 += blockDim.x) {
        const int64_t i = i0 + threadIdx.x;
        const int v = i < n ? s.counts[i] : 0;
        int sum = v;
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += up;
        }
        if (lane == 31) warp_sums[warp] = sum;
        __syncthreads();
        int sums = warp_sums[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, sums, o);
            if (lane >= o) sums += up;
        }
        const int earlier = __shfl_sync(0xFFFFFFFFu, sums, warp > 0 ? warp - 1 : 0);
        if (i < n) s.counts[i] = base + (warp > 0 ? earlier : 0) + sum - v;
        base += __shfl_sync(0xFFFFFFFFu, sums, 31);
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSortThreads) sort_move_kernel(const EmbeddingArgs a, const Sort s, int pass) {
    __shared__ int counts[kDigits][kSortWarps + 1];
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    count_keys(a, s, pass, counts);
    for (int d = threadIdx.x; d < kDigits; d += blockDim.x) {
        int sum = s.counts[int64_t(d) * s.blocks + blockIdx.x];
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = counts[d][w];
            counts[d][w] = sum;
            sum += c;
        }
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = int64_t(blockIdx.x) * kBlockKeys + warp * kWarpKeys;
    for (int i = 0; i < kWarpKeys; i += 32) {
        const int64_t at = first + i + lane;
        const bool here = at < a.tokens;
        const unsigned key = here ? key_at(a, s, pass, at) : 0;
        const int digit = here ? static_cast<int>((key >> (kDigitBits * pass)) % kDigits) : kDigits;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, digit);
        const int before = __popc(same & ((1u << lane) - 1));
        int to = 0;
        if (here) to = counts[digit][warp] + before;
        __syncwarp();
        if (here && before == 0) counts[digit][warp] += __popc(same);
        __syncwarp();
        if (here) {
            s.key[pass & 1][to] = key;
            s.pos[pass & 1][to] = pass > 0 ? s.pos[(pass - 1) & 1][at] : static_cast<int>(at);
        }
    }
}

// ---- gradient -----------------------------------------------------------------
// Zeros for the whole table.
__global__ void __launch_bounds__(kEmbedThreads) embedding_clear_kernel(const EmbeddingArgs a, int bytes) {
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int64_t n = a.vocab * a.hidden;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        if (bytes == 4) static_cast<uint32_t*>(a.out)[i] = 0;
        else static_cast<uint16_t*>(a.out)[i] = 0;
    }
}

// A block per sorted position: the first of an id sums all of it.
template <typename T, typename D, int G>
__global__ void __launch_bounds__(kEmbedThreads)
    embedding_sum_kernel(const EmbeddingArgs a, const unsigned* keys, const int* pos) {
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int H = static_cast<int>(a.hidden);
    const int64_t first = blockIdx.x;
    const unsigned id = keys[first];
    if (id >= a.vocab || (first > 0 && keys[first - 1] == id)) return;
    D* out = static_cast<D*>(a.out) + int64_t(id) * H;
    for (int vi = threadIdx.x; vi < (H + 255) / 256 * 32; vi += blockDim.x) {
        const dev::Cols<G> c(vi, H);
        float sum[8] = {}, f[8];
        for (int64_t i = first; i < a.tokens && keys[i] == id; ++i) {
            dev::load_cols<G>(static_cast<const T*>(a.in) + int64_t(pos[i]) * H, c, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += f[j];
        }
        float old[8] = {};
        if (a.accumulate) dev::load_cols<G>(out, c, old);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = fmaf(sum[j], a.scale, old[j]);
        dev::store_cols<G>(out, c, sum);
    }
}

}  // namespace

cudaError_t launch_embedding(const EmbeddingArgs& a, int dtype, cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 && all_aligned(a.in, a.out);
    return by_types(dtype, dtype, [&](auto t, auto) {
        using T = decltype(t);
        return launch_pdl(vec ? embedding_kernel<T, 8> : embedding_kernel<T, 1>,
                          dim3(static_cast<unsigned>(a.tokens)), dim3(kEmbedThreads), 0, stream, a);
    });
}

size_t embedding_backward_workspace(int64_t tokens, int64_t vocab, int64_t hidden) {
    return size_t((tokens + 3) / 4 * 4) * 16 + size_t(kDigits) * sort_blocks(tokens) * 4;
}

cudaError_t launch_embedding_backward(const EmbeddingArgs& a, int dtype, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (!a.accumulate) {
        e = launch_pdl(embedding_clear_kernel, dim3(sm_count() * 8), dim3(kEmbedThreads), 0, stream, a,
                       a.grad_f32 || dtype == 2 ? 4 : 2);
        if (e != cudaSuccess) return e;
    }
    if (a.tokens == 0) return e;
    const Sort s = sort_of(a);
    const int passes = (id_bits(a.vocab) + kDigitBits - 1) / kDigitBits;
    for (int pass = 0; pass < passes; ++pass) {
        e = launch_pdl(sort_count_kernel, dim3(s.blocks), dim3(kSortThreads), 0, stream, a, s, pass);
        if (e == cudaSuccess) e = launch_pdl(sort_scan_kernel, dim3(1), dim3(1024), 0, stream, a, s);
        if (e == cudaSuccess)
            e = launch_pdl(sort_move_kernel, dim3(s.blocks), dim3(kSortThreads), 0, stream, a, s, pass);
        if (e != cudaSuccess) return e;
    }
    const unsigned* keys = s.key[(passes - 1) & 1];
    const int* pos = s.pos[(passes - 1) & 1];
    const bool vec = a.hidden % 8 == 0 && all_aligned(a.in, a.out);
    return by_types(dtype, a.grad_f32 ? 2 : dtype, [&](auto t, auto d) {
        using T = decltype(t);
        using D = decltype(d);
        return launch_pdl(vec ? embedding_sum_kernel<T, D, 8> : embedding_sum_kernel<T, D, 1>,
                          dim3(static_cast<unsigned>(a.tokens)), dim3(kEmbedThreads), 0, stream, a, keys, pos);
    });
}

}  // namespace ct
