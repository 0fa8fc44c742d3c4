// ct_embedding.cu -- the embedding: rows of a table by token id, scaled, and
// the gradient of the table, the tokens sorted by id.
//
// Bound by HBM.  Measured, one GB300, of the measured copy rate: 16384 rows of 6144
// bf16 44.5 us (278 MB of distinct rows and output, 0.92); the gradient of 16384
// tokens into 65536x4096 fp32 213 us (1208 MB, 0.84).  Of that the zeros of the rows
// without a token take 154 us (908 MB: 5.9 TB/s, what stores alone reach here),
// beside which the sort costs nothing; the sums 43 us, the join of frequent ids 8.
// The gradient is deterministic: the sort is stable, an id's rows are added in the
// order of the tokens within a chunk, and the chunks in theirs.
#include "ct_device.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"
#include "ct_vec.cuh"

#include <algorithm>
#include <atomic>
#include <cooperative_groups.h>

namespace ct {
namespace {

__device__ __forceinline__ int64_t id_of(const EmbeddingArgs& a, int64_t t) {
    return a.index64 ? static_cast<const int64_t*>(a.idx)[t] : static_cast<const int32_t*>(a.idx)[t];
}

constexpr int kEmbedThreads = 256;

// A block per token; a thread's kEmbedItems loads are in flight together.
constexpr int kEmbedItems = 4;

template <typename T, int G>
__global__ void __launch_bounds__(kEmbedThreads) embedding_kernel(const EmbeddingArgs a) {
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int H = static_cast<int>(a.hidden);
    const int64_t t = blockIdx.x, id = id_of(a, t);
    const bool inside = id >= 0 && id < a.vocab;
    const T* row = static_cast<const T*>(a.in) + (inside ? id : 0) * H;
    T* out = static_cast<T*>(a.out) + t * H;
    for (int v0 = threadIdx.x; v0 < (H + 255) / 256 * 32; v0 += kEmbedItems * blockDim.x) {
        dev::RawCols<G, T> raw[kEmbedItems];
        if (inside)
#pragma unroll
            for (int i = 0; i < kEmbedItems; ++i) raw[i].load(row, dev::Cols<G>(v0 + i * blockDim.x, H));
#pragma unroll
        for (int i = 0; i < kEmbedItems; ++i) {
            float f[8] = {};
            if (inside) {
                raw[i].get(f);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] *= a.scale;
            }
            dev::store_cols<G>(out, dev::Cols<G>(v0 + i * blockDim.x, H), f);
        }
    }
}

// ---- sort --------------------------------------------------------------------
// A stable radix sort of the ids, the position of each along, from the lowest
// digit.  Ids outside the table get the number `vocab`, and so come last.  Up to
// kClusterKeys of them are sorted by one cluster in its shared memory; the fill
// of the table, which needs nothing but the ids, runs beside it.  More go through
// global memory: per digit a count per block, the sums of the counts, and the
// movement.
constexpr int kDigitBits = 8, kDigits = 1 << kDigitBits;
constexpr int kSortWarps = 8, kSortThreads = 32 * kSortWarps;
constexpr int kWarpKeys = 256, kBlockKeys = kWarpKeys * kSortWarps;

struct Sort {
    unsigned* key[2];     // [tokens], a pass reads one and writes the other
    int* pos[2];
    int* counts;          // [digits][blocks]
    float* parts;         // [chunks][2][stride], see embedding_sum_kernel
    int* leaves;          // [chunks]: an id of more than kShort tokens begins in the chunk and goes on
    int64_t stride;
    int blocks;
    int chunk, chunks;    // tokens in sorted order, by the chunk
};
int sort_blocks(int64_t tokens) { return static_cast<int>((tokens + kBlockKeys - 1) / kBlockKeys); }
int id_bits(int64_t vocab) {
    int bits = 1;
    while (bits < 31 && (int64_t(1) << bits) <= vocab) ++bits;
    return bits;
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

// ---- sort in one cluster ------------------------------------------------------
// Every block holds `share` consecutive positions, every thread KEYS of them in
// registers.  A pass: the rank of a key among its warp's with the same digit from
// a count per digit and warp, the sums of those over the warps, then over the
// blocks (read from their shared memory), and the key goes to its place in some
// block's shared memory, in the last pass to global memory.
constexpr int kClusterBlocks = 8, kSmallCluster = 4, kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32;
constexpr int kClusterMaxPerThread = 16;
constexpr int64_t kClusterKeys = int64_t(kClusterBlocks) * kClusterThreads * kClusterMaxPerThread;
constexpr int kClusterMaxBits = 9;                  // of a digit
constexpr int kHistRow = kClusterWarps + 1;         // so that neither a row's nor a column's entries share a bank

struct ClusterSort {
    unsigned* keys;       // [tokens] sorted
    int* pos;
    int blocks;           // of the cluster
    int share;            // positions per block
    int bits, passes;     // of a digit; digits
    int fill_blocks;      // blocks after the cluster's, which clear the table
};
size_t cluster_smem(const ClusterSort& s) {
    return size_t(s.share) * 8 + (size_t(1) << s.bits) * (kHistRow + 2) * 4;
}

// Clears the rows of the table that no token has, some of them per block: a bit
// for each row of the range that an id falls into.
constexpr int kFillRows = 32768;

template <typename D, int ROWS>
__device__ void clear_rows(const EmbeddingArgs& a, unsigned* used, int block, int blocks) {
    const int64_t begin = a.vocab * block / blocks, end = a.vocab * (block + 1) / blocks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t H = a.hidden;
    const bool vec = H * sizeof(D) % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
    for (int64_t q = begin; q < end; q += ROWS) {
        const int rows = static_cast<int>(min(end - q, int64_t(ROWS)));
        for (int i = threadIdx.x; i < (rows + 31) / 32; i += blockDim.x) used[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int64_t t = threadIdx.x; t < a.tokens; t += blockDim.x) {
            const int64_t r = id_of(a, t) - q;
            if (r >= 0 && r < rows) atomicOr(used + (r >> 5), 1u << (r & 31));
        }
        __syncthreads();
        for (int r = warp; r < rows; r += warps) {
            if ((used[r >> 5] >> (r & 31)) & 1) continue;
            D* row = static_cast<D*>(a.out) + (q + r) * H;
            if (vec) {
                uint4* w = reinterpret_cast<uint4*>(row);
                for (int64_t i = lane; i < H * int(sizeof(D)) / 16; i += 32) __stcs(w + i, make_uint4(0, 0, 0, 0));
            } else {
                for (int64_t i = lane; i < H; i += 32) row[i] = D{};
            }
        }
        __syncthreads();
    }
}

template <int KEYS, typename D>
__global__ void __launch_bounds__(kClusterThreads, 1)
    embedding_sort_kernel(const EmbeddingArgs a, const ClusterSort s) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    if (int(blockIdx.x) >= s.blocks) {
        clear_rows<D, kFillRows>(a, reinterpret_cast<unsigned*>(smem), blockIdx.x - s.blocks, s.fill_blocks);
        return;
    }
    const auto cluster = cooperative_groups::this_cluster();
    const int rank = blockIdx.x, digits = 1 << s.bits;
    uint2* kv = reinterpret_cast<uint2*>(smem);                     // [share]
    int* hist = reinterpret_cast<int*>(kv + s.share);               // [digits][kHistRow]
    int* own = hist + digits * kHistRow;                            // [digits]: keys of this block
    int* base = own + digits;                                       // [digits]: where they go
    const int64_t first = int64_t(rank) * s.share;
    const int count = static_cast<int>(max(int64_t(0), min(int64_t(s.share), a.tokens - first)));
    unsigned key[KEYS];
    int pos[KEYS], at[KEYS];
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
        const int p = (warp * KEYS + i) * 32 + lane;
        int64_t id = a.vocab;
        if (p < count) id = id_of(a, first + p);
        key[i] = static_cast<unsigned>(id >= 0 && id < a.vocab ? id : a.vocab);
        pos[i] = static_cast<int>(first) + p;
    }
    for (int pass = 0; pass < s.passes; ++pass) {
        const int shift = pass * s.bits;
        for (int i = tid; i < digits * kHistRow; i += kClusterThreads) hist[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const bool here = (warp * KEYS + i) * 32 + lane < count;
            const int digit = (key[i] >> shift) & (digits - 1);
            unsigned same = __ballot_sync(0xFFFFFFFFu, here);
            same = here ? same : 0;
            for (int b = 0; b < s.bits; ++b) {
                const bool bit = (digit >> b) & 1;
                const unsigned set = __ballot_sync(0xFFFFFFFFu, bit);
                same &= bit ? set : ~set;
            }
            int* entry = hist + digit * kHistRow + warp;
            const int before = __popc(same & ((1u << lane) - 1));
            at[i] = here ? *entry + before : 0;
            __syncwarp();
            if (here && before == 0) *entry += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        for (int d = tid; d < digits; d += kClusterThreads) {
            int* row = hist + d * kHistRow;
            int sum = 0;
#pragma unroll 8
            for (int w = 0; w < kClusterWarps; ++w) {
                const int c = row[w];
                row[w] = sum;
                sum += c;
            }
            own[d] = sum;
        }
        cluster.sync();                     // and everyone has its keys in registers
        int before = 0, total = 0;          // digits <= threads: a thread per digit
        if (tid < digits)
            for (int o = 0; o < s.blocks; ++o) {
                const int c = cluster.map_shared_rank(own, o)[tid];
                before += o < rank ? c : 0;
                total += c;
            }
        int sum = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += up;
        }
        if (lane == 31) warp_sums[warp] = sum;
        __syncthreads();
        int sums = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, sums, o);
            if (lane >= o) sums += up;
        }
        const int earlier = __shfl_sync(0xFFFFFFFFu, sums, warp > 0 ? warp - 1 : 0);
        if (tid < digits) base[tid] = (warp > 0 ? earlier : 0) + sum - total + before;
        __syncthreads();
        const bool last = pass + 1 == s.passes;
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            if ((warp * KEYS + i) * 32 + lane >= count) continue;
            const int digit = (key[i] >> shift) & (digits - 1);
            const unsigned to = base[digit] + hist[digit * kHistRow + warp] + at[i];
            if (last) {
                s.keys[to] = key[i];
                s.pos[to] = pos[i];
            } else {
                const unsigned block = to / s.share;
                cluster.map_shared_rank(kv, block)[to - block * s.share] = make_uint2(key[i], pos[i]);
            }
        }
        cluster.sync();                     // the last time: before a block leaves that others read from
        if (last) break;
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const int p = (warp * KEYS + i) * 32 + lane;
            if (p < count) {
                const uint2 v = kv[p];
                key[i] = v.x;
                pos[i] = static_cast<int>(v.y);
            }
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

// Sums of the rows of each id, in sorted order.  A block takes a chunk of the
// sorted tokens and some columns; kRows rows are loaded at a time, whichever ids
// they have.  An id of at most kShort tokens is summed and written by the block of
// the chunk that it begins in, which goes on past its chunk for that; of one with
// more every chunk's sum goes to the workspace: place 0 where the id began in an
// earlier chunk, else place 1.  (Unless such a one begins and ends in one chunk.)
constexpr int kMaxChunk = 1024;
constexpr int kShort = 32;                       // a warp's lanes look at as many keys
constexpr unsigned kNone = 0xFFFFFFFFu;

template <typename D, int G>
__device__ __forceinline__ void put_row(const EmbeddingArgs& a, unsigned id, const dev::Cols<G>& c, float (&sum)[8]) {
    D* out = static_cast<D*>(a.out) + int64_t(id) * a.hidden;
    float old[8] = {};
    if (a.accumulate) dev::load_cols<G>(out, c, old);
#pragma unroll
    for (int j = 0; j < 8; ++j) old[j] = fmaf(sum[j], a.scale, old[j]);
    dev::store_cols<G>(out, c, old);
}

// Of at most kShort: how many keys before (step -1) or from (step 1) p on are id.
__device__ __forceinline__ int same_keys(const unsigned* p, int step, unsigned id) {
    const unsigned other = __ballot_sync(0xFFFFFFFFu, p[step * int(threadIdx.x & 31)] != id);
    return other ? __ffs(other) - 1 : kShort;
}

template <typename T, typename D, int G>
__global__ void __launch_bounds__(kEmbedThreads)
    embedding_sum_kernel(const EmbeddingArgs a, const Sort s, const unsigned* keys, const int* pos) {
    __shared__ unsigned window[kMaxChunk + 2 * kShort + 1];      // the chunk's keys and those around it
    __shared__ int row[kMaxChunk + kShort];
    constexpr int kRows = sizeof(T) == 4 ? 4 : 8;
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int H = static_cast<int>(a.hidden), chunk = blockIdx.x;
    const int64_t lo = int64_t(chunk) * s.chunk;
    const int n = static_cast<int>(min(int64_t(s.chunk), a.tokens - lo));
    const unsigned* key = window + kShort;
    for (int i = threadIdx.x; i < n + 2 * kShort + 1; i += blockDim.x) {
        const int64_t p = lo + i - kShort;
        window[i] = p >= 0 && p < a.tokens ? keys[p] : kNone;
        if (i < n + kShort && lo + i < a.tokens) row[i] = pos[lo + i];
    }
    __syncthreads();
    // [begin, end): what this block sums.  Its first id may have begun before, its
    // last one may go on.
    int begin = 0, end = n;
    const int earlier = same_keys(key - 1, -1, key[0]);
    const bool began = earlier == kShort || (earlier > 0 && key[kShort - earlier] == key[0]);
    if (earlier > 0 && !began)
        for (begin = 1; begin < n && key[begin] == key[0];) ++begin;
    if (begin < n && key[n] == key[n - 1]) {
        const int inside = same_keys(key + n - 1, -1, key[n - 1]);     // these may lie before the chunk, too
        if (inside < kShort && key[n - inside + kShort] != key[n - 1]) end = n + same_keys(key + n, 1, key[n - 1]);
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        const bool whole = began && key[0] == key[n - 1];
        s.leaves[chunk] = end == n && key[n] == key[n - 1] && key[n] < a.vocab && begin < n && !whole;
    }
    for (int vi = blockIdx.y * blockDim.x + threadIdx.x; vi < (H + 255) / 256 * 32; vi += gridDim.y * blockDim.x) {
        const dev::Cols<G> c(vi, H);
        float sum[8] = {};
        bool part = began;                       // of an id that began in an earlier chunk
        for (int i0 = begin; i0 < end; i0 += kRows) {
            if (key[i0] >= a.vocab) break;
            dev::RawCols<G, T> raw[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                raw[r].load(static_cast<const T*>(a.in) + int64_t(row[min(i0 + r, end - 1)]) * H, c);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int i = i0 + r;
                if (i >= end || key[i] >= a.vocab) break;
                float f[8];
                raw[r].get(f);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += f[j];
                const bool goes_on = key[i + 1] == key[i];
                if (goes_on && i + 1 < end) continue;
                if (part || goes_on)
                    dev::store_cols<G>(s.parts + (2 * int64_t(chunk) + (part ? 0 : 1)) * s.stride, c, sum);
                else
                    put_row<D>(a, key[i], c, sum);
                part = false;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
            }
        }
    }
}

// The ids of more than kShort tokens that lie in more than one chunk: the sums of
// the chunks, every kJoinWays-th by a warp.  A block looks at some chunks for those
// that such an id begins in.
constexpr int kJoinWays = 8, kJoinThreads = 32 * kJoinWays;
constexpr int kJoinColumns = 128;                // of a step: four for every lane
constexpr int kJoinBatch = 8;
constexpr int kJoinBlocks = 64;

template <typename D>
__global__ void __launch_bounds__(kJoinThreads)
    embedding_join_kernel(const EmbeddingArgs a, const Sort s, const unsigned* keys) {
    __shared__ float4 sums[kJoinWays][32];
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // frequent ids lie side by side: every gridDim.x-th chunk
    for (int64_t group = blockIdx.x; group < s.chunks; group += 32 * int64_t(gridDim.x)) {
        const int64_t mine = group + lane * int64_t(gridDim.x);
        unsigned left = __ballot_sync(0xFFFFFFFFu, mine < s.chunks && s.leaves[min(mine, int64_t(s.chunks) - 1)]);
        for (; left; left &= left - 1) {
            const int64_t chunk = group + (__ffs(left) - 1) * int64_t(gridDim.x), next = (chunk + 1) * s.chunk;
            const unsigned id = keys[next];
            int64_t more = 0;                    // the chunks after this one that begin with the id
            for (;; more += 32) {
                const int64_t p = next + (more + lane) * s.chunk;
                const unsigned end = __ballot_sync(0xFFFFFFFFu, p >= a.tokens || keys[min(p, a.tokens - 1)] != id);
                if (end) {
                    more += __ffs(end) - 1;
                    break;
                }
            }
            for (int64_t c0 = int64_t(blockIdx.y) * kJoinColumns; c0 < a.hidden;
                 c0 += int64_t(gridDim.y) * kJoinColumns) {
                const int64_t col = c0 + 4 * lane;   // the workspace's rows are whole multiples of four
                const bool here = col < a.hidden;
                const float* part = s.parts + 2 * chunk * s.stride + (here ? col : 0);
                float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (warp == 0) sum = *reinterpret_cast<const float4*>(part + s.stride);
                for (int64_t i0 = 1 + warp; i0 <= more; i0 += kJoinWays * kJoinBatch) {
                    float4 v[kJoinBatch];
#pragma unroll
                    for (int i = 0; i < kJoinBatch; ++i)
                        v[i] = dev::load_now(reinterpret_cast<const float4*>(part + 2 * min(i0 + i * kJoinWays, more) * s.stride));
#pragma unroll
                    for (int i = 0; i < kJoinBatch; ++i) {
                        const bool use = i0 + i * kJoinWays <= more;
                        sum.x += use ? v[i].x : 0.0f;
                        sum.y += use ? v[i].y : 0.0f;
                        sum.z += use ? v[i].z : 0.0f;
                        sum.w += use ? v[i].w : 0.0f;
                    }
                }
                __syncthreads();
                sums[warp][lane] = sum;
                __syncthreads();
                if (warp != 0) continue;
                for (int w = 1; w < kJoinWays; ++w) {
                    const float4 v = sums[w][lane];
                    sum.x += v.x;
                    sum.y += v.y;
                    sum.z += v.z;
                    sum.w += v.w;
                }
                const float f[4] = {sum.x, sum.y, sum.z, sum.w};
                D* out = static_cast<D*>(a.out) + int64_t(id) * a.hidden + col;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col + j < a.hidden)
                        dev::from_f32(out[j], fmaf(f[j], a.scale, a.accumulate ? dev::to_f32(out[j]) : 0.0f));
            }
        }
    }
}

// ---- few tokens -------------------------------------------------------------------
// Without a sort, in one launch: a block per token looks at all the ids, and where no
// earlier token has its own it sums the rows of those that do.  kFewWays groups of
// threads take consecutive parts of them, whose sums are added in their order.  The
// blocks after those clear the rows without a token.
//
// Measured with its zeros, us, against the sort: 1000 tokens into 2000x512 bf16 7.4
// against 14.7, 512 into 65536x4096 82.5 against 93.  What limits it is an id that
// most tokens have, which has one block for its columns (and no ways for rows past
// 1024): 1024 equal ids 18 against 14 with 512 columns, 66 against 16 with 4096.
constexpr int kFewTokens = 1024, kFewTokensWide = 512, kFewWide = 1024;
inline bool few_tokens(int64_t tokens, int64_t hidden) {
    return tokens <= (hidden > kFewWide ? kFewTokensWide : kFewTokens);
}
constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
constexpr int kFewFillRows = 8192;               // as kFillRows

template <typename T, typename D, int G>
__global__ void __launch_bounds__(kFewThreads)
    embedding_few_kernel(const EmbeddingArgs a, int fill_blocks, int ways) {
    __shared__ union {
        struct {
            int rows[kFewTokens];
            float sums[kFewThreads][9];          // a thread's eight columns, banks apart
        } own;
        unsigned used[kFewFillRows / 32];
    } mem;
    __shared__ int counts[kFewWarps + 1];
    constexpr int kRows = sizeof(T) == 4 ? 4 : 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = static_cast<int>(a.tokens);
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    if (int(blockIdx.x) >= n) {
        if (blockIdx.y == 0) clear_rows<D, kFewFillRows>(a, mem.used, blockIdx.x - n, fill_blocks);
        return;
    }
    const int64_t id = id_of(a, blockIdx.x);
    if (id < 0 || id >= a.vocab) return;
    // the tokens with the id, in order: each warp's part of the ids, then all of them
    constexpr int kParts = kFewTokens / kFewThreads;         // of 32 ids per warp
    unsigned same[kParts];
    int found = 0;
    bool earlier = false;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const int t = (warp * kParts + i) * 32 + lane;
        const bool here = t < n && id_of(a, min(t, n - 1)) == id;
        earlier |= here && t < int(blockIdx.x);
        same[i] = __ballot_sync(0xFFFFFFFFu, here);
        found += __popc(same[i]);
    }
    if (__syncthreads_or(earlier)) return;
    if (lane == 0) counts[warp] = found;
    __syncthreads();
    int at = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
        at += w < warp ? counts[w] : 0;
        all += counts[w];
    }
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        if ((same[i] >> lane) & 1) mem.own.rows[at + __popc(same[i] & ((1u << lane) - 1))] = (warp * kParts + i) * 32 + lane;
        at += __popc(same[i]);
    }
    __syncthreads();
    const int H = static_cast<int>(a.hidden), group = kFewThreads / ways, way = tid / group;
    const int begin = all * way / ways, end = all * (way + 1) / ways;
    const int items = (H + 255) / 256 * 32;
    for (int v0 = blockIdx.y * group; v0 < items; v0 += gridDim.y * group) {
        const dev::Cols<G> c(v0 + tid % group, H);
        float sum[8] = {};
        for (int i0 = begin; i0 < end; i0 += kRows) {
            dev::RawCols<G, T> raw[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                raw[r].load(static_cast<const T*>(a.in) + int64_t(mem.own.rows[min(i0 + r, end - 1)]) * H, c);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float f[8];
                raw[r].get(f);
                const bool use = i0 + r < end;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += use ? f[j] : 0.0f;
            }
        }
        if (ways > 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) mem.own.sums[tid][j] = sum[j];
            __syncthreads();
            if (way == 0)
                for (int w = 1; w < ways; ++w)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] += mem.own.sums[tid + w * group][j];
            __syncthreads();
        }
        if (way == 0) put_row<D>(a, static_cast<unsigned>(id), c, sum);
    }
}

template <typename T, typename D>
cudaError_t launch_few(const EmbeddingArgs& a, bool vec, cudaStream_t stream) {
    const int items = static_cast<int>((a.hidden + 255) / 256 * 32);
    const int ways = items <= 32 ? 8 : items <= 64 ? 4 : items <= 128 ? 2 : 1;
    // blocks for the columns while there are few of tokens
    const int slices = std::min((items + kFewThreads - 1) / kFewThreads, 16);
    int64_t fill = 0;
    if (!a.accumulate)
        fill = std::min<int64_t>(int64_t(sm_count()) * 4,
                                 std::max<int64_t>(1, a.vocab * a.hidden * int64_t(sizeof(D)) / 16384));
    return launch_pdl(vec ? embedding_few_kernel<T, D, 8> : embedding_few_kernel<T, D, 1>,
                      dim3(static_cast<unsigned>(a.tokens + fill), slices), dim3(kFewThreads), 0, stream, a,
                      static_cast<int>(fill), ways);
}

// The tokens by chunks: 16 each, more where those would be more than 2048.
void set_chunks(Sort& s, int64_t tokens, int64_t hidden) {
    s.chunk = static_cast<int>(std::min<int64_t>(kMaxChunk, std::max<int64_t>(16, (tokens + 2047) / 2048)));
    s.chunks = static_cast<int>((tokens + s.chunk - 1) / s.chunk);
    s.stride = (hidden + 3) / 4 * 4;
}
Sort sort_of(const EmbeddingArgs& a) {
    Sort s = {};
    const int64_t n = (a.tokens + 3) / 4 * 4;
    const int copies = a.tokens > kClusterKeys ? 2 : 1;
    unsigned* w = static_cast<unsigned*>(a.workspace);
    for (int i = 0; i < copies; ++i, w += 2 * n) {
        s.key[i] = w;
        s.pos[i] = reinterpret_cast<int*>(w + n);
    }
    set_chunks(s, a.tokens, a.hidden);
    s.parts = reinterpret_cast<float*>(w);
    s.leaves = reinterpret_cast<int*>(s.parts + 2 * s.chunks * s.stride);
    s.blocks = sort_blocks(a.tokens);
    s.counts = s.leaves + s.chunks;
    return s;
}

// Before the first launch on a device: allows the kernels the shared memory that
// they may ask for.  Gives the clusters of `blocks` blocks (kClusterBlocks or
// kSmallCluster) that are resident at a time.
template <typename D>
cudaError_t prepare_sort(int blocks, int* clusters) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[2][kDevices];  // 0: not yet
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const bool keep = device >= 0 && device < kDevices;
    std::atomic<int>* place = known[blocks == kClusterBlocks] + (keep ? device : 0);
    if (keep && (*clusters = place->load(std::memory_order_acquire)) > 0) return cudaSuccess;
    ClusterSort most = {};
    most.share = kClusterThreads * kClusterMaxPerThread;
    most.bits = kClusterMaxBits;
    const size_t smem = cluster_smem(most);
    for (auto* kernel : {embedding_sort_kernel<1, D>, embedding_sort_kernel<2, D>, embedding_sort_kernel<4, D>,
                         embedding_sort_kernel<8, D>, embedding_sort_kernel<16, D>}) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(clusters, embedding_sort_kernel<16, D>, &cfg);
    if (e != cudaSuccess) return e;
    *clusters = std::max(1, *clusters);
    if (keep) place->store(*clusters, std::memory_order_release);
    return cudaSuccess;
}

template <typename D>
cudaError_t launch_cluster_sort(const EmbeddingArgs& a, const Sort& to, cudaStream_t stream) {
    ClusterSort s = {};
    s.keys = to.key[0];
    s.pos = to.pos[0];
    s.blocks = !a.accumulate && a.tokens <= kSmallCluster * kClusterThreads * 8 ? kSmallCluster : kClusterBlocks;
    s.share = static_cast<int>((a.tokens + s.blocks - 1) / s.blocks);
    const int all = id_bits(a.vocab);
    s.passes = (all + kClusterMaxBits - 1) / kClusterMaxBits;
    s.bits = (all + s.passes - 1) / s.passes;
    const int keys = (s.share + kClusterThreads - 1) / kClusterThreads;
    auto* kernel = keys <= 1 ? embedding_sort_kernel<1, D> : keys <= 2 ? embedding_sort_kernel<2, D>
                 : keys <= 4 ? embedding_sort_kernel<4, D> : keys <= 8 ? embedding_sort_kernel<8, D>
                             : embedding_sort_kernel<16, D>;
    int clusters = 0;
    cudaError_t e = prepare_sort<D>(s.blocks, &clusters);
    if (e != cudaSuccess) return e;
    if (!a.accumulate) {
        // as many as are resident beside the sort's, each with 64 KB at least
        const int64_t bytes = a.vocab * a.hidden * int64_t(sizeof(D));
        const int64_t room = (clusters - 1) * s.blocks;
        const int64_t want = std::max<int64_t>(1, std::min<int64_t>(room, (bytes + 65535) / 65536));
        s.fill_blocks = static_cast<int>((want + s.blocks - 1) / s.blocks * s.blocks);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(s.blocks + s.fill_blocks);
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = std::max<size_t>(cluster_smem(s), kFillRows / 8);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = s.blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, s);
}

cudaError_t launch_grid_sort(const EmbeddingArgs& a, const Sort& s, int grad_bytes, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (!a.accumulate)
        e = launch_pdl(embedding_clear_kernel, dim3(sm_count() * 8), dim3(kEmbedThreads), 0, stream, a, grad_bytes);
    const int passes = (id_bits(a.vocab) + kDigitBits - 1) / kDigitBits;
    for (int pass = 0; pass < passes && e == cudaSuccess; ++pass) {
        e = launch_pdl(sort_count_kernel, dim3(s.blocks), dim3(kSortThreads), 0, stream, a, s, pass);
        if (e == cudaSuccess) e = launch_pdl(sort_scan_kernel, dim3(1), dim3(1024), 0, stream, a, s);
        if (e == cudaSuccess)
            e = launch_pdl(sort_move_kernel, dim3(s.blocks), dim3(kSortThreads), 0, stream, a, s, pass);
    }
    return e;
}

}  // namespace

cudaError_t launch_embedding(const EmbeddingArgs& a, int dtype, cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 && all_aligned(a.in, a.out);
    return by_types(dtype, dtype, [&](auto t, auto) {
        using T = decltype(t);
        const int items = static_cast<int>((a.hidden + 255) / 256 * 32);
        const int threads = std::min(kEmbedThreads, (items / 32 + kEmbedItems - 1) / kEmbedItems * 32);
        return launch_pdl(vec ? embedding_kernel<T, 8> : embedding_kernel<T, 1>,
                          dim3(static_cast<unsigned>(a.tokens)), dim3(threads), 0, stream, a);
    });
}

size_t embedding_backward_workspace(int64_t tokens, int64_t vocab, int64_t hidden) {
    if (few_tokens(tokens, hidden)) return 0;
    Sort s = {};
    set_chunks(s, tokens, hidden);
    const size_t lists = size_t((tokens + 3) / 4 * 4) * 8, parts = size_t(s.chunks) * (2 * s.stride + 1) * 4;
    return tokens > kClusterKeys ? 2 * lists + parts + size_t(kDigits) * sort_blocks(tokens) * 4 : lists + parts;
}

cudaError_t launch_embedding_backward(const EmbeddingArgs& a, int dtype, cudaStream_t stream) {
    const Sort s = sort_of(a);
    const bool vec = a.hidden % 8 == 0 && all_aligned(a.in, a.out);
    return by_types(dtype, a.grad_f32 ? 2 : dtype, [&](auto t, auto d) {
        using T = decltype(t);
        using D = decltype(d);
        if (few_tokens(a.tokens, a.hidden)) return launch_few<T, D>(a, vec, stream);
        const bool grid = a.tokens > kClusterKeys;
        cudaError_t e = grid ? launch_grid_sort(a, s, sizeof(D), stream) : launch_cluster_sort<D>(a, s, stream);
        if (e != cudaSuccess) return e;
        const int last = grid ? ((id_bits(a.vocab) + kDigitBits - 1) / kDigitBits - 1) & 1 : 0;
        const int items = static_cast<int>((a.hidden + 255) / 256 * 32);
        const int threads = std::min(items, kEmbedThreads);
        e = launch_pdl(vec ? embedding_sum_kernel<T, D, 8> : embedding_sum_kernel<T, D, 1>,
                       dim3(s.chunks, std::min((items + threads - 1) / threads, 64)), dim3(threads), 0, stream, a, s,
                       s.key[last], s.pos[last]);
        if (e != cudaSuccess) return e;
        const int columns = static_cast<int>(std::min<int64_t>((a.hidden + kJoinColumns - 1) / kJoinColumns, 32));
        return launch_pdl(embedding_join_kernel<D>, dim3(std::min(s.chunks, kJoinBlocks), columns),
                          dim3(kJoinThreads), 0, stream, a, s, s.key[last]);
    });
}

}  // namespace ct
