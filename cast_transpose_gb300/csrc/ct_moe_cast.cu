// ct_moe_cast.cu -- rows gathered into expert order, weighted, cast to FP8 and
// transposed in one pass: q[r] = fp8(w[s] * x[s / K] * scale), s = src[r].
#include "ct_device.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"

#include <type_traits>

namespace ct {
namespace {

constexpr int kCastThreads = 256;
constexpr int kStripTiles = 4;

// Token of a sorted row and its weight; -1 for padding.
__device__ __forceinline__ int token_of(const SortedCastArgs& a, int64_t row, float& w) {
    const int s = a.src[row];
    w = 0.0f;
    if (s < 0 || s >= a.tokens * a.topk) return -1;
    if (a.weights) w = a.weights[s];
    return s / a.topk;
}

__device__ __forceinline__ unsigned max_bits(unsigned m, float v) {
    return max(m, __float_as_uint(v) & 0x7FFFFFFFu);
}

// Tiles of 128x128 of the sorted matrix: hidden a multiple of 8, x 16-byte and
// out 8-byte aligned; with the transpose, rows a multiple of 16 and out_t
// 16-byte aligned.  Bound by HBM: 2 bytes read per element of x, 2 written per
// element of the sorted matrix.
//
// A block takes kStripTiles tiles side by side, so that the look-up of their
// rows' tokens (a load that everything else waits for) is paid once, and has
// the next tile's loads in flight while it transposes this one.  Blocks go down
// the rows of one strip before the next: a token's K copies then find the
// strip of its row in L2 (T * 1 KB in all; DRAM reads x once).
//
// 16384 tokens, K = 4, 6144 columns, E4M3, 1.02 GB: 165 us, 6.2 TB/s, 0.91 of
// the measured copy rate; the rest is issue (60% of the slots) and the last
// wave of blocks.  With the sort before it: one tile a block 217 us, strips of
// 2 / 4 / 8 196 / 190 / 208; whole tiles without checks, 180; one barrier a
// tile, 175; single tiles in the last wave, 173.  Tiles stacked down the rows
// instead of side by side: 187.  Four blocks per SM hold a thread to 64
// registers: with the transpose it spills one word, with the weights six, but
// three blocks with more registers take 204.
template <int FMT, bool WEIGHTED, bool TRANSPOSE>
__global__ void __launch_bounds__(kCastThreads, 4)
    sorted_cast_kernel(const SortedCastArgs a, int tile_rows, int tile_cols, int whole_strips) {
    __shared__ __align__(16) uint8_t sq2[2][TRANSPOSE ? 128 * 128 : 16];   // FP8 copies, in turn
    __shared__ int token[128];
    __shared__ float weight[WEIGHTED ? 128 : 1];
    __shared__ unsigned warp_max[kCastThreads / 32];
    dev::pdl_launch_dependents();
    // the first blocks take a strip of a tile row each, the others one tile
    const int single = static_cast<int>(blockIdx.x) - whole_strips;
    const int item = single < 0 ? blockIdx.x : whole_strips + single / kStripTiles;
    const int strip = item / tile_rows;
    const int first = strip * kStripTiles + (single < 0 ? 0 : single % kStripTiles);
    const int last = min(single < 0 ? first + kStripTiles : first + 1, tile_cols);
    const int64_t row0 = int64_t(item - strip * tile_rows) * 128;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    if (tid < 128) {
        float w = 0.0f;
        token[tid] = row0 + tid < a.rows ? token_of(a, row0 + tid, w) : -1;
        if (WEIGHTED) weight[tid] = w;
    }
    const float scale = *a.scale;
    // no padding and no end among the block's rows: most blocks
    const bool whole_rows = __syncthreads_and(tid >= 128 || token[tid & 127] >= 0);

    unsigned most = 0;
    uint4 v[8];
    // columns 8c .. 8c+7 of rows rg + 16 i: all eight loads in flight at once
    const int c = tid & 15, rg = tid >> 4;
    // rows 16b .. 16b+15 of the four columns of word w
    const int b = lane & 7, w4 = warp * 4 + (lane >> 3);
    const uint16_t* x = a.x + 8 * c;
    uint8_t* const q0 = a.out + (row0 + rg) * a.hidden + 8 * c;
    uint8_t* const t0 = TRANSPOSE ? a.out_t + int64_t(4 * w4) * a.rows + row0 + 16 * b : nullptr;
    const int64_t q_step = 16 * a.hidden;

    // WHOLE: every row and column of the tile is there.
    auto load = [&](auto whole, int64_t col0) {
        constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int t = token[rg + 16 * i];
            const uint4* p = reinterpret_cast<const uint4*>(x + t * a.hidden + col0);
            if (WHOLE)
                v[i] = __ldcg(p);
            else
                v[i] = col0 + 8 * c < a.hidden && t >= 0 ? __ldcg(p) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto cast = [&](auto whole, int64_t col0, uint8_t* sq) {
        constexpr bool WHOLE = decltype(whole)::value;
        const bool col_ok = WHOLE || col0 + 8 * c < a.hidden;
        uint8_t* q = q0 + col0;
#pragma unroll
        for (int i = 0; i < 8; ++i, q += q_step) {
            const int r = rg + 16 * i;
            uint2 q8;
            if constexpr (WEIGHTED) {
                // the product with the weight is a rounded fp32 value: it is
                // what amax is taken of and what the scale multiplies; a
                // padding row's weight and x are 0
                const float w = weight[r];
                const uint32_t word[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float lo, hi;
                    dev::mul2_rn(dev::bf16_lo(word[e]), dev::bf16_hi(word[e]), w, lo, hi);
                    most = max_bits(max_bits(most, lo), hi);
                    dev::mul2_rn(lo, hi, scale, lo, hi);
                    h[e] = dev::cvt_fp8x2<FMT>(lo, hi);
                }
                q8 = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
            } else {
                most = dev::absmax_pair(most, v[i].x);
                most = dev::absmax_pair(most, v[i].y);
                most = dev::absmax_pair(most, v[i].z);
                most = dev::absmax_pair(most, v[i].w);
                q8 = dev::cast8<FMT>(v[i], scale);
            }
            if (WHOLE || (col_ok && row0 + r < a.rows)) __stcs(reinterpret_cast<uint2*>(q), q8);
            if constexpr (TRANSPOSE)
                *reinterpret_cast<uint2*>(sq + r * 128 + ((2 * c) ^ dev::swz(r)) * 4) = q8;
        }
    };
    auto is_whole = [&](int ct) { return whole_rows && int64_t(ct + 1) * 128 <= a.hidden; };
    auto load_tile = [&](int ct) {
        if (is_whole(ct))
            load(std::true_type{}, int64_t(ct) * 128);
        else
            load(std::false_type{}, int64_t(ct) * 128);
    };
    load_tile(first);
    for (int ct = first; ct < last; ++ct) {
        const int64_t col0 = int64_t(ct) * 128;
        const bool whole = is_whole(ct), more = ct + 1 < last;
        uint8_t* sq = sq2[ct & 1];
        if (whole)
            cast(std::true_type{}, col0, sq);
        else
            cast(std::false_type{}, col0, sq);
        if (more) load_tile(ct + 1);
        if constexpr (TRANSPOSE) {
            // once a tile: whoever overwrites this copy, two tiles on, has
            // passed the next tile's barrier, and so has everyone's reading
            __syncthreads();
            const uint32_t* sq32 = reinterpret_cast<const uint32_t*>(sq);
            uint32_t in[16], o[4][4];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int r = 16 * b + j;
                in[j] = sq32[r * 32 + (w4 ^ dev::swz(r))];
            }
#pragma unroll
            for (int g = 0; g < 4; ++g)
                dev::transpose4x4(in[4 * g], in[4 * g + 1], in[4 * g + 2], in[4 * g + 3], o[0][g],
                                  o[1][g], o[2][g], o[3][g]);
            uint8_t* t = t0 + col0 * a.rows;
#pragma unroll
            for (int k = 0; k < 4; ++k, t += a.rows)
                if (whole || (row0 + 16 * b < a.rows && col0 + 4 * w4 + k < a.hidden))
                    __stcs(reinterpret_cast<uint4*>(t), make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]));
        }
    }
    most = __reduce_max_sync(0xFFFFFFFFu, WEIGHTED ? most : dev::pair_to_f32_bits(most));
    if (lane == 0) warp_max[warp] = most;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int i = 1; i < kCastThreads / 32; ++i) most = max(most, warp_max[i]);
        if (most) atomicMax(reinterpret_cast<unsigned*>(a.amax), most);
        if (blockIdx.x == 0) *a.scale_inv = __fdiv_rn(1.0f, scale);
    }
}

// Any shape and alignment, without the transpose: one block per sorted row.
// G = 2: columns in pairs (hidden even, x 4-byte and out 2-byte aligned).
template <int FMT, int G>
__global__ void __launch_bounds__(kCastThreads) sorted_cast_any_kernel(const SortedCastArgs a) {
    __shared__ unsigned warp_max[kCastThreads / 32];
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const float scale = *a.scale;
    float w;
    const int t = token_of(a, row, w);
    unsigned most = 0;
    for (int item = tid;; item += kCastThreads) {
        const dev::Cols<G> c(item, static_cast<int>(a.hidden));
        if (!c.any()) break;
        float f[8];
        if (t >= 0) {
            dev::load_cols<G>(reinterpret_cast<const __nv_bfloat16*>(a.x) + t * a.hidden, c, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (a.weights) f[j] = __fmul_rn(w, f[j]);
                if (c.has(j)) most = max_bits(most, f[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.0f;
        }
        uint8_t* q = a.out + row * a.hidden;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const uint32_t two = dev::cvt_fp8x2<FMT>(__fmul_rn(f[j], scale), __fmul_rn(f[j + 1], scale));
            if constexpr (G == 2) {
                if (c.has(j)) *reinterpret_cast<uint16_t*>(q + c.at(j)) = static_cast<uint16_t>(two);
            } else {
                if (c.has(j)) q[c.at(j)] = static_cast<uint8_t>(two);
                if (c.has(j + 1)) q[c.at(j + 1)] = static_cast<uint8_t>(two >> 8);
            }
        }
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if ((tid & 31) == 0) warp_max[tid >> 5] = most;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int i = 1; i < kCastThreads / 32; ++i) most = max(most, warp_max[i]);
        if (most) atomicMax(reinterpret_cast<unsigned*>(a.amax), most);
        if (row == 0) *a.scale_inv = __fdiv_rn(1.0f, scale);
    }
}

bool at16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int FMT>
cudaError_t launch_fmt(const SortedCastArgs& a, cudaStream_t stream) {
    const bool fast = a.hidden % 8 == 0 && at16(a.x) && reinterpret_cast<uintptr_t>(a.out) % 8 == 0;
    const bool together = a.out_t && fast && a.rows % 16 == 0 && at16(a.out_t);
    cudaError_t e;
    if (fast) {
        const int tile_rows = static_cast<int>((a.rows + 127) / 128);
        const int tile_cols = static_cast<int>((a.hidden + 127) / 128);
        // Whole strips for as many full waves of blocks as there are, single
        // tiles for the rest, so that the last wave ends evenly: 16384x4x6144
        // 172.8 us with the sort, whole strips alone 174.4; 8192x2x4096
        // weighted 43.1 and 44.1.
        const int items = tile_rows * ((tile_cols + kStripTiles - 1) / kStripTiles);
        const int wave = 4 * sm_count(), whole_strips = items / wave * wave;
        const dim3 grid(static_cast<unsigned>(whole_strips + (items - whole_strips) * kStripTiles));
        auto* kernel = a.weights ? (together ? sorted_cast_kernel<FMT, true, true>
                                             : sorted_cast_kernel<FMT, true, false>)
                                 : (together ? sorted_cast_kernel<FMT, false, true>
                                             : sorted_cast_kernel<FMT, false, false>);
        e = launch_pdl(kernel, grid, dim3(kCastThreads), 0, stream, a, tile_rows, tile_cols,
                       whole_strips);
    } else {
        const bool pairs = a.hidden % 2 == 0 && reinterpret_cast<uintptr_t>(a.x) % 4 == 0 &&
                           reinterpret_cast<uintptr_t>(a.out) % 2 == 0;
        e = launch_pdl(pairs ? sorted_cast_any_kernel<FMT, 2> : sorted_cast_any_kernel<FMT, 1>,
                       dim3(static_cast<unsigned>(a.rows)), dim3(kCastThreads), 0, stream, a);
    }
    if (e != cudaSuccess || !a.out_t || together) return e;
    // rows that are no multiple of 16, or odd alignments: the byte transpose of
    // what was just written
    const bool aligned_t = a.rows % 16 == 0 && a.hidden % 16 == 0 && at16(a.out) && at16(a.out_t);
    return launch_transpose(a.out, a.rows, a.hidden, a.out_t, a.noop, aligned_t, stream);
}

}  // namespace

cudaError_t launch_sorted_cast(const SortedCastArgs& a, int fmt, cudaStream_t stream) {
    return fmt == 0 ? launch_fmt<0>(a, stream) : launch_fmt<1>(a, stream);
}

}  // namespace ct
