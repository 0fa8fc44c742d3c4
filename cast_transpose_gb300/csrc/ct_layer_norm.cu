// ct_layer_norm.cu -- the junction between two blocks whose norm is a layer
// norm: the branch's dropout, the residual sum and the norm, forward and
// backward.
//
// Forward reads u and res and writes res_out and y, backward reads dy, res_out and
// dres_out and writes dres and du: HBM would bound both, if the work on a column
// were less.  A row takes two sums over its columns before anything of y or dres is
// known, and a dropout some 11 instructions a column for its random bits alone.
// Measured, one GB300, bf16, p = 0.1, of the measured copy rate: forward 8191x6144
// 75.4 us (403 MB, 0.79; without dropout 70, 0.84), 8192x12288 152 (0.78; 127,
// 0.93), backward with its join 8192x12288 173.7 us (1007 MB, 0.85), 8191x6144 94
// (0.79).  Instructions issue on 60 to 65% of the cycles; warps wait little for
// memory.  So:
//   - rows come by asynchronous copies into rings of shared memory, stages ahead,
//     so that no register holds what has not arrived and no warp waits for it;
//   - a row takes one exchange between its warps and one barrier, two slots in turn
//     (a forward pass that began the next row before it, so that the barrier found
//     every warp with work left, was slower: 8191x6144 83 us);
//   - arithmetic on pairs of columns, 16 to 32 columns a thread.
// Launches of fewer rows than blocks fit take a kernel of a block per row, those
// whose rows are not aligned to 16 bytes, too; its backward pass sums columns in a
// kernel of its own.
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
    // with PER = 1 everything is on its way before the first of it is used
    constexpr bool AHEAD = PER == 1;
    dev::RawCols<G, R> res[PER];
    dev::RawCols<G, T> u[PER];
    float v[PER][8], w[8], b[8];
    float sum = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        res[p].load(static_cast<const R*>(a.res) + at, cols(p));
        if (a.u) u[p].load(static_cast<const T*>(a.u) + at, cols(p));
    }
    if (AHEAD) {
        load_param<T>(a.weight, a.param_f32, 0, a.weight_offset, cols(0), w);
        load_bias<T>(a.bias, a.param_f32, 0, cols(0), b);
    }
    const Drops drops(a.drop);
    const float scale = a.scale ? *a.scale : 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        res[p].get(v[p]);
        if (a.u) {
            float f[8];
            u[p].get(f);
            if (drops.some) drops.apply<G>(static_cast<uint32_t>(row), p * blockDim.x + tid, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[p][j] += f[j];
            dev::store_cols<G>(static_cast<R*>(a.res_out) + at, cols(p), v[p]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[p][j] = cols(p).has(j) ? v[p][j] : 0.0f;
            sum += v[p][j];
        }
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
    unsigned most = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        if (!AHEAD) {
            load_param<T>(a.weight, a.param_f32, 0, a.weight_offset, cols(p), w);
            load_bias<T>(a.bias, a.param_f32, 0, cols(p), b);
        }
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
    constexpr bool AHEAD = PER == 1;
    dev::RawCols<G, T> dy[PER];
    dev::RawCols<G, R> res[PER], down[AHEAD ? PER : 1];
    float g[PER][8], x[PER][8];
    float sum_g = 0.0f, sum_gx = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        dy[p].load(static_cast<const T*>(a.dy) + at, cols(p));
        res[p].load(static_cast<const R*>(a.res_out) + at, cols(p));
        if (AHEAD && a.dres_out) down[p].load(static_cast<const R*>(a.dres_out) + at, cols(p));
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        float w[8];
        load_param<T>(a.weight, a.param_f32, 0, a.weight_offset, cols(p), w);
        dy[p].get(g[p]);
        res[p].get(x[p]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool has = cols(p).has(j);
            x[p][j] = has ? (x[p][j] - mean) * rstd : 0.0f;
            g[p][j] = has ? g[p][j] * w[j] : 0.0f;
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
        if (a.dres_out) {
            if (!AHEAD) down[0].load(static_cast<const R*>(a.dres_out) + at, cols(p));
            down[AHEAD ? p : 0].get(d);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, g[p][j] - level - x[p][j] * along, d[j]);
        dev::store_cols<G>(static_cast<R*>(a.dres) + at, cols(p), d);
        if (!a.du) continue;
        if (drops.some) drops.apply<G>(static_cast<uint32_t>(row), p * blockDim.x + tid, d);
        dev::store_cols<G>(static_cast<T*>(a.du) + at, cols(p), d);
    }
}

// ---- many rows -----------------------------------------------------------------
// A block takes every gridDim.x-th row, a thread PER vectors of eight columns.
// Rows arrive in a ring of shared-memory stages by asynchronous copies that are
// issued stages ahead; a thread copies what it will read itself, so that no
// barrier is needed for it.
//
// SHIFT: rows that are not whole vectors, in 16-byte-aligned tensors.  Row r begins
// s = r H mod 8 columns after an aligned vector, in every tensor alike, and with
// gridDim.x a multiple of 8 that is the same s for all of a block's rows.  So the
// vectors are taken where they are aligned, s columns before the row's first: a
// thread keeps its columns from row to row, and only the vectors at the row's ends
// are not whole.
// Threads of an SM, and of a block at most: with 80 registers each, or 128 in the
// shifted backward pass, or 168 with four vectors.  (What does not fit goes through
// L2: nearly all of the SM's memory is the ring's.  Backward with two vectors and 80
// registers, of which 16 bytes do not: 8192x12288 190 us, so: 174.)  Forward, bf16,
// p = 0.1, us, at 8191x6144, 8192x8192 and 8192x6144 with an fp32 residual:
//   two vectors, 80 registers       75    113   121
//   three, 128 (512 threads)        74    118   123
//   three, 96 (640; 32 bytes out)  100    181   150
//   four, 168                       74    120   131
constexpr int ring_threads(int per, bool more) { return per == 4 ? 384 : per == 2 && more ? 512 : 768; }
// Short shifted rows, few to a block: with one vector per thread a row's way through
// the backward pass is shorter, though its warps do more besides the columns.  us,
// one vector against two (bf16; fp16 with an fp32 residual):
//            4099 rows                  16384 rows
//   259    17.4, 18.9; 18.3, 19.7     37.6, 35.3; 39.8, 42.4
//   515    19.6, 20.6; 21.4, 25.2     48.4, 52.4; 52.2, 66.4
//   777    21.6, 22.6; 23.9, 26.5     59.4, 51.8; 66.0, 67.0
//  1001    23.0, 25.4; 26.3, 28.5     60.3, 54.6; 69.6, 73.0
// Six rows are where the slower widths change over (12000x777 bf16 45.8, 41.9; 515
// columns never do).  With up to 2432 rows of less than 512 columns a block per row
// would be faster (2000x259 8.9, so 13.1): not in the rule.
constexpr int kFewRows = 6, kFewColumns = 1024 - 7;
// Rows of whole vectors that fit a warp (ONE) need no exchange between warps: up to
// 512 columns with two vectors per thread and, where the exchange is most of the
// rest, in the backward pass, 1024 with four.  Blocks of an SM, by their registers
// (more blocks with fewer are slower: backward 16384x1024 37.8 us with 8, 50.5 with
// 12; two warps per row 45.7).
constexpr int one_blocks(int per, bool sums) { return per == 4 ? 8 : sums ? 12 : 16; }
constexpr int kOneRows = 4;             // of a block with four vectors, at least: 2048x1024 17.0 us, else 16.0
constexpr int ring_block(int per, bool one, bool more) { return one ? 32 : ring_threads(per, more); }
constexpr int kRingStages = 4;                  // at most
constexpr int kRingSmem = 226 * 1024;           // of an SM's blocks together
constexpr int kShiftRows = 8;

// How a launch of many rows is divided.
struct RingShape {
    int per, threads, blocks;           // blocks 0: not a launch of many rows
    int stages;
    bool one;                           // a warp per row
    bool once;                          // backward: dres_out has one place beside the stages
    size_t smem;
};

// Eight columns from `first` on, of which some may lie outside [0, H).
template <bool SHIFT>
struct Vec {
    int first, H;
    __device__ __forceinline__ bool any() const { return first < H; }
    __device__ __forceinline__ bool whole() const { return SHIFT ? first >= 0 && first + 8 <= H : first < H; }
    __device__ __forceinline__ bool has(int j) const { return SHIFT ? unsigned(first + j) < unsigned(H) : first < H; }

    template <typename T>
    __device__ __forceinline__ void store(T* row, const V8& v) const {
        float f[8];
        floats(v, f);
        if (whole()) {
            dev::store8(row + first, f);
        } else if (SHIFT) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (has(j)) dev::from_f32(row[first + j], f[j]);
        }
    }
    __device__ __forceinline__ void store_codes(uint8_t* row, const float (&f)[8], float scale, int fmt) const {
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = __fmul_rn(f[2 * j], scale), hi = __fmul_rn(f[2 * j + 1], scale);
            h[j] = fmt == 0 ? dev::cvt_fp8x2<0>(lo, hi) : dev::cvt_fp8x2<1>(lo, hi);
        }
        if (whole()) {
            *reinterpret_cast<uint2*>(row + first) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
        } else if (SHIFT) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (has(j)) row[first + j] = static_cast<uint8_t>(h[j >> 1] >> (8 * (j & 1)));
        }
    }
    // A parameter's columns, `none` where there is no parameter.
    template <typename T>
    __device__ __forceinline__ V8 param(const void* p, int f32, float offset, float none) const {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = none;
        if (p) {
            if constexpr (SHIFT) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (has(j))
                        f[j] = offset + (f32 ? static_cast<const float*>(p)[first + j]
                                             : dev::to_f32(static_cast<const T*>(p)[first + j]));
            } else {
                load_param<T>(p, f32, 0, offset, dev::Cols<8>(first / 8, H), f);
            }
        }
        return pairs(f);
    }
    // 0 outside the row.  Without SHIFT a vector that is outside is so as a whole,
    // and adds nothing by sum().
    __device__ __forceinline__ void cut(V8& v) const {
        if (!SHIFT || whole()) return;
        float f[8];
        floats(v, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = has(j) ? f[j] : 0.0f;
        v = pairs(f);
    }
    __device__ __forceinline__ float sum(uint64_t part) const { return SHIFT || any() ? lanes_sum(part) : 0.0f; }
};

// A tensor's rows in the ring.
template <typename T, bool SHIFT, int PER>
struct Staged {
    const T* base;          // null: left out
    int64_t rows;
    int H, shift;
    static constexpr int kWords = sizeof(T) / 2;        // 16-byte words of a vector

    static __host__ __device__ constexpr uint32_t bytes(int threads) { return threads * PER * 16 * kWords; }
    __device__ __forceinline__ void fetch(uint8_t* stage, int64_t row) const {
        if (!base) return;
        const int tid = threadIdx.x, n = blockDim.x;
        // a row's last vector may go on for seven elements after it
        const bool inside = !SHIFT || (rows - 1 - row) * H >= 7;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            int first = (p * n + tid) * 8 - shift;
            if (first >= H) first = -shift;             // any place will do
            const int64_t at = row * H + first;
            const uint8_t* from = reinterpret_cast<const uint8_t*>(base + at);
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                uint8_t* to = stage + ((p * kWords + w) * n + tid) * 16;
                if (inside) {
                    dev::cp_async16(to, from + 16 * w, 16);
                } else {                                // no more than what the tensor has
                    const int64_t left = (rows * H - at) * int64_t(sizeof(T)) - 16 * w;
                    dev::cp_async16(to, left > 0 ? from + 16 * w : reinterpret_cast<const uint8_t*>(base),
                                    left > 0 ? static_cast<int>(min(left, int64_t(16))) : 0);
                }
            }
        }
    }
    __device__ __forceinline__ V8 get(const uint8_t* stage, int p) const {
        dev::Raw8<T> r;
        float f[8];
#pragma unroll
        for (int w = 0; w < kWords; ++w)
            r.v[w] = *reinterpret_cast<const uint4*>(stage + ((p * kWords + w) * blockDim.x + threadIdx.x) * 16);
        dev::unpack8(r, f);
        return pairs(f);
    }
};

// Drops columns of the thread's vectors of a row.  Vector i begins `shift` columns
// before group i: it takes the last bits of group i - 1, from the lane before or, as
// the warp's first, from a lane that made them besides.  The whole warp has to call
// it.
template <bool SHIFT, int PER>
struct RowDrops {
    const Drops& drops;
    uint32_t row;
    int shift;
    uint32_t before;        // lane p: the bits of the group before the warp's vector p

    __device__ __forceinline__ RowDrops(const Drops& drops_, int64_t row_, int shift_)
        : drops(drops_), row(static_cast<uint32_t>(row_)), shift(shift_), before(0) {
        if (!SHIFT || !shift) return;
        const int lane = threadIdx.x & 31, p = lane < PER ? lane : 0;
        before = Drops::bits(drops.words(row, p * blockDim.x + (threadIdx.x - lane) - 1), drops.cut);
    }
    __device__ __forceinline__ void apply(int p, V8& v) const {
        const int item = p * blockDim.x + threadIdx.x;
        float f[8];
        floats(v, f);
        if (!SHIFT || !shift) {
            drops.apply<8>(row, item, f);
        } else {
            const uint32_t own = Drops::bits(drops.words(row, item), drops.cut);
            const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, own, 1), first = __shfl_sync(0xFFFFFFFFu, before, p);
            const uint32_t kept = (((threadIdx.x & 31) == 0 ? first : up) | own << 8) >> (8 - shift);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = (kept >> j) & 1 ? f[j] * drops.scale : 0.0f;
        }
        v = pairs(f);
    }
};

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Waits for the thread's copies but those of the last `ahead` commits.
__device__ __forceinline__ void wait_copies(int ahead) {
    if (ahead == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (ahead == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (ahead == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (ahead == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else asm volatile("cp.async.wait_group 5;" ::: "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <bool SHIFT>
__device__ __forceinline__ int shift_of(int H) {
    return SHIFT ? static_cast<int>(int64_t(blockIdx.x) * H % kShiftRows) : 0;
}

// Forward.  The mean and the squares about it need one exchange: a warp leaves the
// sum S_w of its n_w columns and their squares Q_w about a number c_w next to its
// own mean, S_w times 1 / n_w, from which everyone gets
//   M2 = sum over warps of Q_w + (c_w - mean) (n_w (c_w - mean) + 2 (S_w - n_w c_w))
// without the cancellation of a difference of squares.  This holds for any c_w, so
// that its rounding adds nothing; S_w - n_w c_w is one fused multiply-add.  (Quotients
// S_w / n_w, for which the last term is 0, cost 4%: 8191x6144 78.8 us against 75.9.)
template <typename T, typename R, bool SHIFT, int PER, bool ONE>
__global__ void __launch_bounds__(ring_block(PER, ONE, false), ONE ? one_blocks(PER, false) : 1)
    layer_norm_kernel(const LayerNormArgs a, int stages) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 slots[2][32];
    __shared__ unsigned block_max;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, H = a.hidden;
    const int shift = shift_of<SHIFT>(H);
    auto vec = [&](int p) { return Vec<SHIFT>{int(p * blockDim.x + tid) * 8 - shift, H}; };
    if (tid == 0) block_max = 0;
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const Staged<R, SHIFT, PER> res{static_cast<const R*>(a.res), a.rows, H, shift};
    const Staged<T, SHIFT, PER> u{static_cast<const T*>(a.u), a.rows, H, shift};
    const uint32_t second = res.bytes(blockDim.x), stage_bytes = second + (a.u ? u.bytes(blockDim.x) : 0);
    auto fetch = [&](int64_t row, int to) {
        if (row < a.rows) {
            res.fetch(smem + to * stage_bytes, row);
            u.fetch(smem + to * stage_bytes + second, row);
        }
        commit_copies();
    };
    for (int i = 0; i + 1 < stages; ++i) fetch(blockIdx.x + int64_t(i) * gridDim.x, i);
    const Drops drops(a.drop);
    const float scale = a.scale ? *a.scale : 0.0f;
    V8 w[PER], b[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        w[p] = vec(p).template param<T>(a.weight, a.param_f32, a.weight_offset, 1.0f);
        b[p] = vec(p).template param<T>(a.bias, a.param_f32, 0.0f, 0.0f);
    }
    // columns of a warp that are inside the row: some, for every warp
    auto columns_of = [&](int of) {
        int n = 0;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int first = 256 * (p * warps + of) - shift;
            n += max(0, min(first + 256, H) - max(first, 0));
        }
        return static_cast<float>(n);
    };
    const float own_columns = columns_of(warp), lane_columns = lane < warps ? columns_of(lane) : 1.0f;
    const float per_own = 1.0f / own_columns, per_lane = 1.0f / lane_columns, per_column = 1.0f / H;
    unsigned most = 0;
    int stage = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t at = row * H;
        wait_copies(stages - 2);
        const uint8_t* here = smem + stage * stage_bytes;
        V8 v[PER];
        float sum_w = 0.0f, squares_w = 0.0f;
        if (a.u) {
            V8 x[PER];
#pragma unroll
            for (int p = 0; p < PER; ++p) x[p] = u.get(here + second, p);
            if (drops.some) {
                const RowDrops<SHIFT, PER> of(drops, row, shift);
#pragma unroll
                for (int p = 0; p < PER; ++p) of.apply(p, x[p]);
            }
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                v[p] = res.get(here, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[p].p[j] = add2(v[p].p[j], x[p].p[j]);
                vec(p).store(static_cast<R*>(a.res_out) + at, v[p]);
            }
        } else {
#pragma unroll
            for (int p = 0; p < PER; ++p) v[p] = res.get(here, p);
        }
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            vec(p).cut(v[p]);
            sum_w += vec(p).sum(add2(add2(v[p].p[0], v[p].p[1]), add2(v[p].p[2], v[p].p[3])));
        }
        // the stage before this one is free
        fetch(row + int64_t(stages - 1) * gridDim.x, stage == 0 ? stages - 1 : stage - 1);
        if (++stage == stages) stage = 0;
        sum_w = dev::warp_sum(sum_w);
        const float mean_w = ONE ? sum_w / H : __fmul_rn(sum_w, per_own);
        const uint64_t away = pair(-mean_w, -mean_w);
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            V8 d;
            uint64_t part = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) d.p[j] = add2(v[p].p[j], away);
            vec(p).cut(d);
#pragma unroll
            for (int j = 0; j < 4; ++j) part = fma2(d.p[j], d.p[j], part);
            squares_w += vec(p).sum(part);
        }
        squares_w = dev::warp_sum(squares_w);
        float mean = mean_w, squares = squares_w;
        if (!ONE) {
            if (lane == 0) slots[turn][warp] = make_float2(sum_w, squares_w);
            __syncthreads();
            const float2 other = lane < warps ? slots[turn][lane] : make_float2(0.0f, 0.0f);
            turn ^= 1;
            mean = dev::warp_sum(other.x) / H;
            // c of this lane's warp, as that has it; where there is none, no columns
            const float c = __fmul_rn(other.x, per_lane), left = fmaf(-lane_columns, c, other.x);
            const float apart = lane < warps ? c - mean : 0.0f;
            squares = max_nan(dev::warp_sum(fmaf(apart, fmaf(lane_columns, apart, left + left), other.y)), 0.0f);
        }
        const float rstd = rsqrtf(fmaf(squares, per_column, a.eps));
        if (tid == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        const uint64_t mean2 = pair(-mean, -mean), rstd2 = pair(rstd, rstd);
#pragma unroll
        for (int p = 0; p < PER; ++p) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[p].p[j] = fma2(mul2(add2(v[p].p[j], mean2), rstd2), w[p].p[j], b[p].p[j]);
            if (!a.scale) {
                vec(p).store(static_cast<T*>(a.y) + at, v[p]);
                continue;
            }
            float f[8];
            floats(v[p], f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (vec(p).has(j)) most = max(most, __float_as_uint(f[j]) & 0x7FFFFFFFu);
            vec(p).store_codes(static_cast<uint8_t*>(a.y) + at, f, scale, a.fmt);
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
// read from the stage a second time instead.  dres_out, which only the second half of
// a row's work needs, may have a single place, into which a thread copies the next
// row's as soon as it has read this one's (ONCE): where whole stages would be too few.
template <typename T, typename R, bool SHIFT, int PER, bool ONE, bool ONCE>
__global__ void __launch_bounds__(ring_block(PER, ONE, SHIFT), ONE ? one_blocks(PER, true) : 1)
    layer_norm_backward_kernel(const LayerNormBackwardArgs a, int stages) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 slots[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, H = a.hidden;
    const int shift = shift_of<SHIFT>(H);
    auto vec = [&](int p) { return Vec<SHIFT>{int(p * blockDim.x + tid) * 8 - shift, H}; };
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const Staged<R, SHIFT, PER> res{static_cast<const R*>(a.res_out), a.rows, H, shift};
    const Staged<R, SHIFT, PER> down{static_cast<const R*>(a.dres_out), a.rows, H, shift};
    const Staged<T, SHIFT, PER> dy{static_cast<const T*>(a.dy), a.rows, H, shift};
    const uint32_t second = res.bytes(blockDim.x), third = second + dy.bytes(blockDim.x);
    const uint32_t stage_bytes = third + (a.dres_out && !ONCE ? second : 0);
    auto fetch = [&](int64_t row, int to) {
        if (row < a.rows) {
            res.fetch(smem + to * stage_bytes, row);
            dy.fetch(smem + to * stage_bytes + second, row);
            if (!ONCE) down.fetch(smem + to * stage_bytes + third, row);
        }
        commit_copies();
    };
    auto fetch_down = [&](int64_t row) {
        if (!ONCE) return;
        if (row < a.rows) down.fetch(smem + stages * stage_bytes, row);
        commit_copies();
    };
    // the commits are those of the loop: a stage's and, with dres_out apart, its own
    for (int i = 0; i + 1 < stages; ++i) {
        fetch(blockIdx.x + int64_t(i) * gridDim.x, i);
        if (ONCE && i + 2 < stages) commit_copies();
    }
    fetch_down(blockIdx.x);
    const Drops drops(a.drop);
    V8 w[PER], dw[PER] = {}, db[PER] = {};
#pragma unroll
    for (int p = 0; p < PER; ++p)
        w[p] = vec(p).template param<T>(a.weight, a.param_f32, a.weight_offset, 1.0f);
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
        wait_copies(ONCE ? 2 * stages - 3 : stages - 2);
        const uint8_t* here = smem + stage * stage_bytes;
        // the stage before this one is free
        fetch(row + int64_t(stages - 1) * gridDim.x, stage == 0 ? stages - 1 : stage - 1);
        if (++stage == stages) stage = 0;
        const uint64_t mean2 = pair(-mean, -mean), rstd2 = pair(rstd, rstd);
        float one = 0.0f, two = 0.0f;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            V8 x = res.get(here, p), g = dy.get(here + second, p);
            uint64_t sum_g = 0, sum_gx = 0;
            vec(p).cut(x);
            vec(p).cut(g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t hat = mul2(add2(x.p[j], mean2), rstd2), gw = mul2(g.p[j], w[p].p[j]);
                dw[p].p[j] = fma2(g.p[j], hat, dw[p].p[j]);
                db[p].p[j] = add2(db[p].p[j], g.p[j]);
                sum_g = add2(sum_g, gw);
                sum_gx = fma2(gw, hat, sum_gx);
            }
            one += vec(p).sum(sum_g);
            two += vec(p).sum(sum_gx);
        }
        one = dev::warp_sum(one);
        two = dev::warp_sum(two);
        if (!ONE) {
            if (lane == 0) slots[turn][warp] = make_float2(one, two);
            __syncthreads();
            const float2 other = lane < warps ? slots[turn][lane] : make_float2(0.0f, 0.0f);
            turn ^= 1;
            one = dev::warp_sum(other.x);
            two = dev::warp_sum(other.y);
        }
        const float level = -one * per_column, along = -two * per_column;
        const uint64_t level2 = pair(level, level), along2 = pair(along, along);
        if (ONCE) wait_copies(1);
        const uint8_t* down_here = ONCE ? smem + stages * stage_bytes : here + third;
        const RowDrops<SHIFT, PER> of(drops, row, drops.some ? shift : 0);
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const V8 x = res.get(here, p), g = dy.get(here + second, p);
            V8 d = {};
            if (a.dres_out) d = down.get(down_here, p);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t hat = mul2(add2(x.p[j], mean2), rstd2);
                d.p[j] = fma2(rstd2, fma2(hat, along2, fma2(g.p[j], w[p].p[j], level2)), d.p[j]);
            }
            vec(p).store(static_cast<R*>(a.dres) + at, d);
            if (!a.du) continue;
            if (drops.some) of.apply(p, d);
            vec(p).store(static_cast<T*>(a.du) + at, d);
        }
        fetch_down(row + gridDim.x);
        mean = next_mean;
        rstd = next_rstd;
    }
    dev::pdl_launch_dependents();
    if (!a.dweight && !a.dbias) return;
    float* sums = a.workspace + 2 * int64_t(blockIdx.x) * H;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        float f[2][8];
        floats(dw[p], f[0]);
        floats(db[p], f[1]);
        if (!SHIFT && !vec(p).any()) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float* to = sums + k * H + vec(p).first;
            if constexpr (!SHIFT) {
                dev::store8(to, f[k]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (vec(p).has(j)) to[j] = f[k][j];
            }
        }
    }
}

// Threads of a block that holds a row of `hidden` columns, PER vectors of eight each.
int row_threads(int hidden, int per) { return (hidden + 256 * per - 1) / (256 * per) * 32; }
int row_per(int hidden) { return hidden <= 8192 ? 1 : hidden <= 16384 ? 2 : 4; }

// column_bytes: of a column in a stage, extra_bytes: of what may be once beside the
// stages instead; sums: the kernel keeps column sums; few: one vector per thread.
RingShape ring_shape(int64_t rows, int hidden, bool shifted, int column_bytes, int extra_bytes, bool sums,
                     bool few = false) {
    RingShape s = {};
    s.one = !shifted && (hidden <= 512 || (sums && hidden <= 1024 &&
                                           rows >= int64_t(kOneRows) * sm_count() * one_blocks(4, true)));
    s.per = sums && !shifted && hidden > 512 ? 4 : few ? 1 : 2;
    s.threads = row_threads(hidden + (shifted ? kShiftRows - 1 : 0), s.per);
    const int sm_threads = s.one ? 32 * one_blocks(s.per, sums) : ring_threads(s.per, sums && shifted);
    const int columns = s.threads * s.per * 8;
    if (s.threads > sm_threads) return s;
    for (int per_sm = sm_threads / s.threads; per_sm > 0; --per_sm) {
        const int room = kRingSmem / per_sm - 2048;
        s.once = false;
        s.stages = std::min(kRingStages, room / (columns * (column_bytes + extra_bytes)));
        if (s.stages < 3 && extra_bytes && !shifted && !s.one) {
            s.once = true;
            s.stages = std::min(kRingStages, (room - columns * extra_bytes) / (columns * column_bytes));
        }
        // A row ahead is enough where many blocks have one each, and forward, which is
        // done with a stage early (8192x6144 all fp32: two blocks with two 175 us, one
        // with four 199).
        if (s.stages < (!sums || s.once || s.one || per_sm == 1 ? 2 : 3)) continue;
        s.smem = size_t(columns) * (s.stages * (column_bytes + (s.once ? 0 : extra_bytes)) + (s.once ? extra_bytes : 0));
        int64_t blocks = int64_t(sm_count()) * per_sm;
        if (shifted) blocks = blocks / kShiftRows * kShiftRows;
        s.blocks = rows > blocks ? static_cast<int>(blocks) : 0;
        return s;
    }
    return s;
}

// The shapes of launches on 16-byte-aligned buffers.  column_bytes: of res and u;
// x_bytes: of dy; res_bytes: of res_out and, where it is given (down), of dres_out.
RingShape forward_shape(int64_t rows, int hidden, int column_bytes) {
    return ring_shape(rows, hidden, hidden % 8 != 0, column_bytes, 0, false);
}
RingShape backward_shape(int64_t rows, int hidden, int x_bytes, int res_bytes, bool down) {
    const bool shifted = hidden % 8 != 0;
    auto shape = [&](bool few) {
        return ring_shape(rows, hidden, shifted, res_bytes + x_bytes, down ? res_bytes : 0, true, few);
    };
    RingShape s = {};
    if (shifted && hidden <= kFewColumns) s = shape(true);
    if (rows >= int64_t(kFewRows) * s.blocks) s = shape(false);        // also where there are none
    return s;
}

// Launches a kernel of many rows for PER vectors per thread, which the shape has to
// be for; the first time on a device it is allowed its shared memory.
template <auto KERNEL, int PER, bool ONE, typename Args>
cudaError_t launch_ring(const RingShape& s, const Args& a, cudaStream_t stream) {
    if (s.per != PER || s.one != ONE || (ONE && s.threads != 32)) return cudaErrorInvalidValue;
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
// takes every so many-th part of 32 columns, kJoinBatch loads at a time.
constexpr int kJoinBatch = 16;

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
        for (int i = 0; i < kJoinBatch; ++i) v[i] = dev::load_now(from + 2 * int64_t(min(i0 + i * ways, parts - 1)) * H);
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) sum += i0 + i * ways < parts ? v[i] : 0.0f;
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || col >= H) return;
    for (int i = 1; i < ways; ++i) sum += sums[i][lane];
    set_param<T>(out, a.param_f32, col, sum);
}

int column_shares(int64_t rows, int64_t hidden) {
    const int64_t blocks = (hidden + 31) / 32;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((rows + 127) / 128, 600 / std::max<int64_t>(blocks, 1))));
}

// Blocks of a backward launch of many rows, at most: the workspace has room for them.
int64_t most_blocks(int64_t rows, int64_t hidden) {
    const int of_rings = ring_threads(2, false) / row_threads(static_cast<int>(std::max<int64_t>(hidden, 1)), 2);
    const int least = sm_count() / kShiftRows * kShiftRows;      // blocks of such a launch
    return rows > least ? std::min(rows, int64_t(sm_count()) * of_rings) : 0;
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, int dtype, int res_dtype, cudaStream_t stream) {
    const bool aligned = all_aligned(a.u, a.res, a.weight, a.bias, a.res_out, a.y), vec = aligned && a.hidden % 8 == 0;
    const int per = row_per(a.hidden);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        const RingShape s = aligned ? forward_shape(a.rows, a.hidden, sizeof(R) + (a.u ? sizeof(T) : 0)) : RingShape{};
        if (s.blocks > 0)
            return s.one ? launch_ring<layer_norm_kernel<T, R, false, 2, true>, 2, true>(s, a, stream)
                 : vec   ? launch_ring<layer_norm_kernel<T, R, false, 2, false>, 2, false>(s, a, stream)
                         : launch_ring<layer_norm_kernel<T, R, true, 2, false>, 2, false>(s, a, stream);
        auto* kernel = per == 1 ? (vec ? layer_norm_row_kernel<T, R, 8, 1> : layer_norm_row_kernel<T, R, 1, 1>)
                     : per == 2 ? (vec ? layer_norm_row_kernel<T, R, 8, 2> : layer_norm_row_kernel<T, R, 1, 2>)
                                : (vec ? layer_norm_row_kernel<T, R, 8, 4> : layer_norm_row_kernel<T, R, 1, 4>);
        return launch_pdl(kernel, dim3(static_cast<unsigned>(a.rows)), dim3(row_threads(a.hidden, per)), 0,
                          stream, a);
    });
}

LayerNormPlan layer_norm_plan(int64_t rows, int hidden, int x_bytes, int res_bytes, bool backward, bool with) {
    const RingShape s = backward ? backward_shape(rows, hidden, x_bytes, res_bytes, with)
                                 : forward_shape(rows, hidden, res_bytes + (with ? x_bytes : 0));
    if (s.blocks == 0) return {};
    return {s.blocks, s.per, s.stages, hidden % 8 != 0, s.one, s.once};
}

size_t layer_norm_backward_workspace(int64_t rows, int64_t hidden) {
    const int shares = column_shares(rows, hidden);
    const int64_t parts = std::max<int64_t>(shares > 1 ? shares : 0, most_blocks(rows, hidden));
    return (size_t(parts) * 2 * hidden * sizeof(float) + 15) / 16 * 16;
}

cudaError_t launch_layer_norm_backward(const LayerNormBackwardArgs& a, int dtype, int res_dtype,
                                       cudaStream_t stream) {
    const bool aligned = all_aligned(a.dy, a.dres_out, a.res_out, a.weight, a.dres, a.du);
    const bool vec = aligned && a.hidden % 8 == 0;
    const int per = row_per(a.hidden);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        const RingShape s = aligned ? backward_shape(a.rows, a.hidden, sizeof(T), sizeof(R), a.dres_out) : RingShape{};
        cudaError_t e = cudaSuccess;
        int parts;
        if (s.blocks > 0) {
            e = s.once ? launch_ring<layer_norm_backward_kernel<T, R, false, 4, false, true>, 4, false>(s, a, stream)
              : s.one  ? (s.per == 2 ? launch_ring<layer_norm_backward_kernel<T, R, false, 2, true, false>, 2, true>(s, a, stream)
                                     : launch_ring<layer_norm_backward_kernel<T, R, false, 4, true, false>, 4, true>(s, a, stream))
              : vec    ? launch_ring<layer_norm_backward_kernel<T, R, false, 4, false, false>, 4, false>(s, a, stream)
              : s.per == 1 ? launch_ring<layer_norm_backward_kernel<T, R, true, 1, false, false>, 1, false>(s, a, stream)
                           : launch_ring<layer_norm_backward_kernel<T, R, true, 2, false, false>, 2, false>(s, a, stream);
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
