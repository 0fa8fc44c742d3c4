// ct_dropout.cu -- dropout of a matrix by a counter-based generator.
//
// Each element is read and written once: HBM bounds fp32, and nearly 16-bit types,
// whose eight columns to a call of the generator cost some 110 instructions, 140
// where rows are not whole groups.  Measured, one GB300, of the measured copy rate:
// 8192x6144 fp32 61.7 us (0.96), 8192x12288 bf16 63.7 us (403 MB, 0.93),
// 8191x12287 bf16 71.1 us (0.83; instructions issue on 65% of the cycles),
// 8191x6145 fp32 62.6 (0.95).
#include "ct_device.cuh"
#include "ct_dropout.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"
#include "ct_vec.cuh"

#include <algorithm>

namespace ct {
namespace {

constexpr int kDropThreads = 256;

// The generator with its rounds' keys at hand: these kernels have the registers.
struct Keyed {
    Drops drops;
    uint2 keys[kPhiloxRounds];

    __device__ __forceinline__ explicit Keyed(const DropArgs& a) : drops(a) {
#pragma unroll
        for (int i = 0; i < kPhiloxRounds; ++i)
            keys[i] = make_uint2(drops.key.x + i * kKeyStep0, drops.key.y + i * kKeyStep1);
    }
    __device__ __forceinline__ uint4 words(uint32_t row, uint32_t group) const {
        uint4 c = make_uint4(group, row, drops.site, drops.step);
#pragma unroll
        for (int i = 0; i < kPhiloxRounds; ++i) c = philox_round(c, keys[i].x, keys[i].y);
        return c;
    }
    __device__ __forceinline__ uint32_t kept8(uint32_t row, uint32_t group) const {
        return Drops::bits(words(row, group), drops.cut);
    }
};

// Eight elements, kept where their bit is set.
template <typename T>
__device__ __forceinline__ dev::Raw8<T> dropped8(const dev::Raw8<T>& raw, uint32_t kept, float scale) {
    float f[8];
    dev::unpack8(raw, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (kept >> j) & 1 ? f[j] * scale : 0.0f;
    return dev::pack8(f, T{});
}

// Rows of whole groups in 16-byte-aligned buffers: a block takes consecutive groups,
// a thread ITEMS at a time, whose loads are in flight together, `rounds` times: four
// twice, or one once where that would not fill the GPU.
constexpr int kDropItems = 4, kDropRounds = 2;

template <typename T, int ITEMS>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const DropoutArgs a, int64_t groups, int rounds) {
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const Keyed keyed(a.drop);
    constexpr int step = kDropThreads;
    const T* x = static_cast<const T*>(a.x);
    T* out = static_cast<T*>(a.out);
    int64_t g0 = int64_t(blockIdx.x) * (rounds * (ITEMS * step)) + threadIdx.x;
    // the row of a group, and its number there
    const uint32_t row_groups = static_cast<uint32_t>(a.cols / 8);
    const uint32_t step_rows = step / row_groups, step_cols = step - step_rows * row_groups;
    uint32_t row = static_cast<uint32_t>((groups >> 32) == 0 ? uint32_t(g0) / row_groups : g0 / row_groups);
    uint32_t col = static_cast<uint32_t>(g0 - int64_t(row) * row_groups);
#pragma unroll 1
    for (int round = 0; round < rounds && g0 < groups; ++round, g0 += ITEMS * step) {
        dev::Raw8<T> raw[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) raw[i] = dev::load8(x + 8 * min(g0 + i * step, groups - 1));
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int64_t g = g0 + i * step;
            if (g >= groups) break;
            if (keyed.drops.some) {
                const uint4 r = keyed.words(row, col);
                const uint32_t w[4] = {r.x, r.y, r.z, r.w};
                float f[8];
                dev::unpack8(raw[i], f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[2 * j] = (w[j] << 16) >= keyed.drops.cut ? f[2 * j] * keyed.drops.scale : 0.0f;
                    f[2 * j + 1] = w[j] >= keyed.drops.cut ? f[2 * j + 1] * keyed.drops.scale : 0.0f;
                }
                raw[i] = dev::pack8(f, T{});
            }
#pragma unroll
            for (int v = 0; v < int(sizeof(T) / 2); ++v) reinterpret_cast<uint4*>(out + 8 * g)[v] = raw[i].v[v];
            row += step_rows;
            col += step_cols;
            if (col >= row_groups) {
                col -= row_groups;
                ++row;
            }
        }
    }
}

// Other rows, where x and out lie alike in their 16 bytes: the matrix as one array
// of aligned vectors of eight elements, whichever rows and groups they lie in.  A
// vector that begins s columns into its group needs the bits of that group and of
// the next, which is the one that the next vector begins in: a lane makes the bits
// of one group and takes the others from the lane after it.  A warp walks over
// steps * 32 vectors, so that the last lane finds its neighbour in the step after
// (which costs one step's bits in `steps`).  Only a vector with the end of a row in
// it may need a group of its own.
constexpr int kFlatSteps = 16, kFlatFewSteps = 8;
constexpr int kFlatMinCols = 256;       // so that 32 vectors have at most one end of a row

template <typename T>
__global__ void __launch_bounds__(kDropThreads)
    dropout_flat_kernel(const DropoutArgs a, int head, int64_t vectors, int steps) {
    constexpr int kFlatBatch = sizeof(T) == 4 ? 2 : 4;      // loads of a lane in flight, 16 registers
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const Keyed keyed(a.drop);
    const float scale = keyed.drops.scale;
    const int lane = threadIdx.x & 31, cols = static_cast<int>(a.cols);
    const T* x = static_cast<const T*>(a.x) + head;
    T* out = static_cast<T*>(a.out) + head;
    const int64_t q0 = (int64_t(blockIdx.x) * (kDropThreads / 32) + (threadIdx.x >> 5)) * 32 * steps;
    if (q0 < vectors) {
        const int64_t first = head + 8 * (q0 + lane);
        uint32_t row = static_cast<uint32_t>((first >> 32) == 0 ? uint32_t(first) / uint32_t(cols) : first / cols);
        int col = static_cast<int>(first - int64_t(row) * cols);
        uint32_t own = keyed.kept8(row, col >> 3);
#pragma unroll 1
        for (int u0 = 0; u0 < steps; u0 += kFlatBatch) {
            const int64_t q = q0 + 32 * u0 + lane;
            if (q - lane >= vectors) break;
            dev::Raw8<T> raw[kFlatBatch];
#pragma unroll
            for (int i = 0; i < kFlatBatch; ++i) raw[i] = dev::load8(x + 8 * min(q + 32 * i, vectors - 1));
#pragma unroll
            for (int i = 0; i < kFlatBatch; ++i) {
                const int end = cols - col;              // elements of this vector's row from its first on
                uint32_t next_row = row;
                int next_col = col + 256;
                if (next_col >= cols) {
                    next_col -= cols;
                    ++next_row;
                }
                const uint32_t ahead = keyed.kept8(next_row, next_col >> 3);
                const uint32_t after = __shfl_sync(0xFFFFFFFFu, lane == 0 ? ahead : own, (lane + 1) & 31);
                const int s = col & 7;
                uint32_t kept = (own | after << 8) >> s;
                if (end <= 8) {                          // the next vector is in the next row
                    uint32_t second = 0;
                    if (s + end > 8) second = keyed.kept8(row, (col >> 3) + 1);
                    kept = (((own | second << 8) >> s) & ((1u << end) - 1)) | after << end;
                }
                if (q + 32 * i < vectors) {
                    const dev::Raw8<T> r = dropped8<T>(raw[i], kept, scale);
#pragma unroll
                    for (int v = 0; v < int(sizeof(T) / 2); ++v)
                        reinterpret_cast<uint4*>(out + 8 * (q + 32 * i))[v] = r.v[v];
                }
                own = ahead;
                row = next_row;
                col = next_col;
            }
        }
    }
    // the elements before the first vector and after the last
    const int64_t n = a.rows * a.cols, rest = n - 8 * vectors;
    if (blockIdx.x == 0 && threadIdx.x < rest) {
        const int64_t e = int(threadIdx.x) < head ? threadIdx.x : 8 * vectors + threadIdx.x;
        const int64_t r = e / a.cols;
        const int c = static_cast<int>(e - r * a.cols);
        const bool kept = (keyed.kept8(static_cast<uint32_t>(r), c >> 3) >> (c & 7)) & 1;
        const float v = dev::to_f32(static_cast<const T*>(a.x)[e]);
        dev::from_f32(static_cast<T*>(a.out)[e], kept ? v * scale : 0.0f);
    }
}

// Anything else: a thread takes eight columns of a row, a warp's 32 apart.
template <typename T>
__global__ void __launch_bounds__(kDropThreads) dropout_general_kernel(const DropoutArgs a, int64_t items) {
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const Drops drops(a.drop);
    const int64_t first = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / 32 * 32;
    const int lane = threadIdx.x & 31;
    const int64_t row_items = (a.cols + 255) / 256 * 32;
    for (int64_t i = first; i < items; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t row = i / row_items;
        const int vi = static_cast<int>(i - row * row_items) + lane;
        const dev::Cols<1> c(vi, static_cast<int>(a.cols));
        dev::RawCols<1, T> raw;
        raw.load(static_cast<const T*>(a.x) + row * a.cols, c);
        float f[8];
        raw.get(f);
        if (drops.some) drops.apply<1>(static_cast<uint32_t>(row), vi, f);
        dev::store_cols<1>(static_cast<T*>(a.out) + row * a.cols, c, f);
    }
}

unsigned blocks_of(int64_t work, int64_t per_block) {
    return static_cast<unsigned>(std::max<int64_t>(1, (work + per_block - 1) / per_block));
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int dtype, cudaStream_t stream) {
    return by_types(dtype, dtype, [&](auto t, auto) {
        using T = decltype(t);
        const int64_t n = a.rows * a.cols;
        if (a.cols % 8 == 0 && all_aligned(a.x, a.out)) {
            // a group per thread: 64x4096 bf16 in 128 blocks, not 16
            if (n / 8 < int64_t(sm_count()) * kDropThreads * kDropItems * kDropRounds)
                return launch_pdl(dropout_kernel<T, 1>, dim3(blocks_of(n / 8, kDropThreads)), dim3(kDropThreads), 0,
                                  stream, a, n / 8, 1);
            return launch_pdl(dropout_kernel<T, kDropItems>,
                              dim3(blocks_of(n / 8, kDropThreads * kDropItems * kDropRounds)), dim3(kDropThreads), 0,
                              stream, a, n / 8, int(kDropRounds));
        }
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(a.x) % 16);
        if (a.drop.cut && a.cols >= kFlatMinCols && off == int(reinterpret_cast<uintptr_t>(a.out) % 16)) {
            const int head = static_cast<int>(std::min<int64_t>(n, (16 - off) % 16 / int(sizeof(T))));
            const int64_t vectors = (n - head) / 8;
            // fewer steps where the blocks would not fill the GPU twice: 16384x777
            // bf16 13.8 us against 17.4; 8191x12287 73.2 against 70.6
            const int steps = vectors < int64_t(sm_count()) * 8 * kDropThreads * kFlatSteps ? kFlatFewSteps : kFlatSteps;
            return launch_pdl(dropout_flat_kernel<T>, dim3(blocks_of(vectors, kDropThreads * steps)),
                              dim3(kDropThreads), 0, stream, a, head, vectors, steps);
        }
        const int64_t items = a.rows * ((a.cols + 255) / 256 * 32);
        return launch_pdl(dropout_general_kernel<T>, dim3(std::min(blocks_of(items, kDropThreads), unsigned(sm_count()) * 8)), dim3(kDropThreads), 0,
                          stream, a, items);
    });
}

}  // namespace ct
