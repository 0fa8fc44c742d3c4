// ct_moe_cast.cu -- rows gathered into expert order, weighted, cast to FP8 and
// transposed in one pass.
#include "ct_device.cuh"
#include "ct_ops.h"

namespace ct {
namespace {

constexpr int kThreads_ = 256;
constexpr int kPitch = 128 + 4;

// One 128x128 tile of the sorted matrix per block, any shape and alignment:
// element by element, with an FP8 copy in shared memory for the transpose.
template <int FMT>
__global__ void __launch_bounds__(kThreads_) sorted_cast_kernel(SortedCastArgs a, int tile_cols) {
    __shared__ uint8_t tile[128 * kPitch];
    __shared__ int slot_of[128];
    __shared__ unsigned amax_bits;
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int tid = threadIdx.x;
    const int64_t row0 = int64_t(blockIdx.x / tile_cols) * 128;
    const int64_t col0 = int64_t(blockIdx.x % tile_cols) * 128;
    const int rows = static_cast<int>(min(int64_t(128), a.rows - row0));
    const int cols = static_cast<int>(min(int64_t(128), a.hidden - col0));
    const float scale = *a.scale;
    if (tid < 128) {
        int s = tid < rows ? a.src[row0 + tid] : -1;
        if (s >= a.tokens * a.topk) s = -1;
        slot_of[tid] = s;
    }
    if (tid == 0) amax_bits = 0;
    __syncthreads();
    unsigned most = 0;
    for (int i = tid; i < 128 * 128; i += kThreads_) {
        const int r = i >> 7, c = i & 127;
        if (r >= rows || c >= cols) continue;
        const int s = slot_of[r];
        float v = 0.0f;
        if (s >= 0) {
            v = __uint_as_float(uint32_t(a.x[int64_t(s / a.topk) * a.hidden + col0 + c]) << 16);
            if (a.weights) v = __fmul_rn(a.weights[s], v);
            most = max(most, __float_as_uint(v) & 0x7FFFFFFFu);
        }
        const uint8_t q = static_cast<uint8_t>(dev::cvt_fp8x2<FMT>(__fmul_rn(v, scale), 0.0f));
        tile[r * kPitch + c] = q;
        a.out[(row0 + r) * a.hidden + col0 + c] = q;
    }
    atomicMax(&amax_bits, most);
    __syncthreads();
    if (a.out_t)
        for (int i = tid; i < 128 * 128; i += kThreads_) {
            const int c = i >> 7, r = i & 127;
            if (r < rows && c < cols) a.out_t[(col0 + c) * a.rows + row0 + r] = tile[r * kPitch + c];
        }
    if (tid == 0) {
        if (amax_bits) atomicMax(reinterpret_cast<unsigned*>(a.amax), amax_bits);
        if (blockIdx.x == 0) *a.scale_inv = __fdiv_rn(1.0f, scale);
    }
}

}  // namespace

cudaError_t launch_sorted_cast(const SortedCastArgs& a, int fmt, cudaStream_t stream) {
    const int tile_cols = static_cast<int>((a.hidden + 127) / 128);
    const int64_t tiles = (a.rows + 127) / 128 * tile_cols;
    auto* kernel = fmt == 0 ? sorted_cast_kernel<0> : sorted_cast_kernel<1>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(tiles)), dim3(kThreads_), 0, stream, a,
                      tile_cols);
}

}  // namespace ct
