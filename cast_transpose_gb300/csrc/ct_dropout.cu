// ct_dropout.cu -- dropout of a matrix by a counter-based generator.
#include "ct_device.cuh"
#include "ct_dropout.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"
#include "ct_vec.cuh"

#include <algorithm>

namespace ct {
namespace {

constexpr int kDropThreads = 256;

// A thread takes eight columns of a row.
template <typename T, int G>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const DropoutArgs a, int64_t items) {
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
        const dev::Cols<G> c(vi, static_cast<int>(a.cols));
        const T* x = static_cast<const T*>(a.x) + row * a.cols;
        T* out = static_cast<T*>(a.out) + row * a.cols;
        float f[8];
        dev::load_cols<G>(x, c, f);
        if (drops.some) drops.apply<G>(static_cast<uint32_t>(row), vi, f);
        dev::store_cols<G>(out, c, f);
    }
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int dtype, cudaStream_t stream) {
    const bool vec = a.cols % 8 == 0 && all_aligned(a.x, a.out);
    const int64_t items = a.rows * ((a.cols + 255) / 256 * 32);
    const int64_t blocks = std::min<int64_t>((items + kDropThreads - 1) / kDropThreads, int64_t(sm_count()) * 8);
    return by_types(dtype, dtype, [&](auto t, auto) {
        using T = decltype(t);
        return launch_pdl(vec ? dropout_kernel<T, 8> : dropout_kernel<T, 1>, dim3(static_cast<unsigned>(blocks)),
                          dim3(kDropThreads), 0, stream, a, items);
    });
}

}  // namespace ct
