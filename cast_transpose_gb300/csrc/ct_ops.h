// ct_ops.h -- kernel arguments and launchers of the expert-movement and
// block-norm operators.  Not installed.
#pragma once

#include "ct_internal.h"

#include <stddef.h>

namespace ct {

// SMs of the device of the first call (152 without one).
inline int sm_count() {
    static const int count = [] {
        int device = 0, n = 0;
        if (cudaGetDevice(&device) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) {
            cudaGetLastError();
            return 152;
        }
        return n;
    }();
    return count;
}

constexpr int kMaxExperts = 1024;      // of moe_sort

struct SortArgs {
    const void* idx;       // [n] int32, or int64 (index64)
    int64_t n, rows;
    int* row_of;           // [n]
    int* src;              // [rows]
    int* offsets;          // [experts + 1]
    int* counts;           // [experts]
    const float* noop;
    int experts, align, index64;
    int expert_bits;       // experts <= 2^expert_bits
};
size_t sort_workspace(int64_t n, int experts);
cudaError_t launch_moe_sort(const SortArgs& a, void* workspace, cudaStream_t stream);

// One struct for the movements between token and expert order.
struct MoveArgs {
    const void* x;         // [tokens, hidden]: dispatch's x, combine_backward's dout
    const void* ys;        // [rows, hidden] read: combine, combine_backward
    void* sorted;          // [rows, hidden] written: dispatch's out, combine_backward's dys
    void* out;             // [tokens, hidden] written: combine
    const int* row_of;     // [tokens, topk]
    const int* src;        // [rows]
    const float* weights;  // [tokens, topk], or null
    float* dweights;       // [tokens, topk], or null
    const float* noop;
    int64_t tokens, rows, hidden;
    int topk, elem_bytes;
};
// Launches that write sorted rows have a block per token, and before those one
// per kPadRows rows.
constexpr int kPadRows = 32;
inline int64_t pad_blocks(int64_t rows) { return (rows + kPadRows - 1) / kPadRows; }
cudaError_t launch_moe_dispatch(const MoveArgs& a, cudaStream_t stream);
cudaError_t launch_moe_combine(const MoveArgs& a, int dtype, cudaStream_t stream);
cudaError_t launch_moe_combine_backward(const MoveArgs& a, int dtype, cudaStream_t stream);

struct SortedCastArgs {
    const uint16_t* x;     // [tokens, hidden]
    const int* src;        // [rows]
    const float* weights;  // [tokens, topk], or null
    const float* scale;
    float* amax;
    float* scale_inv;
    uint8_t* out;          // [rows, hidden]
    uint8_t* out_t;        // [hidden, rows], or null
    const float* noop;
    int64_t tokens, rows, hidden;
    int topk;
};
cudaError_t launch_sorted_cast(const SortedCastArgs& a, int fmt, cudaStream_t stream);

struct NormArgs {
    const void *u, *res, *w_post, *w_pre, *gate;
    void *res_out, *y;
    float *rstd_post, *rstd_pre;
    const float* scale;    // not null: y is FP8
    float* amax;
    float* scale_inv;
    const float* noop;
    int64_t rows, rows_per_gate;
    float eps, branch_scale, residual_scale, weight_offset;
    int hidden, param_f32, post, pre, fmt;
};
cudaError_t launch_block_norm(const NormArgs& a, int dtype, int res_dtype, cudaStream_t stream);

struct NormBackwardArgs {
    const void *dy, *dres_out, *u, *res_out, *w_post, *w_pre, *gate;
    const float *rstd_post, *rstd_pre;
    void *du, *dres, *dw_post, *dw_pre, *dgate;
    float* workspace;
    const float* noop;
    int64_t rows, rows_per_gate;
    float branch_scale, residual_scale, weight_offset;
    int hidden, param_f32, post, pre;
};
size_t norm_backward_workspace(int64_t rows, int64_t hidden);
cudaError_t launch_block_norm_backward(const NormBackwardArgs& a, int dtype, int res_dtype,
                                       cudaStream_t stream);

// The block-norm kernels' own diagnostic word, as read_device_error.
cudaError_t read_norm_error(unsigned* value, bool clear);
// Their give-up path: `blocks` blocks of 64 threads, of which `thread` of the
// first one gives up.
cudaError_t launch_norm_wait_selftest(int blocks, int thread, uint32_t limit_us, cudaStream_t stream);

}  // namespace ct
