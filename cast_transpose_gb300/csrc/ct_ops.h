// ct_ops.h -- kernel arguments and launchers of the operators around the FP8
// casts: expert movement, router, norms, dropout and embedding.  Not installed.
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

// A dropout: 16 random bits below `cut` drop an element, what stays is scaled.
struct DropArgs {
    const uint64_t* rng;   // seed and step; not read where cut is 0
    uint32_t site, cut;
    float scale;
};

struct DropoutArgs {
    DropArgs drop;
    const void* x;
    void* out;
    const float* noop;
    int64_t rows, cols;
};
cudaError_t launch_dropout(const DropoutArgs& a, int dtype, cudaStream_t stream);

struct LayerNormArgs {
    DropArgs drop;
    const void *u, *res, *weight, *bias;
    void *res_out, *y;
    float *mean, *rstd;
    const float* scale;    // not null: y is FP8
    float* amax;
    float* scale_inv;
    const float* noop;
    int64_t rows;
    float eps, weight_offset;
    int hidden, param_f32, fmt;
};
cudaError_t launch_layer_norm(const LayerNormArgs& a, int dtype, int res_dtype, cudaStream_t stream);

struct LayerNormBackwardArgs {
    DropArgs drop;
    const void *dy, *dres_out, *res_out, *weight;
    const float *mean, *rstd;
    void *dres, *du, *dweight, *dbias;
    float* workspace;
    const float* noop;
    int64_t rows;
    float weight_offset;
    int hidden, param_f32;
};
size_t layer_norm_backward_workspace(int64_t rows, int64_t hidden);
// Which kernel a launch on aligned buffers takes: see ct_layer_norm_kernel.
struct LayerNormPlan {
    int blocks, vectors, stages, shifted, warp_per_row, once;
};
LayerNormPlan layer_norm_plan(int64_t rows, int hidden, int x_bytes, int res_bytes, bool backward, bool with);
cudaError_t launch_layer_norm_backward(const LayerNormBackwardArgs& a, int dtype, int res_dtype,
                                       cudaStream_t stream);

struct RouterArgs {
    const void* logits;    // [tokens, experts]
    const uint8_t* mask;   // [tokens], or null
    int* idx;              // [tokens, topk]; read by the backward pass
    float* weights;        // [tokens, topk]
    int* counts;           // [experts + 1]; read by the backward pass
    float* loss;           // or null
    const float* dweights; // or null
    const float* dloss;    // or null
    void* dlogits;         // [tokens, experts]
    void* workspace;
    const float* noop;
    int64_t tokens;
    float balance, z;
    int experts, topk, normalize;
};
size_t router_workspace(int64_t tokens, int experts);
cudaError_t launch_router(const RouterArgs& a, int dtype, cudaStream_t stream);
cudaError_t launch_router_backward(const RouterArgs& a, int dtype, cudaStream_t stream);

struct EmbeddingArgs {
    const void* idx;       // [tokens] int32, or int64 (index64)
    const void* in;        // [vocab, hidden] the table, or [tokens, hidden] dout
    void* out;             // [tokens, hidden], or [vocab, hidden] dtable
    void* workspace;
    const float* noop;
    int64_t tokens, vocab, hidden;
    float scale;
    int index64, accumulate, grad_f32;
};
cudaError_t launch_embedding(const EmbeddingArgs& a, int dtype, cudaStream_t stream);
size_t embedding_backward_workspace(int64_t tokens, int64_t vocab, int64_t hidden);
cudaError_t launch_embedding_backward(const EmbeddingArgs& a, int dtype, cudaStream_t stream);

// The block-norm kernels' own diagnostic word, as read_device_error.
cudaError_t read_norm_error(unsigned* value, bool clear);
// Their give-up path: `blocks` blocks of 64 threads, of which `thread` of the
// first one gives up.
cudaError_t launch_norm_wait_selftest(int blocks, int thread, uint32_t limit_us, cudaStream_t stream);

}  // namespace ct
