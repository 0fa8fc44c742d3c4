// ct_ops_api.cu -- the C ABI of the expert-movement and block-norm operators:
// host-side argument checks and launches.  Like the cast entry points, nothing
// here allocates device memory, synchronises or reads device memory.
#include "ct_checks.h"
#include "ct_ops.h"

namespace {

using ct::cuda_status;

using ct::kMaxExperts;
constexpr int kMaxTopk = 64, kMaxAlign = 1024;
using ct::dtype_ok;
using ct::elem_bytes;
using ct::check_buffers;
using ct::kMaxElements;
using ct::kMaxIndex;
using ct::kMaxNormHidden;
constexpr int64_t kMaxMoveHidden = int64_t(1) << 20;

int check_move(int64_t tokens, int topk, int64_t hidden, int64_t rows, int dtype) {
    if (!dtype_ok(dtype)) return CT_ERR_FORMAT;
    if (topk < 1 || topk > kMaxTopk) return CT_ERR_ARG;
    if (tokens < 0 || hidden < 0 || rows < 0 || hidden > kMaxMoveHidden ||
        tokens > kMaxIndex / topk || rows > kMaxIndex ||
        (hidden > 0 && rows > kMaxElements / hidden))
        return CT_ERR_SHAPE;
    return CT_OK;
}

// Blocks of a launch that writes sorted rows: as many as a grid can have.
bool fits_grid(int64_t tokens, int64_t rows) { return tokens + ct::pad_blocks(rows) <= kMaxIndex; }

}  // namespace

extern "C" {

int64_t moe_sorted_rows(int64_t tokens, int topk, int experts, int align) {
    if (tokens < 0 || topk < 1 || topk > kMaxTopk || experts < 1 || experts > kMaxExperts ||
        align < 1 || align > kMaxAlign || tokens > kMaxIndex / topk)
        return 0;
    const int64_t n = tokens * topk, used = n < experts ? n : experts;
    return (n + used * (align - 1) + align - 1) / align * align;
}

size_t moe_sort_workspace_size(int64_t tokens, int topk, int experts) {
    if (tokens < 0 || topk < 1 || topk > kMaxTopk || experts < 1 || experts > kMaxExperts ||
        tokens > kMaxIndex / topk)
        return 0;
    return ct::sort_workspace(tokens * topk, experts);
}

int moe_sort(const void* expert_idx, int index_bytes, int64_t tokens, int topk, int experts,
             int align, int64_t rows, int* row_of, int* src, int* offsets, int* counts,
             void* workspace, size_t workspace_bytes, const float* noop_flag, void* stream) {
    if (index_bytes != 4 && index_bytes != 8) return CT_ERR_FORMAT;
    if (topk < 1 || topk > kMaxTopk || experts < 1 || experts > kMaxExperts || align < 1 ||
        align > kMaxAlign)
        return CT_ERR_ARG;
    if (tokens < 0 || rows < 0 || tokens > kMaxIndex / topk || rows > kMaxIndex)
        return CT_ERR_SHAPE;
    const int64_t n = tokens * topk;
    const size_t need = ct::sort_workspace(n, experts);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CT_ERR_WORKSPACE;
    const int st = check_buffers({{expert_idx, n * index_bytes, index_bytes, false},
                                  {row_of, 4 * n, 4, true},
                                  {src, 4 * rows, 4, true},
                                  {offsets, 4 * (int64_t(experts) + 1), 4, true},
                                  {counts, 4 * int64_t(experts), 4, true},
                                  {need ? workspace : nullptr, int64_t(need), 16, true, true}});
    if (st != CT_OK) return st;
    ct::SortArgs a;
    a.idx = expert_idx;
    a.n = n;
    a.rows = rows;
    a.row_of = row_of;
    a.src = src;
    a.offsets = offsets;
    a.counts = counts;
    a.noop = noop_flag;
    a.experts = experts;
    a.align = align;
    a.index64 = index_bytes == 8;
    for (a.expert_bits = 0; (1 << a.expert_bits) < experts;) ++a.expert_bits;
    return cuda_status(ct::launch_moe_sort(a, workspace, static_cast<cudaStream_t>(stream)));
}

int moe_dispatch(const void* x, int64_t tokens, int topk, int64_t hidden, int dtype,
                 const int* row_of, const int* src, int64_t rows, void* out,
                 const float* noop_flag, void* stream) {
    int st = check_move(tokens, topk, hidden, rows, dtype);
    if (st != CT_OK) return st;
    if (!fits_grid(tokens, rows)) return CT_ERR_SHAPE;
    if (hidden == 0 || rows == 0) return CT_OK;
    const int b = elem_bytes(dtype);
    st = check_buffers({{x, tokens * hidden * b, b, false},
                        {row_of, 4 * tokens * topk, 4, false},
                        {src, 4 * rows, 4, false},
                        {out, rows * hidden * b, b, true}});
    if (st != CT_OK) return st;
    ct::MoveArgs a = {};
    a.x = x;
    a.sorted = out;
    a.row_of = row_of;
    a.src = src;
    a.noop = noop_flag;
    a.tokens = tokens;
    a.rows = rows;
    a.hidden = hidden;
    a.topk = topk;
    a.elem_bytes = b;
    return cuda_status(ct::launch_moe_dispatch(a, static_cast<cudaStream_t>(stream)));
}

static int combine_impl(const void* ys, int64_t tokens, int topk, int64_t hidden, int dtype,
                        const int* row_of, const float* weights, bool weighted, int64_t rows,
                        void* out, const float* noop_flag, void* stream) {
    int st = check_move(tokens, topk, hidden, rows, dtype);
    if (st != CT_OK) return st;
    if (hidden == 0 || tokens == 0) return CT_OK;
    const int b = elem_bytes(dtype);
    st = check_buffers({{ys, rows * hidden * b, b, false},
                        {row_of, 4 * tokens * topk, 4, false},
                        {weights, 4 * tokens * topk, 4, false, !weighted},
                        {out, tokens * hidden * b, b, true}});
    if (st != CT_OK) return st;
    ct::MoveArgs a = {};
    a.ys = ys;
    a.out = out;
    a.row_of = row_of;
    a.weights = weighted ? weights : nullptr;
    a.noop = noop_flag;
    a.tokens = tokens;
    a.rows = rows;
    a.hidden = hidden;
    a.topk = topk;
    a.elem_bytes = b;
    return cuda_status(ct::launch_moe_combine(a, dtype, static_cast<cudaStream_t>(stream)));
}

int moe_dispatch_backward(const void* dout, int64_t tokens, int topk, int64_t hidden, int dtype,
                          const int* row_of, int64_t rows, void* dx, const float* noop_flag,
                          void* stream) {
    return combine_impl(dout, tokens, topk, hidden, dtype, row_of, nullptr, false, rows, dx,
                        noop_flag, stream);
}

int moe_combine(const void* ys, int64_t tokens, int topk, int64_t hidden, int dtype,
                const int* row_of, const float* weights, int64_t rows, void* out,
                const float* noop_flag, void* stream) {
    return combine_impl(ys, tokens, topk, hidden, dtype, row_of, weights, true, rows, out,
                        noop_flag, stream);
}

int moe_combine_backward(const void* dout, const void* ys, int64_t tokens, int topk,
                         int64_t hidden, int dtype, const int* row_of, const int* src,
                         const float* weights, int64_t rows, void* dys, float* dweights,
                         const float* noop_flag, void* stream) {
    int st = check_move(tokens, topk, hidden, rows, dtype);
    if (st != CT_OK) return st;
    if (!dys && !dweights) return CT_ERR_NULL;
    if (dys && !fits_grid(tokens, rows)) return CT_ERR_SHAPE;
    const int b = elem_bytes(dtype);
    st = check_buffers({{dout, tokens * hidden * b, b, false},
                        {ys, rows * hidden * b, b, false, !dweights},
                        {row_of, 4 * tokens * topk, 4, false},
                        {src, 4 * rows, 4, false, !dys},
                        {weights, 4 * tokens * topk, 4, false, !dys},
                        {dys, rows * hidden * b, b, true, true},
                        {dweights, 4 * tokens * topk, 4, true, true}});
    if (st != CT_OK) return st;
    if (tokens == 0 && (!dys || rows == 0 || hidden == 0)) return CT_OK;
    ct::MoveArgs a = {};
    a.x = dout;
    a.ys = dweights ? ys : nullptr;
    a.sorted = dys;
    a.row_of = row_of;
    a.src = src;
    a.weights = weights;
    a.dweights = dweights;
    a.noop = noop_flag;
    a.tokens = tokens;
    a.rows = rows;
    a.hidden = hidden;
    a.topk = topk;
    a.elem_bytes = b;
    return cuda_status(ct::launch_moe_combine_backward(a, dtype, static_cast<cudaStream_t>(stream)));
}

int fp8_moe_dispatch(const void* x, int64_t tokens, int topk, int64_t hidden, const int* src,
                     int64_t rows, const float* weights, const float* scale, float* amax,
                     float* scale_inv, void* out, void* out_t, int fmt, const float* noop_flag,
                     void* stream) {
    if (fmt != CT_E4M3 && fmt != CT_E5M2) return CT_ERR_FORMAT;
    int st = check_move(tokens, topk, hidden, rows, CT_BF16);
    if (st != CT_OK) return st;
    if (hidden == 0 || rows == 0) return CT_OK;
    st = check_buffers({{x, tokens * hidden * 2, 2, false},
                        {src, 4 * rows, 4, false},
                        {weights, 4 * tokens * topk, 4, false, true},
                        {scale, 4, 4, false},
                        {amax, 4, 4, true},
                        {scale_inv, 4, 4, true},
                        {out, rows * hidden, 1, true},
                        {out_t, rows * hidden, 1, true, true}});
    if (st != CT_OK) return st;
    ct::SortedCastArgs a;
    a.x = static_cast<const uint16_t*>(x);
    a.src = src;
    a.weights = weights;
    a.scale = scale;
    a.amax = amax;
    a.scale_inv = scale_inv;
    a.out = static_cast<uint8_t*>(out);
    a.out_t = static_cast<uint8_t*>(out_t);
    a.noop = noop_flag;
    a.tokens = tokens;
    a.rows = rows;
    a.hidden = hidden;
    a.topk = topk;
    return cuda_status(ct::launch_sorted_cast(a, fmt, static_cast<cudaStream_t>(stream)));
}

// rows_per_gate, no larger than what it can make a difference for.
static int64_t gate_rows(const ct_block_norm_config& c) {
    return c.rows_per_gate < c.rows ? c.rows_per_gate : (c.rows > 0 ? c.rows : 1);
}

// The config's own fields; `groups` receives the gate's rows.
static int check_config(const ct_block_norm_config* c, int64_t* groups) {
    if (!c) return CT_ERR_NULL;
    if (!dtype_ok(c->dtype) || (c->res_dtype != c->dtype && c->res_dtype != CT_FP32) ||
        (c->param_dtype != c->dtype && c->param_dtype != CT_FP32))
        return CT_ERR_FORMAT;
    if (c->flags & ~(CT_NORM_POST | CT_NORM_PRE)) return CT_ERR_ARG;
    if (c->rows < 0 || c->hidden < 0 || c->hidden > kMaxNormHidden || c->rows > kMaxIndex)
        return CT_ERR_SHAPE;
    if (!(c->eps >= 0.0f) || (c->gate && c->rows_per_gate < 1)) return CT_ERR_ARG;
    *groups = c->gate ? (c->rows + gate_rows(*c) - 1) / gate_rows(*c) : 0;
    return CT_OK;
}

int block_norm(const ct_block_norm_config* cfg, const void* u, const void* res, void* res_out,
               void* y, float* rstd_post, float* rstd_pre, const float* scale, float* amax,
               float* scale_inv, int fmt, const float* noop_flag, void* stream) {
    int64_t groups;
    int st = check_config(cfg, &groups);
    if (st != CT_OK) return st;
    const ct_block_norm_config& c = *cfg;
    const bool pre = (c.flags & CT_NORM_PRE) != 0, post = u && (c.flags & CT_NORM_POST) != 0;
    if (scale && fmt != CT_E4M3 && fmt != CT_E5M2) return CT_ERR_FORMAT;
    if (c.rows == 0 || c.hidden == 0) return CT_OK;
    if (!u && !pre) return CT_ERR_ARG;   // nothing to compute
    const int b = elem_bytes(c.dtype), rb = elem_bytes(c.res_dtype), pb = elem_bytes(c.param_dtype);
    const int64_t n = c.rows * c.hidden;
    if (!u && res_out) return CT_ERR_ARG;
    const bool in_place = res_out == res;
    st = check_buffers({{u, n * b, b, false, true},
                        {res, n * rb, rb, in_place && u},
                        {in_place ? nullptr : res_out, n * rb, rb, true, !u || in_place},
                        {pre ? y : nullptr, scale ? n : n * b, scale ? 1 : b, true, !pre},
                        {c.w_post, c.hidden * pb, pb, false, true},
                        {c.w_pre, c.hidden * pb, pb, false, true},
                        {c.gate, groups * c.hidden * pb, pb, false, true},
                        {post ? rstd_post : nullptr, 4 * c.rows, 4, true, true},
                        {pre ? rstd_pre : nullptr, 4 * c.rows, 4, true, true},
                        {scale, 4, 4, false, true},
                        {scale && pre ? amax : nullptr, 4, 4, true, !scale || !pre},
                        {scale && pre ? scale_inv : nullptr, 4, 4, true, !scale || !pre}});
    if (st != CT_OK) return st;
    ct::NormArgs a;
    a.u = u;
    a.res = res;
    a.w_post = c.w_post;
    a.w_pre = c.w_pre;
    a.gate = c.gate;
    a.res_out = res_out;
    a.y = y;
    a.rstd_post = rstd_post;
    a.rstd_pre = rstd_pre;
    a.scale = scale;
    a.amax = amax;
    a.scale_inv = scale_inv;
    a.noop = noop_flag;
    a.rows = c.rows;
    a.rows_per_gate = gate_rows(c);
    a.eps = c.eps;
    a.branch_scale = c.branch_scale;
    a.residual_scale = c.residual_scale;
    a.weight_offset = c.weight_offset;
    a.hidden = static_cast<int>(c.hidden);
    a.param_f32 = c.param_dtype == CT_FP32;
    a.post = post;
    a.pre = pre;
    a.fmt = fmt;
    return cuda_status(ct::launch_block_norm(a, c.dtype, c.res_dtype,
                                             static_cast<cudaStream_t>(stream)));
}

size_t block_norm_backward_workspace_size(int64_t rows, int64_t hidden) {
    if (rows < 0 || hidden < 0 || rows > kMaxIndex || hidden > kMaxNormHidden) return 0;
    return ct::norm_backward_workspace(rows, hidden);
}

int block_norm_backward(const ct_block_norm_config* cfg, const void* dy, const void* dres_out,
                        const void* u, const void* res_out, const float* rstd_post,
                        const float* rstd_pre, void* du, void* dres, void* dw_post, void* dw_pre,
                        void* dgate, void* workspace, size_t workspace_bytes,
                        const float* noop_flag, void* stream) {
    int64_t groups;
    int st = check_config(cfg, &groups);
    if (st != CT_OK) return st;
    const ct_block_norm_config& c = *cfg;
    const bool pre = (c.flags & CT_NORM_PRE) != 0, post = u && (c.flags & CT_NORM_POST) != 0;
    // nothing to compute, or a gradient of something the forward pass does not
    // have (without rows u may be a null pointer that says neither)
    if (c.rows > 0 && ((!u && !pre) || (dw_post && !post) || (dw_pre && !pre) ||
                       (dgate && !(u && c.gate)) || (du && !u)))
        return CT_ERR_ARG;
    if (c.hidden == 0) return CT_OK;
    const int b = elem_bytes(c.dtype), rb = elem_bytes(c.res_dtype), pb = elem_bytes(c.param_dtype);
    const int64_t n = c.rows * c.hidden;
    const size_t need = ct::norm_backward_workspace(c.rows, c.hidden);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CT_ERR_WORKSPACE;
    st = check_buffers({{pre ? dy : nullptr, n * b, b, false, !pre},
                        {dres_out, n * rb, rb, false, true},
                        {u, n * b, b, false, true},
                        {pre ? res_out : nullptr, n * rb, rb, false, !pre},
                        {post ? rstd_post : nullptr, 4 * c.rows, 4, false, !post},
                        {pre ? rstd_pre : nullptr, 4 * c.rows, 4, false, !pre},
                        {c.w_post, c.hidden * pb, pb, false, true},
                        {c.w_pre, c.hidden * pb, pb, false, true},
                        {c.gate, groups * c.hidden * pb, pb, false, true},
                        {du, n * b, b, true, !u},
                        {dres, n * rb, rb, true},
                        {dw_post, c.hidden * pb, pb, true, true},
                        {dw_pre, c.hidden * pb, pb, true, true},
                        {dgate, groups * c.hidden * pb, pb, true, true},
                        {need ? workspace : nullptr, int64_t(need), 16, true, true}});
    if (st != CT_OK) return st;
    ct::NormBackwardArgs a;
    a.dy = dy;
    a.dres_out = dres_out;
    a.u = u;
    a.res_out = res_out;
    a.w_post = c.w_post;
    a.w_pre = c.w_pre;
    a.gate = c.gate;
    a.rstd_post = rstd_post;
    a.rstd_pre = rstd_pre;
    a.du = du;
    a.dres = dres;
    a.dw_post = dw_post;
    a.dw_pre = dw_pre;
    a.dgate = dgate;
    a.workspace = static_cast<float*>(workspace);
    a.noop = noop_flag;
    a.rows = c.rows;
    a.rows_per_gate = gate_rows(c);
    a.branch_scale = c.branch_scale;
    a.residual_scale = c.residual_scale;
    a.weight_offset = c.weight_offset;
    a.hidden = static_cast<int>(c.hidden);
    a.param_f32 = c.param_dtype == CT_FP32;
    a.post = post;
    a.pre = pre;
    return cuda_status(ct::launch_block_norm_backward(a, c.dtype, c.res_dtype,
                                                      static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
