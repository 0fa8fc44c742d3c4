// ct_step_api.cu -- the C ABI of the operators between the token ids and the
// FP8 products: embedding, dropout, layer norm and router.  Host-side argument
// checks and launches; nothing here allocates device memory, synchronises or
// reads device memory.
#include "ct_checks.h"
#include "ct_ops.h"

namespace {

using ct::check_buffers;
using ct::cuda_status;
using ct::dtype_ok;
using ct::elem_bytes;
using ct::kMaxElements;
using ct::kMaxIndex;

constexpr int64_t kMaxHidden = int64_t(1) << 20;
constexpr int kMaxRouterTopk = 64;

// What p stands for; false outside [0, 1) or where nothing would be left.
bool drop_of(float p, const int64_t* rng, uint32_t site, ct::DropArgs* d) {
    if (!(p >= 0.0f && p < 1.0f)) return false;
    d->cut = static_cast<uint32_t>(double(p) * 65536.0 + 0.5);
    if (d->cut > 65535) return false;
    d->scale = static_cast<float>(65536.0 / (65536.0 - d->cut));
    d->rng = reinterpret_cast<const uint64_t*>(rng);
    d->site = site;
    return true;
}
ct::DropArgs no_drop() { return ct::DropArgs{nullptr, 0, 0, 1.0f}; }

int check_matrix(int64_t rows, int64_t cols, int64_t max_cols) {
    if (rows < 0 || cols < 0 || rows > kMaxIndex || cols > max_cols ||
        (cols > 0 && rows > kMaxElements / cols))
        return CT_ERR_SHAPE;
    return CT_OK;
}

int check_norm(const ct_layer_norm_config* c) {
    if (!c) return CT_ERR_NULL;
    if (!dtype_ok(c->dtype) || (c->res_dtype != c->dtype && c->res_dtype != CT_FP32) ||
        (c->param_dtype != c->dtype && c->param_dtype != CT_FP32))
        return CT_ERR_FORMAT;
    return check_matrix(c->rows, c->hidden, ct::kMaxNormHidden);
}

int check_router(const ct_router_config* c) {
    if (!c) return CT_ERR_NULL;
    if (!dtype_ok(c->dtype)) return CT_ERR_FORMAT;
    if (c->experts < 1 || c->experts > ct::kMaxExperts || c->topk < 1 || c->topk > kMaxRouterTopk ||
        c->topk > c->experts || (c->flags & ~CT_ROUTER_NORMALIZE))
        return CT_ERR_ARG;
    return c->tokens < 0 || c->tokens > kMaxIndex / c->topk ? CT_ERR_SHAPE : CT_OK;
}

ct::RouterArgs router_args(const ct_router_config& c) {
    ct::RouterArgs a = {};
    a.tokens = c.tokens;
    a.experts = c.experts;
    a.topk = c.topk;
    a.normalize = (c.flags & CT_ROUTER_NORMALIZE) != 0;
    a.balance = c.balance;
    a.z = c.z;
    return a;
}

int check_embedding(int index_bytes, int64_t tokens, int64_t vocab, int64_t hidden, int dtype) {
    if ((index_bytes != 4 && index_bytes != 8) || !dtype_ok(dtype)) return CT_ERR_FORMAT;
    const int st = check_matrix(tokens, hidden, kMaxHidden);
    return st != CT_OK ? st : check_matrix(vocab, hidden, kMaxHidden);
}

}  // namespace

extern "C" {

int dropout(const void* x, int64_t rows, int64_t cols, int dtype, float p, const int64_t* rng,
            uint32_t site, void* out, const float* noop_flag, void* stream) {
    if (!dtype_ok(dtype)) return CT_ERR_FORMAT;
    int st = check_matrix(rows, cols, int64_t(1) << 30);
    if (st != CT_OK) return st;
    ct::DropoutArgs a;
    if (!drop_of(p, rng, site, &a.drop)) return CT_ERR_ARG;
    if (rows == 0 || cols == 0) return CT_OK;
    const int b = elem_bytes(dtype);
    const int64_t bytes = rows * cols * b;
    const bool in_place = out == x;
    st = check_buffers({{x, bytes, b, in_place},
                        {in_place ? nullptr : out, bytes, b, true, in_place},
                        {a.drop.cut ? rng : nullptr, 16, 8, false, a.drop.cut == 0},
                        {noop_flag, 4, 4, false, true}});
    if (st != CT_OK) return st;
    a.x = x;
    a.out = out;
    a.noop = noop_flag;
    a.rows = rows;
    a.cols = cols;
    return cuda_status(ct::launch_dropout(a, dtype, static_cast<cudaStream_t>(stream)));
}

int layer_norm(const ct_layer_norm_config* cfg, const void* u, const void* res, void* res_out,
               void* y, float* mean, float* rstd, const float* scale, float* amax,
               float* scale_inv, int fmt, const float* noop_flag, void* stream) {
    int st = check_norm(cfg);
    if (st != CT_OK) return st;
    const ct_layer_norm_config& c = *cfg;
    if (!(c.eps >= 0.0f)) return CT_ERR_ARG;
    if (scale && fmt != CT_E4M3 && fmt != CT_E5M2) return CT_ERR_FORMAT;
    ct::LayerNormArgs a;
    a.drop = no_drop();
    if (u && !drop_of(c.p, c.rng, c.site, &a.drop)) return CT_ERR_ARG;
    if (c.rows == 0 || c.hidden == 0) return CT_OK;
    if (!u && res_out) return CT_ERR_ARG;
    const int b = elem_bytes(c.dtype), rb = elem_bytes(c.res_dtype), pb = elem_bytes(c.param_dtype);
    const int64_t n = c.rows * c.hidden;
    const bool in_place = res_out == res;
    st = check_buffers({{u, n * b, b, false, true},
                        {res, n * rb, rb, in_place && u},
                        {in_place ? nullptr : res_out, n * rb, rb, true, !u || in_place},
                        {y, scale ? n : n * b, scale ? 1 : b, true},
                        {c.weight, c.hidden * pb, pb, false, true},
                        {c.bias, c.hidden * pb, pb, false, true},
                        {a.drop.cut ? c.rng : nullptr, 16, 8, false, a.drop.cut == 0},
                        {mean, 4 * c.rows, 4, true, true},
                        {rstd, 4 * c.rows, 4, true, true},
                        {scale, 4, 4, false, true},
                        {scale ? amax : nullptr, 4, 4, true, !scale},
                        {scale ? scale_inv : nullptr, 4, 4, true, !scale},
                        {noop_flag, 4, 4, false, true}});
    if (st != CT_OK) return st;
    a.u = u;
    a.res = res;
    a.weight = c.weight;
    a.bias = c.bias;
    a.res_out = res_out;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.scale = scale;
    a.amax = amax;
    a.scale_inv = scale_inv;
    a.noop = noop_flag;
    a.rows = c.rows;
    a.eps = c.eps;
    a.weight_offset = c.weight_offset;
    a.hidden = static_cast<int>(c.hidden);
    a.param_f32 = c.param_dtype == CT_FP32;
    a.fmt = fmt;
    return cuda_status(ct::launch_layer_norm(a, c.dtype, c.res_dtype, static_cast<cudaStream_t>(stream)));
}

size_t layer_norm_backward_workspace_size(int64_t rows, int64_t hidden) {
    if (check_matrix(rows, hidden, ct::kMaxNormHidden) != CT_OK) return 0;
    return ct::layer_norm_backward_workspace(rows, hidden);
}

int layer_norm_backward(const ct_layer_norm_config* cfg, const void* dy, const void* dres_out,
                        const void* res_out, const float* mean, const float* rstd, void* dres,
                        void* du, void* dweight, void* dbias, void* workspace,
                        size_t workspace_bytes, const float* noop_flag, void* stream) {
    int st = check_norm(cfg);
    if (st != CT_OK) return st;
    const ct_layer_norm_config& c = *cfg;
    ct::LayerNormBackwardArgs a;
    a.drop = no_drop();
    if (du && !drop_of(c.p, c.rng, c.site, &a.drop)) return CT_ERR_ARG;
    if (c.hidden == 0) return CT_OK;
    const int b = elem_bytes(c.dtype), rb = elem_bytes(c.res_dtype), pb = elem_bytes(c.param_dtype);
    const int64_t n = c.rows * c.hidden;
    const size_t need = dweight || dbias ? ct::layer_norm_backward_workspace(c.rows, c.hidden) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return CT_ERR_WORKSPACE;
    st = check_buffers({{dy, n * b, b, false},
                        {dres_out, n * rb, rb, false, true},
                        {res_out, n * rb, rb, false},
                        {mean, 4 * c.rows, 4, false},
                        {rstd, 4 * c.rows, 4, false},
                        {c.weight, c.hidden * pb, pb, false, true},
                        {a.drop.cut ? c.rng : nullptr, 16, 8, false, a.drop.cut == 0 || c.rows == 0},
                        {dres, n * rb, rb, true},
                        {du, n * b, b, true, true},
                        {dweight, c.hidden * pb, pb, true, true},
                        {dbias, c.hidden * pb, pb, true, true},
                        {need ? workspace : nullptr, int64_t(need), 16, true, true},
                        {noop_flag, 4, 4, false, true}});
    if (st != CT_OK) return st;
    a.dy = dy;
    a.dres_out = dres_out;
    a.res_out = res_out;
    a.weight = c.weight;
    a.mean = mean;
    a.rstd = rstd;
    a.dres = dres;
    a.du = du;
    a.dweight = dweight;
    a.dbias = dbias;
    a.workspace = static_cast<float*>(workspace);
    a.noop = noop_flag;
    a.rows = c.rows;
    a.weight_offset = c.weight_offset;
    a.hidden = static_cast<int>(c.hidden);
    a.param_f32 = c.param_dtype == CT_FP32;
    return cuda_status(ct::launch_layer_norm_backward(a, c.dtype, c.res_dtype,
                                                      static_cast<cudaStream_t>(stream)));
}

int ct_layer_norm_kernel(const ct_layer_norm_config* cfg, int backward, int with, ct_layer_norm_plan* plan) {
    if (!plan) return CT_ERR_NULL;
    const int st = check_norm(cfg);
    if (st != CT_OK) return st;
    ct::LayerNormPlan p = {};
    if (cfg->rows > 0 && cfg->hidden > 0)
        p = ct::layer_norm_plan(cfg->rows, static_cast<int>(cfg->hidden), elem_bytes(cfg->dtype),
                                elem_bytes(cfg->res_dtype), backward != 0, with != 0);
    *plan = {p.blocks, p.vectors, p.stages, p.shifted, p.warp_per_row, p.once};
    return CT_OK;
}

size_t moe_router_workspace_size(int64_t tokens, int topk, int experts) {
    if (experts < 1 || experts > ct::kMaxExperts || topk < 1 || topk > kMaxRouterTopk || tokens < 0 ||
        tokens > kMaxIndex / topk)
        return 0;
    return ct::router_workspace(tokens, experts);
}

int moe_router(const ct_router_config* cfg, const void* logits, const uint8_t* mask, int* expert_idx,
               float* weights, int* counts, float* loss, void* workspace, size_t workspace_bytes,
               const float* noop_flag, void* stream) {
    int st = check_router(cfg);
    if (st != CT_OK) return st;
    const ct_router_config& c = *cfg;
    const size_t need = ct::router_workspace(c.tokens, c.experts);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CT_ERR_WORKSPACE;
    const int b = elem_bytes(c.dtype);
    const int64_t slots = c.tokens * c.topk;
    st = check_buffers({{logits, c.tokens * c.experts * b, b, false},
                        {mask, c.tokens, 1, false, true},
                        {expert_idx, 4 * slots, 4, true},
                        {weights, 4 * slots, 4, true},
                        {counts, 4 * (int64_t(c.experts) + 1), 4, true},
                        {loss, 4, 4, true, true},
                        {need ? workspace : nullptr, int64_t(need), 16, true, true},
                        {noop_flag, 4, 4, false, true}});
    if (st != CT_OK) return st;
    ct::RouterArgs a = router_args(c);
    a.logits = logits;
    a.mask = mask;
    a.idx = expert_idx;
    a.weights = weights;
    a.counts = counts;
    a.loss = loss;
    a.workspace = workspace;
    a.noop = noop_flag;
    return cuda_status(ct::launch_router(a, c.dtype, static_cast<cudaStream_t>(stream)));
}

int moe_router_backward(const ct_router_config* cfg, const void* logits, const uint8_t* mask,
                        const int* expert_idx, const int* counts, const float* dweights,
                        const float* dloss, void* dlogits, const float* noop_flag, void* stream) {
    int st = check_router(cfg);
    if (st != CT_OK) return st;
    const ct_router_config& c = *cfg;
    if (c.tokens == 0) return CT_OK;
    if (!dweights && !dloss) return CT_ERR_NULL;
    const int b = elem_bytes(c.dtype);
    const int64_t n = c.tokens * c.experts, slots = c.tokens * c.topk;
    st = check_buffers({{logits, n * b, b, false},
                        {mask, c.tokens, 1, false, true},
                        {expert_idx, 4 * slots, 4, false},
                        {counts, 4 * (int64_t(c.experts) + 1), 4, false},
                        {dweights, 4 * slots, 4, false, true},
                        {dloss, 4, 4, false, true},
                        {dlogits, n * b, b, true},
                        {noop_flag, 4, 4, false, true}});
    if (st != CT_OK) return st;
    ct::RouterArgs a = router_args(c);
    a.logits = logits;
    a.mask = mask;
    a.idx = const_cast<int*>(expert_idx);
    a.counts = const_cast<int*>(counts);
    a.dweights = dweights;
    a.dloss = dloss;
    a.dlogits = dlogits;
    a.noop = noop_flag;
    return cuda_status(ct::launch_router_backward(a, c.dtype, static_cast<cudaStream_t>(stream)));
}

int embedding(const void* idx, int index_bytes, int64_t tokens, const void* table, int64_t vocab,
              int64_t hidden, int dtype, float scale, void* out, const float* noop_flag,
              void* stream) {
    int st = check_embedding(index_bytes, tokens, vocab, hidden, dtype);
    if (st != CT_OK) return st;
    if (tokens == 0 || hidden == 0) return CT_OK;
    const int b = elem_bytes(dtype);
    st = check_buffers({{idx, tokens * index_bytes, index_bytes, false},
                        {table, vocab * hidden * b, b, false},
                        {out, tokens * hidden * b, b, true},
                        {noop_flag, 4, 4, false, true}});
    if (st != CT_OK) return st;
    ct::EmbeddingArgs a = {};
    a.idx = idx;
    a.in = table;
    a.out = out;
    a.noop = noop_flag;
    a.tokens = tokens;
    a.vocab = vocab;
    a.hidden = hidden;
    a.scale = scale;
    a.index64 = index_bytes == 8;
    return cuda_status(ct::launch_embedding(a, dtype, static_cast<cudaStream_t>(stream)));
}

size_t embedding_backward_workspace_size(int64_t tokens, int64_t vocab, int64_t hidden) {
    if (check_embedding(4, tokens, vocab, hidden, CT_BF16) != CT_OK) return 0;
    return ct::embedding_backward_workspace(tokens, vocab, hidden);
}

int embedding_backward(const void* idx, int index_bytes, int64_t tokens, const void* dout,
                       int64_t vocab, int64_t hidden, int dtype, float scale, void* dtable,
                       int grad_dtype, int accumulate, void* workspace, size_t workspace_bytes,
                       const float* noop_flag, void* stream) {
    int st = check_embedding(index_bytes, tokens, vocab, hidden, dtype);
    if (st != CT_OK) return st;
    if (grad_dtype != dtype && grad_dtype != CT_FP32) return CT_ERR_FORMAT;
    if (accumulate != 0 && accumulate != 1) return CT_ERR_ARG;
    if (vocab == 0 || hidden == 0 || (tokens == 0 && accumulate)) return CT_OK;
    const int b = elem_bytes(dtype), gb = elem_bytes(grad_dtype);
    const size_t need = ct::embedding_backward_workspace(tokens, vocab, hidden);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CT_ERR_WORKSPACE;
    st = check_buffers({{idx, tokens * index_bytes, index_bytes, false},
                        {dout, tokens * hidden * b, b, false},
                        {dtable, vocab * hidden * gb, gb, true},
                        {need ? workspace : nullptr, int64_t(need), 16, true, true},
                        {noop_flag, 4, 4, false, true}});
    if (st != CT_OK) return st;
    ct::EmbeddingArgs a = {};
    a.idx = idx;
    a.in = dout;
    a.out = dtable;
    a.workspace = workspace;
    a.noop = noop_flag;
    a.tokens = tokens;
    a.vocab = vocab;
    a.hidden = hidden;
    a.scale = scale;
    a.index64 = index_bytes == 8;
    a.accumulate = accumulate;
    a.grad_f32 = grad_dtype == CT_FP32;
    return cuda_status(ct::launch_embedding_backward(a, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
