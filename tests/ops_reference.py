"""Plain 64-bit forms of the expert-movement and block-norm operators, with
the error that fp32 arithmetic and one final rounding may add to each value.

The bounds are worst cases, fixed before any run: an fp32 operation adds at
most 2^-24 of its result, a sum of n terms in any order at most (n - 1) * 2^-24
of the sum of their magnitudes, the final rounding half a unit in the last
place of the output's type (at most 2^-8 of the value for bf16, 2^-11 for
fp16, 2^-24 for fp32, and 2^-25 in all for fp16's subnormal numbers).
"""
import numpy as np
import torch

F = 2.0 ** -24
U_OUT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: F}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24, torch.float32: 1e-38}


def sort(idx, experts, align, rows):
    """The plan by walking the slots one after another."""
    flat = idx.reshape(-1).tolist()
    lists = [[] for _ in range(experts)]
    for s, e in enumerate(flat):
        if 0 <= e < experts:
            lists[e].append(s)
    row_of = np.full(len(flat), -1, np.int32)
    src = np.full(rows, -1, np.int32)
    offsets, at = [], 0
    for slots in lists:
        offsets.append(min(at, rows))
        for i, s in enumerate(slots):
            if at + i < rows:
                row_of[s] = at + i
                src[at + i] = s
        at += -(-len(slots) // align) * align
    offsets.append(min(at, rows))
    return (row_of.reshape(idx.shape), src, np.array(offsets, np.int32),
            np.array([len(x) for x in lists], np.int32))


def rounded(ref, err, dtype):
    """Bound of an output of `dtype` whose fp32 value is within err of ref."""
    return err + U_OUT[dtype] * (ref.abs() + err) + TINY[dtype]


def close(got, ref, bound, name):
    got, ref = got.detach().double().cpu(), ref.double().cpu()
    off = (got - ref).abs() - bound.cpu()
    bad = torch.isnan(got) != torch.isnan(ref)
    bad |= ~torch.isnan(ref) & torch.isinf(ref) & (got != ref)
    bad |= torch.isfinite(ref) & ~(off <= 0)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} values off, first at "
                           f"{bad.nonzero()[0].tolist()}: {got[bad][0]} for {ref[bad][0]}")


def combine(ys, row_of, weights):
    """(out, error) of moe_combine; weights None: of moe_dispatch_backward."""
    kept = torch.as_tensor(row_of >= 0)
    row = torch.as_tensor(row_of).long().clamp(min=0)
    parts = torch.where(kept[:, :, None], ys.double()[row], 0.0)
    if weights is not None:
        parts = parts * torch.where(kept, weights.double(), 1.0)[:, :, None]
    k = row.shape[1]
    return parts.sum(1), (k + 1) * F * parts.abs().sum(1)


def combine_backward(dout, ys, row_of, weights, rows):
    row_of = torch.as_tensor(row_of).long()
    dys = torch.zeros(rows, dout.shape[1], dtype=torch.float64)
    dw = torch.zeros(weights.shape, dtype=torch.float64)
    dw_err = torch.zeros_like(dw)
    for t in range(row_of.shape[0]):
        for k in range(row_of.shape[1]):
            r = int(row_of[t, k])
            if r < 0:
                continue
            dys[r] = weights[t, k].double() * dout[t].double()
            products = dout[t].double() * ys[r].double()
            dw[t, k] = products.sum()
            dw_err[t, k] = (dout.shape[1] + 1) * F * products.abs().sum()
    return dys, F * dys.abs(), dw, dw_err


class Norm:
    """One junction in 64 bits, with gradients and bounds.  Sums along a row
    are counted as 128 additions deep (a thread's own columns, its warp's, the
    block's), sums along the rows as `rows` deep."""
    DEEP = 128 * F

    def __init__(self, u, res, w_post, w_pre, gate, rows_per_gate, eps, branch_scale,
                 residual_scale, weight_offset, post_norm=True, pre_norm=True):
        self.u = None if u is None else u.double()
        self.res = res.double()
        self.post, self.pre = post_norm and u is not None, pre_norm
        self.eps, self.alpha, self.beta = eps, branch_scale, residual_scale
        rows, self.H = res.shape
        one = torch.ones(self.H, dtype=torch.float64)
        self.a_post = one if w_post is None or not self.post else weight_offset + w_post.double()
        self.a_pre = one if w_pre is None else weight_offset + w_pre.double()
        self.groups = torch.arange(rows) // max(rows_per_gate or rows, 1)
        self.gate = gate
        self.g = one.expand(rows, -1) if gate is None else gate.double()[self.groups]

    def forward(self):
        if self.u is None:
            out, err = self.res, torch.zeros_like(self.res)
            self.rstd_post = None
        else:
            self.rstd_post = torch.ones(len(self.res), dtype=torch.float64)
            if self.post:
                self.rstd_post = (self.u.square().mean(1) + self.eps).rsqrt()
            branch = self.alpha * self.g * self.u * self.rstd_post[:, None] * self.a_post
            out = self.beta * self.res + branch
            err = 4 * F * (self.beta * self.res).abs() + (8 * F + self.DEEP) * branch.abs()
        self.out, self.out_err = out, err
        if self.pre:
            self.rstd_pre = (out.square().mean(1) + self.eps).rsqrt()
            # the mean of squares moves by at most 2 mean |out| err
            self.rstd_err = (self.DEEP + 4 * F + (out.abs() * err).mean(1)
                             * self.rstd_pre.square())
            self.y = out * self.rstd_pre[:, None] * self.a_pre
            self.y_err = (err * self.rstd_pre[:, None] * self.a_pre.abs()
                          + self.y.abs() * (self.rstd_err[:, None] + 4 * F))
        return self

    def backward(self, dy, dres_out, res_out, rstd_post, rstd_pre):
        """Gradients from what the forward pass kept, and their bounds."""
        c = self.DEEP + 16 * F
        rows = len(res_out)
        x = res_out.double()
        d = torch.zeros_like(x) if dres_out is None else dres_out.double()
        size = d.abs()
        r = {}
        if self.pre:
            s = rstd_pre.double()[:, None]
            hat, back = x * s, dy.double() * self.a_pre
            d = d + s * (back - hat * (back * hat).mean(1, keepdim=True))
            size = size + s * (back.abs() + hat.abs() * (back * hat).abs().mean(1, keepdim=True))
            r["dw_pre"] = (dy.double() * hat).sum(0), (rows + 4) * F * (dy.double() * hat).abs().sum(0)
        beta = self.beta if self.u is not None else 1.0
        r["dres"] = beta * d, c * abs(beta) * size
        if self.u is None:
            return r
        s = rstd_post.double()[:, None] if self.post else torch.ones(rows, 1, dtype=torch.float64)
        hat, scale = self.u * s, self.alpha * self.g
        dz, dz_size = scale * d, scale.abs() * size
        back, back_size = dz * self.a_post, dz_size * self.a_post.abs()
        if self.post:
            du = s * (back - hat * (back * hat).mean(1, keepdim=True))
            du_size = s * (back_size + hat.abs() * (back_size * hat.abs()).mean(1, keepdim=True))
            sums = (dz_size * hat.abs()).sum(0)
            r["dw_post"] = (dz * hat).sum(0), (c + (rows + 4) * F) * sums
        else:
            du, du_size = back, back_size
        r["du"] = du, 2 * c * du_size
        if self.gate is not None:
            each, each_size = self.alpha * d * hat * self.a_post, (abs(self.alpha) * size * hat.abs()
                                                                   * self.a_post.abs())
            out = torch.zeros(self.gate.shape, dtype=torch.float64)
            top = torch.zeros_like(out)
            r["dgate"] = (out.index_add_(0, self.groups, each),
                          (c + (rows + 4) * F) * top.index_add_(0, self.groups, each_size))
        return r
