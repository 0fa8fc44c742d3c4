"""One training step of a mixture-of-experts block with FP8 experts, on this
library's operators:

    junction   res, h = block_norm(branch of the block before, res)
    router     probabilities of h @ w_router, the best K of E experts per token
    sort       moe_sort
    dispatch   fp8_moe_dispatch: h in expert order, E4M3, with its transpose
    experts    y_e = x_e @ w_e^T (the weights by fp8_cast_transpose)
    combine    moe_combine with the router's weights
    junction   res, out = block_norm(combined branch, res)

and back, the output gradient of the experts being E5M2 (fp8_moe_dispatch with
the router's weights), then the delayed-scaling update of every FP8 tensor.

The experts' products and the router are plain torch products here, on the FP8
values: they stand for the FP8 matrix products of a real block.  Shapes are
static (the sorted buffers hold any routing); only the loop over the experts
reads their offsets on the host.

    python examples/moe_block.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import cast_transpose_gb300 as ct  # noqa: E402

BF16, ALIGN, HISTORY = torch.bfloat16, 16, 16


class Fp8Meta:
    """Amax history and scales of a set of FP8 tensors, one column each."""

    def __init__(self, names, fmt, device="cuda"):
        self.col = {n: i for i, n in enumerate(names)}
        n = len(self.col)
        self.fmt = fmt
        self.history = torch.zeros(HISTORY, n, device=device)
        self.scale = torch.ones(n, device=device)
        self.recipe_scale_inv = torch.ones(n, device=device)
        self.scale_inv = torch.ones(n, device=device)

    def of(self, name):
        """(scale, amax slot, scale_inv) of one tensor."""
        i = self.col[name]
        return self.scale[i:i + 1], self.history[0, i:i + 1], self.scale_inv[i:i + 1]

    def update(self):
        ct.fp8_amax_and_scale_update(self.history, self.scale, self.recipe_scale_inv, self.fmt)


def values(q, scale_inv, fmt):
    """bf16 values of FP8 codes, before their scale; and the scale to apply."""
    return q.view(ct.TORCH_FP8[fmt]).to(BF16), scale_inv


class MoeBlock:
    def __init__(self, hidden, experts, topk, tokens, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)

        self.hidden, self.experts, self.topk, self.tokens = hidden, experts, topk, tokens
        self.router = normal(hidden, experts, std=hidden ** -0.5)
        self.w = normal(experts, hidden, hidden, std=hidden ** -0.5)
        self.norms = [{"w_post": (1 + normal(hidden, std=0.1)), "w_pre": (1 + normal(hidden, std=0.1)),
                       "gate": normal(1, hidden, std=0.3)} for _ in range(2)]
        self.plan = ct.MoePlan(tokens, topk, experts, align=ALIGN)
        rows = self.plan.rows
        weights = [f"w{e}" for e in range(experts)]
        self.forward_meta = Fp8Meta(["x"] + weights, ct.E4M3)
        self.backward_meta = Fp8Meta(["dy"], ct.E5M2)
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.x, self.x_t = torch.empty(rows, hidden, **u8), torch.empty(hidden, rows, **u8)
        self.dy, self.dy_t = torch.empty(rows, hidden, **u8), torch.empty(hidden, rows, **u8)
        self.wq = torch.empty(experts, hidden, hidden, **u8)
        self.wq_t = torch.empty(experts, hidden, hidden, **u8)
        size = ct.block_norm_backward_workspace_size(tokens, hidden)
        self.workspace = torch.empty(size, **u8)

    # -- forward ---------------------------------------------------------------
    def junction(self, i, u, res):
        rows, n = res.shape[0], self.norms[i]
        kept = {"u": u, "res_out": torch.empty_like(res),
                "rstd_post": torch.empty(rows, device="cuda"),
                "rstd_pre": torch.empty(rows, device="cuda")}
        y = torch.empty_like(u)
        ct.block_norm(u, res, kept["res_out"], y, rstd_post=kept["rstd_post"],
                      rstd_pre=kept["rstd_pre"], **n)
        return kept, y

    def route(self, h):
        logits = (h @ self.router).float()
        best, idx = logits.topk(self.topk, dim=1)
        return torch.softmax(best, 1), idx

    def forward(self, u, res):
        """u, res [tokens, hidden] -> (res_out, out) and what backward needs."""
        m, s = self.forward_meta, {}
        s["first"], s["h"] = self.junction(0, u, res)
        s["weights"], s["idx"] = self.route(s["h"])
        ct.moe_sort(s["idx"], self.plan)
        ct.fp8_moe_dispatch(s["h"], self.plan, *m.of("x"), self.x, self.x_t, m.fmt)
        for e in range(self.experts):
            ct.fp8_cast_transpose(self.w[e], *m.of(f"w{e}"), self.wq[e], self.wq_t[e], m.fmt)
        s["ends"] = self.plan.offsets.tolist()
        s["ys"] = torch.zeros(self.plan.rows, self.hidden, dtype=BF16, device="cuda")
        for e, a, b in self.slices(s["ends"]):
            x, sx = values(self.x[a:b], m.of("x")[2], m.fmt)
            w, sw = values(self.wq[e], m.of(f"w{e}")[2], m.fmt)
            s["ys"][a:b] = (x @ w.t()).float() * (sx * sw)
        branch = torch.empty_like(u)
        ct.moe_combine(s["ys"], self.plan, s["weights"], branch)
        s["second"], out = self.junction(1, branch, s["first"]["res_out"])
        return s["second"]["res_out"], out, s

    def slices(self, ends):
        return [(e, ends[e], ends[e + 1]) for e in range(self.experts) if ends[e] < ends[e + 1]]

    # -- backward --------------------------------------------------------------
    def junction_backward(self, i, kept, dy, dres_out):
        n = self.norms[i]
        grads = {"d" + k: torch.empty_like(v) for k, v in n.items()}
        du, dres = torch.empty_like(kept["u"]), torch.empty_like(kept["res_out"])
        ct.block_norm_backward(dy, dres_out, kept["u"], kept["res_out"], kept["rstd_post"],
                               kept["rstd_pre"], du, dres, workspace=self.workspace, **n, **grads)
        return du, dres, grads

    def backward(self, s, dres_out, dout):
        m, f = self.backward_meta, self.forward_meta
        grads = {}
        dbranch, dres, grads["second"] = self.junction_backward(1, s["second"], dout, dres_out)
        # the experts' output gradients in FP8, the router's in fp32
        ct.fp8_moe_dispatch(dbranch, self.plan, *m.of("dy"), self.dy, self.dy_t, m.fmt,
                            weights=s["weights"])
        dweights = torch.empty_like(s["weights"])
        ct.moe_combine_backward(dbranch, s["ys"], self.plan, s["weights"], None, dweights)
        grads["w"] = torch.zeros_like(self.w)
        dx = torch.zeros(self.plan.rows, self.hidden, dtype=BF16, device="cuda")
        for e, a, b in self.slices(s["ends"]):
            d, sd = values(self.dy[a:b], m.of("dy")[2], m.fmt)
            d_t, _ = values(self.dy_t[:, a:b], m.of("dy")[2], m.fmt)
            x_t, sx = values(self.x_t[:, a:b], f.of("x")[2], f.fmt)
            w_t, sw = values(self.wq_t[e], f.of(f"w{e}")[2], f.fmt)
            dx[a:b] = (d @ w_t.t()).float() * (sd * sw)
            grads["w"][e] = (d_t @ x_t.t()).float() * (sd * sx)
        dh = torch.empty_like(s["h"])
        ct.moe_dispatch_backward(dx, self.plan, dh)
        # through the softmax over the chosen logits, to the router and h
        p = s["weights"]
        dlogits = torch.zeros(self.tokens, self.experts, device="cuda")
        dlogits.scatter_(1, s["idx"], p * (dweights - (p * dweights).sum(1, keepdim=True)))
        dlogits = dlogits.to(BF16)
        grads["router"] = s["h"].t() @ dlogits
        dh += dlogits @ self.router.t()
        du, dres, grads["first"] = self.junction_backward(0, s["first"], dh, dres)
        f.update()
        m.update()
        return du, dres, grads


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=3)
    p.add_argument("--hidden", type=int, default=512)
    p.add_argument("--tokens", type=int, default=1000)
    args = p.parse_args()
    block = MoeBlock(args.hidden, experts=8, topk=2, tokens=args.tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    u, res, d1, d2 = (torch.randn(args.tokens, args.hidden, generator=g, device="cuda").to(BF16)
                      for _ in range(4))
    for step in range(args.steps):
        res_out, out, saved = block.forward(u, res)
        du, dres, grads = block.backward(saved, 1e-3 * d1, 1e-3 * d2)
        print(f"step {step}: |out| {out.float().norm():.3f}  |du| {du.float().norm():.5f}  "
              f"|dw| {grads['w'].float().norm():.4f}  scale of x {block.forward_meta.scale[0]:.3f}, "
              f"of dy {block.backward_meta.scale[0]:.3e}")


if __name__ == "__main__":
    main()
