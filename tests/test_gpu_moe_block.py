"""The example block against the same block in plain torch with autograd: the
FP8 rounding of the experts' operands is the only difference that is left, so
the tolerances are those of E4M3 (2^-4 of a value at most, some 2^-5.5 of its
size on average) and, for what comes back through the experts, E5M2 (2^-3)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


def example():
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def off(got, want):
    got, want = got.double(), want.double()
    return ((got - want).norm() / want.norm()).item()


def plain(block, u, res, saved):
    """(res_out, out) in fp32, with the routing that the block chose."""
    def norm(x, w):
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * w

    def junction(n, u, res):
        res = res + n["gate"] * norm(u, n["w_post"])
        return res, norm(res, n["w_pre"])

    p = {"u": u, "res": res, "router": block.router, "w": block.w,
         **{f"{i}.{k}": v for i, n in enumerate(block.norms) for k, v in n.items()}}
    p = {k: v.detach().float().requires_grad_() for k, v in p.items()}
    n = [{k: p[f"{i}.{k}"] for k in ("w_post", "w_pre", "gate")} for i in range(2)]
    r, h = junction(n[0], p["u"], p["res"])
    weights = torch.softmax((h @ p["router"]).gather(1, saved["idx"]), 1)
    branch = torch.zeros_like(h)
    for e in range(block.experts):
        t, k = (saved["idx"] == e).nonzero(as_tuple=True)
        branch = branch.index_add(0, t, (h[t] @ p["w"][e].t()) * weights[t, k, None])
    return junction(n[1], branch, r), p


@pytest.mark.parametrize("tokens,hidden,experts,topk", [(300, 256, 8, 2), (77, 136, 5, 3), (1, 64, 4, 2)])
def test_block_against_autograd(tokens, hidden, experts, topk):
    m = example()
    block = m.MoeBlock(hidden, experts, topk, tokens, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    u, res, d1, d2 = (torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
                      for _ in range(4))
    for _ in range(2):                       # the second step has real scales
        res_out, out, saved = block.forward(u, res)
        du, dres, grads = block.backward(saved, d1, d2)
    (want_res, want_out), p = plain(block, u, res, saved)
    ((want_res * d1.float()).sum() + (want_out * d2.float()).sum()).backward()
    assert off(res_out, want_res) < 0.03 and off(out, want_out) < 0.03
    for got, name, most in ((du, "u", 0.08), (dres, "res", 0.08), (grads["w"], "w", 0.15),
                            (grads["router"], "router", 0.15), (grads["first"]["dw_pre"], "0.w_pre", 0.15),
                            (grads["first"]["dw_post"], "0.w_post", 0.08),
                            (grads["first"]["dgate"], "0.gate", 0.08),
                            (grads["second"]["dw_pre"], "1.w_pre", 0.08),
                            (grads["second"]["dw_post"], "1.w_post", 0.08),
                            (grads["second"]["dgate"], "1.gate", 0.08)):
        assert off(got, p[name].grad) < most, (name, off(got, p[name].grad))
    assert bool((block.forward_meta.scale != 1).all()) and block.backward_meta.scale.item() != 1
