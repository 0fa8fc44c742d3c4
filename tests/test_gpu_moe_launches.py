"""Expert movement as programs launch it: from several host threads, for many
experts, right behind the library's own kernels, with a plan per layer."""
import threading

import pytest
import torch

import cast_transpose_gb300 as ct
import ops_reference as ref
from test_gpu_moe import check_plan, data, routing, sorted_plan

pytestmark = pytest.mark.gpu


# one block, a cluster, a grid, each with more than 48 KB of counts
@pytest.mark.parametrize("tokens,topk", [(3, 4), (250, 4), (2000, 4), (6000, 4), (9000, 4)])
@pytest.mark.parametrize("experts", [326, 512, 1024])
def test_sort_into_many_experts(tokens, topk, experts):
    idx = routing(tokens, topk, experts, tokens + experts)
    check_plan(sorted_plan(idx, experts, 16), idx)


def test_sorts_of_different_expert_counts_from_two_threads():
    """What one call allows its kernel must not be taken back by another's."""
    sizes, failed = {1024: 1000, 384: 1000}, []
    start = threading.Barrier(len(sizes))
    checks = []

    def work(experts, tokens):
        try:
            idx = routing(tokens, 4, experts, experts)
            plan = ct.MoePlan(tokens, 4, experts, align=16)
            gpu, stream = idx.cuda(), torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            start.wait(60)
            for _ in range(4000):
                ct.moe_sort(gpu, plan, stream=stream)
            stream.synchronize()
            checks.append((plan, idx))
        except Exception as e:  # noqa: BLE001 (reported by the main thread)
            failed.append(f"{experts} experts: {e!r}")

    threads = [threading.Thread(target=work, args=a) for a in sizes.items()]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for plan, idx in checks:
        check_plan(plan, idx)


def test_layers_with_a_plan_each():
    """Two layers forward, then both backward: each gets its own routing's
    gradients, as from a plan that was sorted for it alone."""
    tokens, topk, experts, hidden = 300, 2, 6, 64
    layers = []
    for seed in (1, 2):
        idx = routing(tokens, topk, experts, seed).cuda()
        layers.append((idx, ct.MoePlan(tokens, topk, experts, align=16)))
    w = data((tokens, topk), torch.float32, 3).cuda()
    x, dout = data((tokens, hidden), torch.float32, 4).cuda(), data((tokens, hidden), torch.float32, 5).cuda()

    def forward(idx, plan):
        ct.moe_sort(idx, plan)
        ys = torch.empty(plan.rows, hidden, device="cuda")
        ct.moe_dispatch(x, plan, ys)
        return ys

    def backward(plan, ys):
        dys, dw, dx = torch.empty_like(ys), torch.empty_like(w), torch.empty_like(x)
        ct.moe_combine_backward(dout, ys, plan, w, dys, dw)
        ct.moe_dispatch_backward(dys, plan, dx)
        return dys, dw, dx

    kept = [forward(*layer) for layer in layers]
    got = [backward(layer[1], ys) for layer, ys in zip(reversed(layers), reversed(kept))]
    for (idx, _), ys, grads in zip(layers, kept, reversed(got)):
        alone = ct.MoePlan(tokens, topk, experts, align=16)
        assert torch.equal(forward(idx, alone), ys)
        for a, b in zip(grads, backward(alone, ys)):
            assert torch.equal(a, b)
        rows = ref.sort(idx.cpu(), experts, 16, alone.rows)[0]
        want, err, want_w, err_w = ref.combine_backward(dout.cpu(), ys.cpu(), rows, w.cpu(), alone.rows)
        ref.close(grads[0], want, ref.rounded(want, err, torch.float32), "dys")
        ref.close(grads[1], want_w, err_w + 1e-38, "dweights")


# The writers let their successor start at their first instruction, so that its
# prefetch of x runs while they write: moe_combine and moe_dispatch_backward for
# tens of microseconds, the few-row norm for a few.
def write_combine(state, i):
    ct.moe_combine(state["ys"][i], state["plan"], state["w"], state["x"])


def write_dispatch_backward(state, i):
    ct.moe_dispatch_backward(state["ys"][i], state["plan"], state["x"])


def write_norm(state, i):
    u = state["ys"][i][:len(state["x"])]
    ct.block_norm(u, state["res"], state["res_out"], state["x"])


@pytest.mark.parametrize("sort_between", [False, True])
@pytest.mark.parametrize("writer,tokens", [(write_combine, 4000), (write_dispatch_backward, 4000),
                                           (write_norm, 60)])
def test_dispatch_of_what_the_kernel_before_writes(writer, tokens, sort_between):
    """x has new values each time, from a kernel of the library right before the
    dispatch, or before its sort, without a pause in the stream."""
    topk, experts, hidden, times = 4, 16, 4096, 5
    idx = routing(tokens, topk, experts, 97).cuda()
    plan, source = (ct.MoePlan(tokens, topk, experts, align=16) for _ in range(2))
    ct.moe_sort(idx, plan)
    ct.moe_sort(idx, source)
    state = {"plan": source, "w": torch.rand(tokens, topk, device="cuda"),
             "ys": [torch.randn(source.rows, hidden, device="cuda").to(torch.bfloat16)
                    for _ in range(times)],
             "res": torch.ones(tokens, hidden, device="cuda", dtype=torch.bfloat16),
             "res_out": torch.empty(tokens, hidden, device="cuda", dtype=torch.bfloat16),
             "x": torch.zeros(tokens, hidden, device="cuda", dtype=torch.bfloat16)}
    outs = [torch.empty(plan.rows, hidden, device="cuda", dtype=torch.bfloat16) for _ in range(times)]
    for _ in range(3):
        torch.cuda.synchronize()
        for i in range(times):
            writer(state, i)
            if sort_between:
                ct.moe_sort(idx, plan)
            ct.moe_dispatch(state["x"], plan, outs[i])
        torch.cuda.synchronize()
        slot = plan.src.clamp(min=0).long()
        kept = (plan.src >= 0)[:, None]
        for i in range(times):
            writer(state, i)
            torch.cuda.synchronize()
            assert torch.equal(outs[i], torch.where(kept, state["x"][slot // topk], 0.0))
            outs[i].fill_(float("nan"))
