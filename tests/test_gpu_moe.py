"""Tokens sorted by expert and back, against plain 64-bit forms: every shape
class of the movement (whole 16-byte rows, odd rows), one token to many,
dropped slots, experts without tokens, capacities that are too small."""
import numpy as np
import pytest
import torch

import cast_transpose_gb300 as ct
import ops_reference as ref
import oracle
from gpu_util import Guarded, f32_bits, scalar

pytestmark = pytest.mark.gpu

TYPES = (torch.bfloat16, torch.float16, torch.float32)


def routing(tokens, topk, experts, seed, kind="skewed"):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":                       # every token to the same experts
        return torch.arange(topk).repeat(tokens, 1).int() % experts
    if kind == "none":                      # only padding tokens
        return torch.full((tokens, topk), -1).int()
    logits = torch.randn(tokens, experts, generator=g) + 1.5 * torch.randn(1, experts, generator=g)
    idx = logits.topk(min(topk, experts), dim=1).indices
    if topk > experts:
        idx = torch.cat([idx] * -(-topk // experts), 1)[:, :topk]
    drop = torch.rand(tokens, topk, generator=g)
    idx[drop < 0.05] = -1
    idx[drop > 0.97] = experts + 7          # outside: dropped as well
    return idx.int().contiguous()


def guarded_plan(tokens, topk, experts, align, rows=None):
    rows = ct.moe_sorted_rows(tokens, topk, experts, align) if rows is None else rows
    bufs = {"row_of": (tokens, topk), "src": (rows,), "offsets": (experts + 1,),
            "counts": (experts,)}
    guards = {k: Guarded(int(np.prod(s)), dtype=torch.int32) for k, s in bufs.items()}
    plan = ct.MoePlan(tokens, topk, experts, align=align, rows=rows,
                      **{k: guards[k].t.view(bufs[k]) for k in bufs})
    return plan, guards


def sorted_plan(idx, experts, align, rows=None):
    plan, guards = guarded_plan(idx.shape[0], idx.shape[1], experts, align, rows)
    ct.moe_sort(idx.cuda(), plan)
    torch.cuda.synchronize()
    for g in guards.values():
        g.check()
    return plan


def check_plan(plan, idx):
    want = ref.sort(idx, plan.experts, plan.align, plan.rows)
    for name, w in zip(("row_of", "src", "offsets", "counts"), want):
        got = getattr(plan, name).cpu().numpy()
        assert np.array_equal(got, w), (name, np.argwhere(got != w)[:3].tolist())
    return want


SORTS = [(1, 1, 1, 1), (1, 4, 64, 1), (1, 8, 256, 16), (3, 2, 5, 16), (33, 3, 7, 1),
         (257, 8, 8, 32), (1000, 4, 64, 16), (4099, 2, 1, 16), (777, 64, 1024, 1),
         (5001, 6, 160, 128), (8191, 8, 256, 16), (30011, 4, 33, 7)]


@pytest.mark.parametrize("tokens,topk,experts,align", SORTS)
def test_sort(tokens, topk, experts, align):
    idx = routing(tokens, topk, experts, tokens + experts)
    check_plan(sorted_plan(idx, experts, align), idx)


@pytest.mark.parametrize("kind", ["one", "none"])
@pytest.mark.parametrize("tokens", [1, 700, 20000])
def test_sort_one_sided(kind, tokens):
    idx = routing(tokens, 3, 16, 1, kind)
    check_plan(sorted_plan(idx, 16, 16), idx)


@pytest.mark.parametrize("tokens,rows", [(700, 0), (700, 1), (700, 1111), (20000, 30001)])
def test_sort_capacity_too_small(tokens, rows):
    idx = routing(tokens, 3, 16, 2)
    check_plan(sorted_plan(idx, 16, 16, rows), idx)


def test_sort_no_tokens_and_int64_and_repeats():
    idx = torch.zeros(0, 4).int()
    plan = sorted_plan(idx, 8, 16, rows=48)
    check_plan(plan, idx)
    idx = routing(3001, 4, 24, 3)
    plan, _ = guarded_plan(3001, 4, 24, 16)
    for _ in range(3):                      # the plan's buffers are rewritten
        ct.moe_sort(idx.long().cuda(), plan)
    big = idx.long()
    big[5, 1] = 2 ** 32 + 3                 # not expert 3
    torch.cuda.synchronize()
    check_plan(plan, idx)
    ct.moe_sort(big.cuda(), plan)
    idx[5, 1] = -1
    check_plan(plan, idx)


SHAPES = [(1, 1, 1, 1, 8), (1, 8, 64, 1, 4096), (5, 4, 16, 16, 1), (67, 2, 8, 16, 777),
          (130, 3, 9, 1, 1000), (90, 3, 8, 16, 1002), (40, 2, 4, 4, 30), (300, 8, 32, 16, 520), (64, 5, 6, 32, 12288), (513, 4, 16, 16, 257)]


def data(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,topk,experts,align,hidden", SHAPES)
def test_dispatch_and_backward(tokens, topk, experts, align, hidden, dtype):
    idx = routing(tokens, topk, experts, 7)
    plan = sorted_plan(idx, experts, align)
    row_of, src = ref.sort(idx, experts, align, plan.rows)[:2]
    x = data((tokens, hidden), dtype, 8)
    out = Guarded(plan.rows * hidden, dtype=dtype)
    ct.moe_dispatch(x.cuda(), plan, out.t.view(plan.rows, hidden))
    out.check()
    want = torch.zeros(plan.rows, hidden, dtype=dtype)
    kept = src >= 0
    want[kept] = x[src[kept] // topk]
    got = out.t.view(plan.rows, hidden).cpu()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    dout = data((plan.rows, hidden), dtype, 9)
    dout[torch.as_tensor(~kept)] = float("nan")     # padding rows are not read
    dx = Guarded(tokens * hidden, dtype=dtype)
    ct.moe_dispatch_backward(dout.cuda(), plan, dx.t.view(tokens, hidden))
    dx.check()
    want, err = ref.combine(dout, row_of, None)
    ref.close(dx.t.view(tokens, hidden), want, ref.rounded(want, err, dtype), "dx")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,topk,experts,align,hidden", SHAPES)
def test_combine_and_backward(tokens, topk, experts, align, hidden, dtype):
    idx = routing(tokens, topk, experts, 17)
    plan = sorted_plan(idx, experts, align)
    row_of, src = ref.sort(idx, experts, align, plan.rows)[:2]
    pad = torch.as_tensor(src < 0)
    ys, dout = data((plan.rows, hidden), dtype, 18), data((tokens, hidden), dtype, 19)
    ys[pad] = float("inf")
    weights = data((tokens, topk), torch.float32, 20)
    weights[torch.as_tensor(row_of < 0)] = float("nan")     # of dropped slots: not used
    out = Guarded(tokens * hidden, dtype=dtype)
    ct.moe_combine(ys.cuda(), plan, weights.cuda(), out.t.view(tokens, hidden))
    out.check()
    want, err = ref.combine(ys, row_of, weights)
    ref.close(out.t.view(tokens, hidden), want, ref.rounded(want, err, dtype), "out")
    dys, dw = Guarded(plan.rows * hidden, dtype=dtype), Guarded(tokens * topk, dtype=torch.float32)
    ct.moe_combine_backward(dout.cuda(), ys.cuda(), plan, weights.cuda(),
                            dys.t.view(plan.rows, hidden), dw.t.view(tokens, topk))
    dys.check()
    dw.check()
    want, err, want_w, err_w = ref.combine_backward(dout, ys, row_of, weights, plan.rows)
    got = dys.t.view(plan.rows, hidden)
    ref.close(got, want, ref.rounded(want, err, dtype), "dys")
    assert not got.cpu()[pad].any()
    ref.close(dw.t.view(tokens, topk), want_w, err_w + 1e-38, "dweights")
    # either gradient alone
    dw2 = torch.full((tokens, topk), 7.0, device="cuda")
    ct.moe_combine_backward(dout.cuda(), ys.cuda(), plan, weights.cuda(), None, dw2)
    assert torch.equal(dw2, dw.t.view(tokens, topk))
    dys2 = torch.full((plan.rows, hidden), 7.0, dtype=dtype, device="cuda")
    ct.moe_combine_backward(dout.cuda(), None, plan, weights.cuda(), dys2, None)
    assert torch.equal(dys2, got)


@pytest.mark.parametrize("shift", [1, 2, 4])
@pytest.mark.parametrize("dtype", TYPES)
def test_unaligned_buffers(dtype, shift):
    """Buffers that start off a 16-byte boundary."""
    tokens, topk, experts, hidden = 50, 4, 8, 256
    idx = routing(tokens, topk, experts, 27)
    plan = sorted_plan(idx, experts, 16)
    row_of, src = ref.sort(idx, experts, 16, plan.rows)[:2]

    def off(t):
        b = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        b[shift:] = t.reshape(-1).cuda()
        return b[shift:].view(t.shape)

    x, ys = data((tokens, hidden), dtype, 28), data((plan.rows, hidden), dtype, 29)
    weights = data((tokens, topk), torch.float32, 30)
    got = off(torch.empty(plan.rows, hidden, dtype=dtype))
    ct.moe_dispatch(off(x), plan, got)
    kept = src >= 0
    assert torch.equal(got.cpu()[kept], x[src[kept] // topk]) and not got.cpu()[~kept].any()
    out = off(torch.empty(tokens, hidden, dtype=dtype))
    ct.moe_combine(off(ys), plan, weights.cuda(), out)
    want, err = ref.combine(ys, row_of, weights)
    ref.close(out, want, ref.rounded(want, err, dtype), "out")
    dys, dw = off(torch.empty_like(ys)), torch.empty(tokens, topk, device="cuda")
    ct.moe_combine_backward(off(x), off(ys), plan, weights.cuda(), dys, dw)
    want, err, want_w, err_w = ref.combine_backward(x, ys, row_of, weights, plan.rows)
    ref.close(dys, want, ref.rounded(want, err, dtype), "dys")
    ref.close(dw, want_w, err_w, "dweights")


def test_no_tokens_and_no_rows():
    plan = sorted_plan(torch.zeros(0, 2).int(), 4, 16, rows=32)
    out = torch.full((32, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    ct.moe_dispatch(torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), plan, out)
    assert not out.any()
    out.fill_(3.0)
    none = torch.empty(0, 2, device="cuda")
    ct.moe_combine_backward(torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), None, plan,
                            none, out, None)
    assert not out.any()
    idx = routing(9, 2, 4, 5)
    plan = sorted_plan(idx, 4, 1, rows=0)       # every slot dropped
    y = torch.full((9, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    empty = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(9, 2, device="cuda")
    ct.moe_combine(empty, plan, w, y)
    assert not y.any()
    dw = torch.ones(9, 2, device="cuda")
    ct.moe_combine_backward(y, empty, plan, w, None, dw)
    assert not dw.any()


def test_indexes_outside_the_buffers_are_dropped():
    """A plan that was not made by moe_sort cannot send a kernel out of range."""
    plan = sorted_plan(routing(10, 2, 4, 5), 4, 16)
    x = data((10, 64), torch.bfloat16, 1).cuda()
    plan.row_of.fill_(plan.rows + 5)
    plan.src.fill_(10 ** 9)
    out = Guarded(plan.rows * 64, dtype=torch.bfloat16)
    ct.moe_dispatch(x, plan, out.t.view(plan.rows, 64))
    out.check()
    assert not out.t.any()
    y = Guarded(10 * 64, dtype=torch.bfloat16)
    ct.moe_combine(out.t.view(plan.rows, 64), plan, torch.ones(10, 2, device="cuda"),
                   y.t.view(10, 64))
    y.check()
    assert not y.t.any()
    q, qt = torch.ones(plan.rows, 64, device="cuda").byte(), torch.ones(64, plan.rows).byte().cuda()
    ct.fp8_moe_dispatch(x, plan, scalar(1.0), scalar(0.0), scalar(0.0), q, qt)
    assert not q.any() and not qt.any()


# ---------------------------------------------------------------- FP8
FP8_SHAPES = SHAPES + [(700, 4, 16, 16, 1024), (1500, 2, 8, 128, 640), (900, 3, 5, 1, 144),
                       (260, 2, 4, 16, 24), (5000, 8, 64, 16, 384)]


@pytest.mark.parametrize("fmt", [ct.E4M3, ct.E5M2])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("tokens,topk,experts,align,hidden", FP8_SHAPES)
def test_fp8_dispatch(tokens, topk, experts, align, hidden, weighted, fmt):
    """Bit for bit the cast-transpose of the weighted, sorted rows."""
    idx = routing(tokens, topk, experts, 37)
    plan = sorted_plan(idx, experts, align)
    rows = plan.rows
    src = ref.sort(idx, experts, align, rows)[1]
    x = data((tokens, hidden), torch.bfloat16, 38)
    if hidden > 8:
        x[0, 1], x[tokens // 2, 3], x[-1, 5] = -0.0, 1e-30, 3e4
    weights = data((tokens, topk), torch.float32, 39)
    scale = 448.0 / 5.5
    q, qt = Guarded(rows * hidden), Guarded(rows * hidden)
    s, amax, sinv = scalar(scale), scalar(0.25), scalar(-1.0)
    ct.fp8_moe_dispatch(x.cuda(), plan, s, amax, sinv, q.t.view(rows, hidden),
                        qt.t.view(hidden, rows), fmt, weights=weights.cuda() if weighted else None)
    q.check()
    qt.check()
    kept = src >= 0
    v = torch.zeros(rows, hidden)
    v[kept] = x[src[kept] // topk].float()
    if weighted:
        v[kept] *= weights.reshape(-1)[src[kept]][:, None]
    want = oracle.fp8_encode(np.ascontiguousarray((v * s.cpu()).numpy()), fmt).reshape(rows, hidden)
    got = q.numpy().reshape(rows, hidden)
    assert np.array_equal(got, want), np.argwhere(got != want)[:4].tolist()
    assert np.array_equal(qt.numpy().reshape(hidden, rows), want.T)
    assert f32_bits(amax.item()) == f32_bits(max(0.25, v.abs().max().item() if v.numel() else 0.0))
    assert f32_bits(sinv.item()) == f32_bits(1.0 / np.float32(scale))
    q2 = Guarded(rows * hidden)
    ct.fp8_moe_dispatch(x.cuda(), plan, s, amax, sinv, q2.t.view(rows, hidden), None, fmt,
                        weights=weights.cuda() if weighted else None)
    q2.check()
    assert torch.equal(q2.t, q.t)


@pytest.mark.parametrize("hidden,align", [(256, 16), (100, 1)])
def test_fp8_dispatch_special_values(hidden, align):
    idx = routing(40, 2, 4, 47)
    idx[:4] = torch.tensor([0, 1])
    plan = sorted_plan(idx, 4, align)
    src = ref.sort(idx, 4, align, plan.rows)[1]
    x = data((40, hidden), torch.bfloat16, 48)
    x[1, 2], x[2, 7], x[3, 9] = float("inf"), float("-inf"), float("nan")
    q = torch.empty(plan.rows, hidden, dtype=torch.uint8, device="cuda")
    qt = torch.empty(hidden, plan.rows, dtype=torch.uint8, device="cuda")
    amax, sinv = scalar(0.0), scalar(0.0)
    ct.fp8_moe_dispatch(x.cuda(), plan, scalar(2.0), amax, sinv, q, qt, ct.E4M3)
    v = torch.zeros(plan.rows, hidden)
    kept = src >= 0
    v[kept] = x[src[kept] // 2].float()
    want = oracle.fp8_encode((v * 2.0).numpy(), ct.E4M3).reshape(v.shape)
    assert np.array_equal(q.cpu().numpy(), want) and np.array_equal(qt.cpu().numpy(), want.T)
    assert np.isnan(amax.item())


@pytest.mark.parametrize("offset", [1, 4, 8])
def test_fp8_dispatch_unaligned_outputs(offset):
    idx = routing(200, 2, 4, 57)
    plan = sorted_plan(idx, 4, 16)
    x = data((200, 128), torch.bfloat16, 58).cuda()
    outs = []
    for o in (0, offset):
        q, qt = Guarded(plan.rows * 128, offset=o), Guarded(plan.rows * 128, offset=o)
        ct.fp8_moe_dispatch(x, plan, scalar(50.0), scalar(0.0), scalar(0.0),
                            q.t.view(-1, 128), qt.t.view(128, -1))
        q.check()
        qt.check()
        outs.append((q.t.clone(), qt.t.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("hidden", [1000, 24])
@pytest.mark.parametrize("weighted", [False, True])
def test_fp8_dispatch_many_tiles(hidden, weighted):
    """More tiles than a wave of blocks: strips of tiles, then single ones."""
    tokens, topk, experts = 31000, 4, 32
    idx = routing(tokens, topk, experts, 87)
    plan = sorted_plan(idx, experts, 16)
    x = data((tokens, hidden), torch.bfloat16, 88).cuda()
    weights = data((tokens, topk), torch.float32, 89).cuda()
    scale, amax, sinv = scalar(70.0), scalar(0.0), scalar(0.0)
    q = torch.empty(plan.rows, hidden, dtype=torch.uint8, device="cuda")
    qt = torch.empty(hidden, plan.rows, dtype=torch.uint8, device="cuda")
    ct.fp8_moe_dispatch(x, plan, scale, amax, sinv, q, qt, weights=weights if weighted else None)
    slot = torch.as_tensor(ref.sort(idx, experts, 16, plan.rows)[1]).cuda().long()
    v = torch.where((slot >= 0)[:, None], x[slot.clamp(min=0) // topk].float(), 0.0)
    if weighted:
        v = torch.where((slot >= 0)[:, None], v * weights.reshape(-1)[slot.clamp(min=0)][:, None], 0.0)
    want = (v * scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(q, want) and torch.equal(qt, want.t())
    assert f32_bits(amax.item()) == f32_bits(v.abs().max().item())


# ---------------------------------------------------------------- gradients and use
def test_gradients_against_differences():
    """<gradient, direction> against central differences of the 64-bit forward
    (which is linear in each argument: no truncation error)."""
    tokens, topk, experts, hidden = 40, 3, 6, 96
    idx = routing(tokens, topk, experts, 67)
    plan = sorted_plan(idx, experts, 16)
    row_of, src = ref.sort(idx, experts, 16, plan.rows)[:2]
    ys, weights = data((plan.rows, hidden), torch.float32, 68), data((tokens, topk), torch.float32, 69)
    dout = data((tokens, hidden), torch.float32, 70)
    dys, dw = torch.empty(plan.rows, hidden).cuda(), torch.empty(tokens, topk).cuda()
    ct.moe_combine_backward(dout.cuda(), ys.cuda(), plan, weights.cuda(), dys, dw)

    def loss(y, w):
        return (ref.combine(y, row_of, w)[0] * dout.double()).sum()

    for seed in range(3):
        a = data(ys.shape, torch.float64, seed)
        b = data(weights.shape, torch.float64, seed + 10)
        for moved, slope in (((ys + 0.5 * a, weights), (ys - 0.5 * a, weights)),
                             (dys.cpu().double() * a).sum()), \
                            (((ys, weights + 0.5 * b), (ys, weights - 0.5 * b)),
                             (dw.cpu().double() * b).sum()):
            diff = loss(*moved[0]) - loss(*moved[1])
            assert abs(diff - slope) <= 1e-4 * max(1.0, abs(diff)), (diff, slope)


def test_noop_flag_stream_and_graph():
    tokens, topk, experts, hidden = 300, 4, 8, 512
    idx = routing(tokens, topk, experts, 77)
    x, w = data((tokens, hidden), torch.bfloat16, 78).cuda(), data((tokens, topk), torch.float32, 79).cuda()
    plan, _ = guarded_plan(tokens, topk, experts, 16)
    rows = plan.rows
    bufs = [plan.row_of, plan.src, plan.offsets, plan.counts,
            torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda"),
            torch.empty(rows, hidden, dtype=torch.uint8, device="cuda"),
            torch.empty(hidden, rows, dtype=torch.uint8, device="cuda"), scalar(0.0), scalar(0.0),
            torch.empty_like(x), torch.empty_like(x),
            torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda"), torch.empty_like(w)]
    gidx, flag, scale = idx.cuda(), scalar(0.0), scalar(40.0)

    def step(noop=None):
        ct.moe_sort(gidx, plan, noop_flag=noop)
        ct.moe_dispatch(x, plan, bufs[4], noop_flag=noop)
        ct.fp8_moe_dispatch(x, plan, scale, bufs[7], bufs[8], bufs[5], bufs[6], weights=w,
                            noop_flag=noop)
        ct.moe_dispatch_backward(bufs[4], plan, bufs[9], noop_flag=noop)
        ct.moe_combine(bufs[4], plan, w, bufs[10], noop_flag=noop)
        ct.moe_combine_backward(x, bufs[4], plan, w, bufs[11], bufs[12], noop_flag=noop)

    step()
    want = [b.clone() for b in bufs]
    for b in bufs:
        b.fill_(9)
    flag.fill_(1.0)
    step(flag)
    assert all(bool((b == 9).all()) for b in bufs)
    flag.fill_(0.0)
    bufs[7].zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(flag)
    side.synchronize()
    assert all(torch.equal(b, v) for b, v in zip(bufs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(flag)
    for k in range(2):
        for b in bufs:
            b.fill_(0 if b is bufs[7] else 9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b, v) for b, v in zip(bufs, want))


def test_dispatch_sees_x_written_by_the_preceding_kernel():
    """x is asked for in L2 while the kernel before still runs: what that kernel
    writes is what is moved."""
    tokens, topk, experts, hidden = 4000, 4, 16, 4096
    idx = routing(tokens, topk, experts, 97)
    plan = sorted_plan(idx, experts, 16)
    kept = plan.src >= 0
    slot = plan.src.clamp(min=0).long()
    x = data((tokens, hidden), torch.bfloat16, 98).cuda()
    out = torch.empty(plan.rows, hidden, dtype=torch.bfloat16, device="cuda")
    for i in range(20):
        x.neg_()
        if i % 2:
            ct.moe_sort(idx.cuda(), plan)
            x.neg_()
        ct.moe_dispatch(x, plan, out)
        want = torch.where(kept[:, None], x[slot // topk], 0.0)
        assert torch.equal(out, want)


def test_offsets_past_32_bits():
    """Sorted buffers of more than 2^31 elements: the last rows are right."""
    tokens, topk, hidden = 33000, 8, 8192
    idx = torch.zeros(tokens, topk).int()
    plan = sorted_plan(idx, 1, 1)
    assert plan.rows * hidden > 2 ** 31
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    x[-1] = 2.0
    out = torch.full((plan.rows, hidden), 5.0, dtype=torch.bfloat16, device="cuda")
    ct.moe_dispatch(x, plan, out)
    assert bool((out[-topk:] == 2.0).all()) and not out[:-topk].any()
    y = torch.empty_like(x)
    ct.moe_dispatch_backward(out, plan, y)
    assert bool((y[-1] == 2.0 * topk).all()) and not y[:-1].any()
    q = torch.empty(plan.rows, hidden, dtype=torch.uint8, device="cuda")
    qt = torch.empty(hidden, plan.rows, dtype=torch.uint8, device="cuda")
    amax = scalar(0.0)
    ct.fp8_moe_dispatch(x, plan, scalar(1.0), amax, scalar(0.0), q, qt)
    two = int(oracle.fp8_encode(np.array([2.0], np.float32), ct.E4M3)[0])
    assert bool((q[-topk:] == two).all()) and not q[:-topk].any()
    assert bool((qt[:, -topk:] == two).all()) and not qt[:, :-topk].any()
    assert amax.item() == 2.0
