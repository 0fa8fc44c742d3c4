"""The embedding and its gradient against their 64-bit forms with worst-case
bounds of the fp32 arithmetic."""
import pytest
import torch

import cast_transpose_gb300 as ct
import ops_reference as base
import step_reference as ref
from gpu_util import Guarded, scalar

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def data(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def ids(T, V, seed=0, kind="text", dtype=torch.int64):
    g = torch.Generator().manual_seed(seed + T + V)
    if kind == "text":
        idx = (torch.rand(T, generator=g, dtype=torch.float64) * torch.log(torch.tensor(V + 1.0))).exp().long() - 1
    elif kind == "uniform":
        idx = torch.randint(0, V, (T,), generator=g)
    elif kind == "one":
        idx = torch.full((T,), V // 2)
    elif kind == "two":
        idx = torch.randint(0, 2, (T,), generator=g) * (V - 1)
    elif kind == "runs":
        idx = (torch.arange(T) // 37) % V
    elif kind == "descending":
        idx = (V - 1 - torch.arange(T)) % V
    elif kind == "none":
        idx = torch.full((T,), -1)
    idx = idx.clamp(-1, V - 1)
    if kind in ("text", "uniform") and T > 4:
        idx[::5] = torch.tensor([-1, V, -7, 2 ** 31 - 1])[torch.arange(len(idx[::5])) % 4]
    return idx.to(dtype)


@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (1, 100, 4096), (5, 7, 777), (64, 1000, 1024), (300, 50, 515),
                                   (4, 30, 12288), (9, 20, 20001)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_lookup(T, V, H, dtype):
    table = data((V, H), dtype, V)
    for index in (torch.int32, torch.int64):
        idx = ids(T, V, dtype=index)
        g = Guarded(T * H, dtype=dtype)
        out = g.t.view(T, H)
        ct.embedding(idx.cuda(), table.cuda(), out, scale=1.7)
        torch.cuda.synchronize()
        g.check()
        want, err = ref.embedding(idx.long(), table, 1.7)
        base.close(out, want, base.rounded(want, err, dtype), "out")


def test_lookup_of_infinities_and_outside():
    table = data((6, 520), BF, 1)
    table[2] = float("inf")
    table[0] = float("nan")
    idx = torch.tensor([2, -1, 6, 0, 3, -2 ** 63, 2 ** 40], device="cuda")
    out = torch.full((7, 520), 7.0, dtype=BF, device="cuda")
    ct.embedding(idx, table.cuda(), out, scale=2.0)
    out = out.cpu()
    assert (out[0] == float("inf")).all() and torch.isnan(out[3]).all()
    assert not out[[1, 2, 5, 6]].any()
    ct.embedding(idx, table.cuda(), (o := torch.empty(7, 520, dtype=BF, device="cuda")), scale=float("inf"))
    assert not o.cpu()[[1, 2, 5, 6]].any()


def backward(idx, dout, V, grad, scale=1.3, old=None, shift=0):
    T, H = dout.shape
    g = Guarded(V * H, dtype=grad, offset=shift)
    out = g.t.view(V, H)
    if old is not None:
        out.copy_(old)
    ws = Guarded(ct.embedding_backward_workspace_size(T, V, H))
    ct.embedding_backward(idx.cuda(), dout.cuda(), out, ws.t, scale=scale, accumulate=old is not None)
    torch.cuda.synchronize()
    g.check()
    ws.check()
    want, err, some = ref.embedding_backward(idx.long(), dout, V, scale, old)
    base.close(out, want, base.rounded(want, err, grad), "dtable")
    if old is not None:
        assert torch.equal(out.cpu()[~some], old[~some])
    else:
        assert not out.cpu()[~some].any()
    return out


SIZES = [(1, 1, 1), (1, 100, 4096), (5, 7, 777), (64, 1000, 1024), (300, 50, 515), (40, 30, 12288),
         (2100, 700, 264), (3, 20, 20001), (5000, 40000, 40), (9000, 3, 72)]


@pytest.mark.parametrize("T,V,H", SIZES)
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (HF, HF), (HF, F32), (F32, F32)])
def test_gradient(T, V, H, types):
    idx, dout = ids(T, V, dtype=torch.int32), data((T, H), types[0], T)
    backward(idx, dout, V, types[1])
    backward(idx.long(), dout, V, types[1], old=data((V, H), types[1], 3))


@pytest.mark.parametrize("kind", ["uniform", "one", "two", "runs", "descending", "none"])
@pytest.mark.parametrize("T,V,H", [(33, 10, 64), (1024, 400, 264), (1025, 400, 264), (500, 3, 2056), (512, 90, 1032), (513, 90, 1032), (4097, 300, 72), (4096, 70000, 8), (20000, 2000, 16),
                                   (1000, 65536, 13), (70000, 257, 8), (300000, 1 << 18, 1)])
def test_distributions(kind, T, V, H):
    idx, dout = ids(T, V, kind=kind), data((T, H), BF, T)
    backward(idx, dout, V, F32)
    if T < 10000:
        backward(idx, dout, V, BF, old=data((V, H), BF, 3))


def test_gradient_of_odd_addresses():
    idx, dout = ids(200, 30), data((200, 520), BF, 4)
    n = dout.numel()
    for i in (1, 3):
        odd = torch.cat([dout.reshape(-1)[:i], dout.reshape(-1)]).cuda()[i:i + n].view(dout.shape)
        T, V, H = 200, 30, 520
        out = torch.empty(V, H, dtype=BF, device="cuda")
        ws = torch.empty(ct.embedding_backward_workspace_size(T, V, H), dtype=torch.uint8, device="cuda")
        ct.embedding_backward(idx.cuda(), odd, out, ws)
        want, err, _ = ref.embedding_backward(idx, dout, V, 1.0)
        base.close(out, want, base.rounded(want, err, BF), "dtable")
        backward(idx, dout, V, BF, shift=i)


def test_what_padding_rows_hold_does_not_matter():
    idx, dout = ids(500, 40), data((500, 72), BF, 4)
    dout[(idx < 0) | (idx >= 40)] = float("nan")
    clean = torch.where(((idx < 0) | (idx >= 40))[:, None], 0.0, dout.float()).to(BF)
    assert torch.equal(backward(idx, clean, 40, F32), run(idx, dout, 40))


def run(idx, dout, V):
    out = torch.empty(V, dout.shape[1], device="cuda")
    ws = torch.empty(ct.embedding_backward_workspace_size(len(idx), V, dout.shape[1]), dtype=torch.uint8,
                     device="cuda")
    ct.embedding_backward(idx.cuda(), dout.cuda(), out, ws, scale=1.3)
    return out


def test_the_same_from_call_to_call():
    idx, dout = ids(20000, 3000), data((20000, 264), BF, 4)
    assert torch.equal(run(idx, dout, 3000), run(idx, dout, 3000))


def test_no_tokens_and_noop():
    out = torch.full((9, 24), 7.0, device="cuda")
    ws = torch.empty(ct.embedding_backward_workspace_size(50, 9, 24), dtype=torch.uint8, device="cuda")
    none, rows = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 24, device="cuda")
    ct.embedding_backward(none, rows, out, ws, accumulate=True)
    assert (out == 7).all()
    idx, dout = ids(50, 9).cuda(), torch.ones(50, 24, device="cuda")
    ct.embedding_backward(idx, dout, out, ws, noop_flag=scalar(1.0))
    ct.embedding_backward(idx, dout, out, ws, accumulate=True, noop_flag=scalar(1.0))
    ct.embedding(idx, out, dout, noop_flag=scalar(1.0))
    assert (out == 7).all() and (dout == 1).all()
    ct.embedding_backward(none, rows, out, ws)
    assert not out.any()
    ct.embedding(none, out, rows)


def test_offsets_past_32_bits():
    """A table of more than 2^32 bytes, of which the first and last rows are used."""
    V, H = 600000, 4096
    table = torch.zeros(V, H, dtype=BF, device="cuda")
    table[-1], table[-300000] = 2.0, 3.0
    idx = torch.tensor([V - 1, 0, V - 300000], device="cuda")
    out = torch.empty(3, H, dtype=BF, device="cuda")
    ct.embedding(idx, table, out)
    assert (out[0] == 2).all() and not out[1].any() and (out[2] == 3).all()
    ws = torch.empty(ct.embedding_backward_workspace_size(3, V, H), dtype=torch.uint8, device="cuda")
    table.fill_(9.0)
    ct.embedding_backward(idx, out, table, ws)
    assert (table[-1] == 2).all() and (table[-300000] == 3).all() and not table[0].any()
    assert table.sum(dtype=torch.float64).item() == 5.0 * H


def test_gradient_past_32_bits():
    """More than 2^31 elements of gradients come in, of many tokens."""
    T, V, H = 600000, 100, 4096
    idx = torch.arange(T, device="cuda") % V
    dout = torch.ones(T, H, dtype=BF, device="cuda")
    dout[-1] = 3.0
    out = torch.empty(V, H, device="cuda")
    ws = torch.empty(ct.embedding_backward_workspace_size(T, V, H), dtype=torch.uint8, device="cuda")
    ct.embedding_backward(idx, dout, out, ws)
    assert (out[:-1] == T // V).all() and (out[-1] == T // V + 2).all()
