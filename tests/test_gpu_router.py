"""The router of a mixture-of-experts block, forward and backward, against its
64-bit form with worst-case bounds of the fp32 arithmetic."""
import numpy as np
import pytest
import torch

import cast_transpose_gb300 as ct
import ops_reference as base
import step_reference as ref
from gpu_util import Guarded, scalar

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")


class Case:
    def __init__(self, T, E, K, dtype=F32, normalize=True, masked=False, balance=0.3, z=0.02, seed=0, std=1.0):
        g = torch.Generator().manual_seed(seed + T + E)
        self.logits = (torch.randn(T, E, generator=g) * std + torch.randn(1, E, generator=g)).to(dtype)
        self.mask = torch.rand(T, generator=g) > 0.3 if masked else None
        self.dweights = torch.randn(T, K, generator=g)
        self.T, self.E, self.K, self.dtype = T, E, K, dtype
        self.kw = dict(normalize=normalize, balance=balance, z=z)
        self.dloss = 1.5

    def reference(self):
        return ref.Router(self.logits, self.mask, self.K, **self.kw).forward()

    def forward(self, loss=True, noop=None):
        T, E, K = self.T, self.E, self.K
        g = {"expert_idx": Guarded(T * K, dtype=torch.int32), "weights": Guarded(T * K, dtype=F32),
             "counts": Guarded(E + 1, dtype=torch.int32), "loss": Guarded(1, dtype=F32)}
        out = {k: v.t.view(T, K) if k in ("expert_idx", "weights") else v.t for k, v in g.items()}
        if not loss:
            out["loss"] = None
        ws = Guarded(ct.moe_router_workspace_size(T, K, E))
        ct.moe_router(self.logits.cuda(), mask=None if self.mask is None else self.mask.cuda(), workspace=ws.t,
                      noop_flag=noop, **out, **self.kw)
        torch.cuda.synchronize()
        ws.check()
        for v in g.values():
            v.check()
        return out

    def check(self):
        out, w = self.forward(), self.reference()
        assert torch.equal(out["expert_idx"].cpu(), w.idx)
        assert torch.equal(out["counts"].cpu(), w.counts)
        base.close(out["weights"], w.weights, w.w_err, "weights")
        base.close(out["loss"], w.loss.view(1), torch.as_tensor(w.loss_err).view(1) + 1e-37, "loss")
        return w

    def backward(self, dweights=True, dloss=True):
        w = self.reference()
        g = Guarded(self.T * self.E, dtype=self.dtype)
        dl = g.t.view(self.T, self.E)
        dw, d = self.dweights if dweights else None, self.dloss if dloss else None
        ct.moe_router_backward(None if dw is None else dw.cuda(), None if d is None else scalar(d),
                               self.logits.cuda(), w.idx.cuda(), w.counts.cuda(), dl,
                               mask=None if self.mask is None else self.mask.cuda(), **self.kw)
        torch.cuda.synchronize()
        g.check()
        value, err = w.backward(dw, d or 0.0)
        base.close(dl, value, base.rounded(value, err, self.dtype), "dlogits")
        return dl


SIZES = [(1, 1, 1), (1, 8, 2), (4, 64, 4), (7, 8, 8), (5, 33, 3), (33, 128, 8), (64, 256, 8), (9, 300, 5),
         (3, 1024, 40), (2, 1000, 64), (300, 64, 6), (1000, 16, 2), (2600, 8, 1), (700, 256, 8), (513, 1024, 4)]


@pytest.mark.parametrize("T,E,K", SIZES)
@pytest.mark.parametrize("normalize", [False, True])
def test_forward_and_backward(T, E, K, normalize):
    c = Case(T, E, K, normalize=normalize, masked=T > 3)
    c.check()
    c.backward()


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("normalize", [False, True])
def test_types(dtype, normalize):
    """Half of bf16's logits here share their value with another."""
    for E in (8, 64, 200):
        c = Case(257, E, min(E, 6), dtype=dtype, normalize=normalize, masked=True)
        c.check()
        c.backward()


def test_equal_logits_go_to_the_lowest_index():
    for E, K in ((8, 3), (64, 64), (256, 8), (1000, 7)):
        c = Case(40, E, K)
        c.logits.fill_(0.25)
        c.check()
        c.logits[:, 1::2] = 0.5
        c.check()
        c.logits.zero_()
        c.logits[:, ::3] = -0.0            # equal to 0
        c.check()


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_a_few_equal_logits_of_either_sign(dtype):
    """Groups of equal logits at the choice's edge, fewer than a warp has lanes."""
    for E, K in ((100, 5), (128, 16), (256, 8), (1024, 30)):
        c = Case(60, E, K, dtype=dtype)
        g = torch.Generator().manual_seed(E)
        high = torch.rand(60, E, generator=g) < 20 / E
        level = torch.randint(0, 4, (60, E), generator=g).float()
        c.logits = torch.where(high, level * 0.25 - 1.0, c.logits.float() - 50.0).to(dtype)
        c.logits[30:][high[30:] & (level[30:] == 0)] = 300.0
        c.logits[20:30][high[20:30] & (level[20:30] == 3)] = -0.0
        w = c.check()
        assert len(set(w.idx[0].tolist())) == K
        c.backward()


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("lowest", [-INF, torch.finfo(F32).min])
def test_masked_experts(normalize, lowest):
    c = Case(50, 40, 4, normalize=normalize)
    c.logits[:, 5:30] = lowest
    c.logits[3] = lowest                    # -inf: a padding token
    c.logits[4, 2:] = lowest                # two experts left
    c.logits[5, 1:] = lowest                # one
    if lowest != -INF:
        c.kw["z"] = 0.0                     # its logsumexp's square is past fp32
        c.logits[3] = 1.0
    w = c.check()
    c.backward()
    if lowest == -INF:
        assert w.idx[3].tolist() == [-1] * 4 and w.idx[4, 2:].tolist() == [-1] * 2
        assert w.counts[-1] == 49


def test_a_row_of_the_lowest_number_without_a_z_loss():
    """A mask by the lowest number that leaves a token nothing; its logsumexp's
    square, past fp32, counts for nothing."""
    for T in (4, 2000):
        c = Case(T, 40, 4)
        c.logits[3] = torch.finfo(F32).min
        c.kw["z"] = 0.0
        c.check()
        c.backward()


def test_all_padding():
    for T in (3, 900):
        c = Case(T, 16, 2, masked=True)
        c.mask.zero_()
        c.logits.fill_(float("nan"))
        out = c.forward()
        assert (out["expert_idx"] == -1).all() and not out["weights"].any()
        assert not out["counts"].any() and out["loss"].item() == 0.0
        dl = torch.full((T, 16), 7.0, device="cuda")
        ct.moe_router_backward(torch.full((T, 2), float("nan"), device="cuda"), scalar(1.0), c.logits.cuda(),
                               out["expert_idx"], out["counts"], dl, mask=c.mask.cuda(), **c.kw)
        assert not dl.any()


@pytest.mark.parametrize("normalize", [False, True])
def test_what_a_padding_token_holds_does_not_matter(normalize):
    c = Case(70, 24, 3, normalize=normalize, masked=True)
    clean = c.forward()
    clean_dl = c.backward()
    c.logits[~c.mask] = torch.tensor([float("nan"), INF, -INF]).repeat(8)
    c.dweights[~c.mask] = float("nan")
    dirty = c.forward()
    for k in clean:
        assert torch.equal(clean[k], dirty[k]), k
    dl = torch.empty_like(clean_dl)
    ct.moe_router_backward(c.dweights.cuda(), scalar(c.dloss), c.logits.cuda(), dirty["expert_idx"],
                           dirty["counts"], dl, mask=c.mask.cuda(), **c.kw)
    assert torch.equal(dl, clean_dl)


def test_a_nan_is_chosen_first_and_spoils_its_token_alone():
    c = Case(20, 16, 2)
    c.logits[7, 3] = float("nan")
    out = c.forward()
    assert out["expert_idx"][7, 0].item() == 3
    assert torch.isnan(out["weights"][7]).all() and torch.isnan(out["loss"]).item()
    others = torch.arange(20) != 7
    w = c.reference()
    base.close(out["weights"].cpu()[others], w.weights[others], w.w_err[others], "weights")


def test_dropped_slots_gradients_are_not_read():
    """Experts left out after the choice (a slot set to -1, out of range)."""
    for normalize in (False, True):
        c = Case(30, 16, 4, normalize=normalize)
        w = c.reference()
        idx, dw = w.idx.clone(), c.dweights.clone()
        idx[::3, 1], idx[1::3, 3] = -1, 16
        dw[idx < 0] = float("nan")
        dw[idx >= 16] = float("nan")
        dl = torch.empty(30, 16, device="cuda")
        ct.moe_router_backward(dw.cuda(), scalar(1.0), c.logits.cuda(), idx.cuda(), w.counts.cuda(), dl, **c.kw)
        assert torch.isfinite(dl).all()


@pytest.mark.parametrize("normalize", [False, True])
def test_an_expert_twice(normalize):
    """idx as another choice may leave it: each slot counts."""
    for E, K in ((16, 4), (64, 3), (256, 8), (1000, 32), (1000, 40)):
        c = Case(45, E, K, normalize=normalize)
        w = c.reference()
        w.idx[::2, 1] = w.idx[::2, 0]
        w.idx[::4] = w.idx[::4, :1].clone()
        w.weights = w.p.gather(1, w.idx.long())
        if normalize:
            w.weights /= w.weights.sum(1, keepdim=True)
        value, err = w.backward(c.dweights, c.dloss)
        dl = torch.empty(45, E, device="cuda")
        ct.moe_router_backward(c.dweights.cuda(), scalar(c.dloss), c.logits.cuda(), w.idx.cuda(), w.counts.cuda(), dl,
                               **c.kw)
        base.close(dl, value, base.rounded(value, err, F32), "dlogits")


def test_a_part_of_the_gradient():
    for normalize in (False, True):
        c = Case(90, 40, 4, normalize=normalize)
        c.backward(dweights=False)
        c.backward(dloss=False)
        c.forward(loss=False)


def test_large_logits():
    c = Case(40, 32, 4, std=60.0)
    c.check()
    c.backward()


def test_no_tokens():
    c = Case(0, 8, 2)
    out = c.forward()
    assert not out["counts"].any() and out["loss"].item() == 0.0


def test_noop_flag():
    for T in (4, 2000):
        c = Case(T, 16, 2)
        idx, counts = (torch.full(s, 7, dtype=torch.int32, device="cuda") for s in ((T, 2), (17,)))
        w, loss, dl = (torch.full(s, 7.0, device="cuda") for s in ((T, 2), (1,), (T, 16)))
        ws = torch.empty(ct.moe_router_workspace_size(T, 2, 16), dtype=torch.uint8, device="cuda")
        ct.moe_router(c.logits.cuda(), idx, w, counts, loss, workspace=ws, noop_flag=scalar(1.0))
        ct.moe_router_backward(w, loss, c.logits.cuda(), idx, counts, dl, noop_flag=scalar(1.0))
        for t in (idx, counts, w, loss, dl):
            assert (t == 7).all()


def test_the_same_from_call_to_call():
    c = Case(3000, 64, 4)
    one, two = c.forward(), c.forward()
    for k in one:
        assert torch.equal(one[k], two[k])


def test_offsets_past_32_bits():
    """More than 2^31 logits: the last tokens are those of a small call."""
    T, E, K, last = 2100003, 1024, 2, 5
    logits = torch.empty(T, E, dtype=BF, device="cuda").normal_()
    idx, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    counts = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(ct.moe_router_workspace_size(T, K, E), dtype=torch.uint8, device="cuda")
    ct.moe_router(logits, idx, w, counts, workspace=ws)
    r = ref.Router(logits[-last:].cpu(), None, K, True, 0.0, 0.0).forward()
    assert torch.equal(idx[-last:].cpu(), r.idx) and counts[E].item() == T
    assert counts[:E].sum().item() == T * K
    base.close(w[-last:], r.weights, r.w_err, "weights")
    dl = torch.empty_like(logits)
    ct.moe_router_backward(torch.ones(T, K, device="cuda") * torch.tensor([1.0, -1.0], device="cuda"), None, logits,
                           idx, counts, dl)
    value, err = r.backward(torch.tensor([[1.0, -1.0]]).expand(last, K), 0.0)
    base.close(dl[-last:], value, base.rounded(value, err, BF), "dlogits")
