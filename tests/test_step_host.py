"""Host-side refusals of dropout, layer norm, router and embedding (no GPU
needed): status codes of the C ABI and errors of the binding.  The pointers
passed are never dereferenced."""
import pytest
import torch

import cast_transpose_gb300 as ct
from cast_transpose_gb300.moe import _router_config
from cast_transpose_gb300.norms import _pack_layer_config

OK, NULL, SHAPE, ALIGN, FORMAT, ARG, ALIAS, WORKSPACE = range(8)
A, B, C, D, E, F, G, H, I, J, K, M = (0x100000000 * (i + 1) for i in range(12))
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    return ct.lib()


def test_dropout_rejects(L):
    def call(x=A, rows=10, cols=64, dtype=0, p=0.1, rng=B, site=0, out=C):
        return L.dropout(x, rows, cols, dtype, p, rng, site, out, None, None)
    assert call(dtype=3) == FORMAT
    for kw in (dict(rows=-1), dict(cols=-1), dict(rows=2 ** 31), dict(cols=2 ** 30 + 1),
               dict(rows=2 ** 20, cols=2 ** 21)):
        assert call(**kw) == SHAPE
    for p in (-0.1, 1.0, 1.5, NAN, 0.999999):
        assert call(p=p) == ARG
    for kw in (dict(x=None), dict(out=None), dict(rng=None)):
        assert call(**kw) == NULL
    for kw in (dict(x=A + 1), dict(out=C + 1), dict(rng=B + 4), dict(dtype=2, x=A + 2)):
        assert call(**kw) == ALIGN
    for kw in (dict(out=A + 2), dict(out=B - 8), dict(out=A - 2)):
        assert call(**kw) == ALIAS
    assert call(rows=0, x=None) == OK and call(cols=0, out=None) == OK


def config(**kw):
    c = dict(rows=10, hidden=64, weight=K, bias=M, rng=J, eps=1e-5, weight_offset=0.0, p=0.1, site=0, dtype=0,
             res_dtype=0, param_dtype=0)
    c.update({k: v for k, v in kw.items() if k in c})
    return _pack_layer_config(*(0 if v is None else v for v in c.values())), {k: v for k, v in kw.items() if k not in c}


def test_layer_norm_rejects(L):
    def call(**kw):
        cfg, kw = config(**kw)
        a = dict(u=A, res=B, res_out=C, y=D, mean=E, rstd=F, scale=None, amax=None, si=None, fmt=0)
        a.update(kw)
        return L.layer_norm(cfg, *a.values(), None, None)
    assert L.layer_norm(None, A, B, C, D, E, F, None, None, None, 0, None, None) == NULL
    for kw in (dict(dtype=3), dict(dtype=0, res_dtype=1), dict(dtype=1, res_dtype=0), dict(param_dtype=1),
               dict(dtype=2, res_dtype=0), dict(scale=G, amax=H, si=I, fmt=2)):
        assert call(**kw) == FORMAT
    for kw in (dict(rows=-1), dict(hidden=-1), dict(hidden=32769), dict(rows=2 ** 31)):
        assert call(**kw) == SHAPE
    for kw in (dict(eps=-1.0), dict(eps=NAN), dict(p=1.0), dict(p=-0.5), dict(p=NAN), dict(u=None)):
        assert call(**kw) == ARG
    for kw in (dict(res=None), dict(res_out=None), dict(y=None), dict(rng=None), dict(scale=G, amax=H),
               dict(scale=G, si=H)):
        assert call(**kw) == NULL
    for kw in (dict(u=A + 1), dict(res=B + 1), dict(mean=E + 2), dict(rng=J + 4), dict(weight=K + 1),
               dict(scale=G + 1, amax=H, si=I), dict(param_dtype=2, bias=M + 2)):
        assert call(**kw) == ALIGN
    for kw in (dict(res_out=A), dict(res_out=B + 2), dict(y=A), dict(y=B), dict(y=C), dict(rstd=E), dict(mean=K),
               dict(y=J), dict(scale=G, amax=G, si=I)):
        assert call(**kw) == ALIAS
    assert call(rows=0, y=None) == OK and call(hidden=0, res=None) == OK


def test_layer_norm_backward_rejects(L):
    def call(**kw):
        cfg, kw = config(**kw)
        a = dict(dy=A, dres_out=B, res_out=C, mean=D, rstd=E, dres=F, du=G, dweight=H, dbias=I, ws=J + 4096,
                 wsb=1 << 30)
        a.update(kw)
        return L.layer_norm_backward(cfg, *a.values(), None, None)
    for kw in (dict(dtype=-1), dict(res_dtype=1), dict(param_dtype=1)):
        assert call(**kw) == FORMAT
    for kw in (dict(rows=-1), dict(hidden=32769)):
        assert call(**kw) == SHAPE
    assert call(p=1.0) == ARG
    for kw in (dict(dy=None), dict(res_out=None), dict(mean=None), dict(rstd=None), dict(dres=None),
               dict(rng=None)):
        assert call(**kw) == NULL
    for kw in (dict(dy=A + 1), dict(du=G + 1), dict(dbias=I + 1), dict(rstd=E + 2)):
        assert call(**kw) == ALIGN
    for kw in (dict(dres=A), dict(dres=B), dict(dres=C), dict(du=F), dict(dweight=I), dict(dbias=K), dict(du=A)):
        assert call(**kw) == ALIAS
    need = L.layer_norm_backward_workspace_size(8192, 4096)
    assert need > 0 and L.layer_norm_backward_workspace_size(-1, 64) == 0
    big = dict(rows=8192, hidden=4096)
    far = {k: 0x100000000000 * (i + 1) for i, k in enumerate(("dy", "dres_out", "res_out", "mean", "rstd", "dres",
                                                             "du", "dweight", "dbias"))}
    for kw in (dict(ws=None), dict(wsb=need - 1)):
        assert call(**big, **far, **kw) == WORKSPACE
    assert call(**big, **far, ws=J + 4) == ALIGN
    assert call(**big, **far, ws=far["dres"]) == ALIAS
    assert call(hidden=0) == OK


def router(**kw):
    c = dict(tokens=10, experts=8, topk=2, dtype=2, flags=1, balance=0.1, z=0.1)
    c.update({k: v for k, v in kw.items() if k in c})
    return _router_config(*c.values()), {k: v for k, v in kw.items() if k not in c}


BAD_ROUTERS = [(dict(dtype=3), FORMAT), (dict(experts=0), ARG), (dict(experts=1025), ARG), (dict(topk=0), ARG),
               (dict(topk=9), ARG), (dict(experts=100, topk=65), ARG), (dict(flags=2), ARG),
               (dict(tokens=-1), SHAPE), (dict(tokens=2 ** 30), SHAPE)]


def test_router_rejects(L):
    def call(**kw):
        cfg, kw = router(**kw)
        a = dict(logits=A, mask=B, idx=C, weights=D, counts=E, loss=F, ws=G, wsb=1 << 30)
        a.update(kw)
        return L.moe_router(cfg, *a.values(), None, None)
    assert L.moe_router(None, A, B, C, D, E, F, G, 0, None, None) == NULL
    for kw, status in BAD_ROUTERS:
        assert call(**kw) == status
    for kw in (dict(logits=None), dict(idx=None), dict(weights=None), dict(counts=None)):
        assert call(**kw) == NULL
    for kw in (dict(logits=A + 2), dict(idx=C + 2), dict(loss=F + 1)):
        assert call(**kw) == ALIGN
    for kw in (dict(idx=A), dict(weights=C), dict(counts=B), dict(loss=E + 32), dict(weights=A + 16)):
        assert call(**kw) == ALIAS
    need = L.moe_router_workspace_size(100000, 2, 8)
    assert need > 0
    for kw in (dict(ws=None), dict(wsb=need - 1)):
        assert call(tokens=100000, **kw) == WORKSPACE
    assert call(tokens=100000, ws=G + 4) == ALIGN
    for bad in ((-1, 2, 8), (10, 0, 8), (10, 65, 100), (10, 2, 0), (10, 2, 1025), (2 ** 31, 1, 8)):
        assert L.moe_router_workspace_size(*bad) == 0


def test_router_backward_rejects(L):
    def call(**kw):
        cfg, kw = router(**kw)
        a = dict(logits=A, mask=B, idx=C, counts=D, dweights=E, dloss=F, dlogits=G)
        a.update(kw)
        return L.moe_router_backward(cfg, *a.values(), None, None)
    for kw, status in BAD_ROUTERS:
        assert call(**kw) == status
    for kw in (dict(logits=None), dict(idx=None), dict(counts=None), dict(dlogits=None),
               dict(dweights=None, dloss=None)):
        assert call(**kw) == NULL
    assert call(dlogits=G + 2) == ALIGN and call(dloss=F + 2) == ALIGN
    assert call(dlogits=A) == ALIAS and call(dlogits=E + 4) == ALIAS
    assert call(tokens=0) == OK


def test_embedding_rejects(L):
    def call(idx=A, ib=8, tokens=10, table=B, vocab=100, hidden=64, dtype=0, out=C):
        return L.embedding(idx, ib, tokens, table, vocab, hidden, dtype, 1.0, out, None, None)
    assert call(ib=2) == FORMAT and call(dtype=3) == FORMAT
    for kw in (dict(tokens=-1), dict(tokens=2 ** 31), dict(vocab=-1), dict(vocab=2 ** 31), dict(hidden=-1),
               dict(hidden=2 ** 20 + 1), dict(vocab=2 ** 21, hidden=2 ** 20)):
        assert call(**kw) == SHAPE
    for kw in (dict(idx=None), dict(table=None), dict(out=None)):
        assert call(**kw) == NULL
    assert call(idx=A + 4) == ALIGN and call(table=B + 1) == ALIGN and call(out=C + 1) == ALIGN
    assert call(out=B + 2) == ALIAS and call(out=A) == ALIAS
    assert call(tokens=0) == OK and call(hidden=0) == OK


def test_embedding_backward_rejects(L):
    def call(idx=A, ib=8, tokens=10, dout=B, vocab=100, hidden=64, dtype=0, dtable=C, grad=2, acc=0, ws=D,
             wsb=1 << 30):
        return L.embedding_backward(idx, ib, tokens, dout, vocab, hidden, dtype, 1.0, dtable, grad, acc, ws, wsb,
                                    None, None)
    assert call(ib=3) == FORMAT and call(dtype=-1) == FORMAT and call(grad=1) == FORMAT
    assert call(acc=2) == ARG
    for kw in (dict(tokens=-1), dict(vocab=2 ** 31), dict(hidden=2 ** 20 + 1)):
        assert call(**kw) == SHAPE
    for kw in (dict(idx=None), dict(dout=None), dict(dtable=None)):
        assert call(**kw) == NULL
    assert call(dtable=C + 2) == ALIGN
    assert call(dtable=B) == ALIAS and call(dtable=A) == ALIAS
    need = L.embedding_backward_workspace_size(5000, 100, 64)
    assert need > 0 and L.embedding_backward_workspace_size(10, 100, 64) == 0
    assert call(tokens=5000, ws=None) == WORKSPACE and call(tokens=5000, wsb=need - 1) == WORKSPACE
    assert call(tokens=5000, ws=D + 4) == ALIGN and call(tokens=5000, ws=B) == ALIAS
    assert call(hidden=0) == OK and call(vocab=0) == OK and call(tokens=0, acc=1) == OK
    for bad in ((-1, 10, 10), (10, -1, 10), (10, 10, -1), (2 ** 31, 1, 1)):
        assert L.embedding_backward_workspace_size(*bad) == 0


# ---- the binding: what it refuses before any address is taken
class Fake:
    """In place of the library: every call is kept."""
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return getattr(self.real, name)
        return lambda *args: self.calls.append((name, args)) or 0


MODULES = ("dropouts", "embeddings", "moe", "norms")


@pytest.fixture
def fake(monkeypatch, L):
    """CPU tensors pass for the device's, and calls go to a recorder."""
    import importlib
    f = Fake(L)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(ct, "_stream", lambda stream: 0)
    for m in MODULES:
        monkeypatch.setattr(importlib.import_module("cast_transpose_gb300." + m), "lib", lambda: f)
    return f


BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 8, dtype=BF)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ct.dropout(x, x.clone(), 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        ct.layer_norm(x, x.clone(), x.clone(), x.clone())
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        ct.embedding(torch.zeros(3, dtype=torch.int64), x, x.clone())


def test_dropout_binding(fake):
    x, out, rng = torch.zeros(4, 8, dtype=BF), torch.zeros(4, 8, dtype=BF), torch.zeros(2, dtype=torch.int64)
    ct.dropout(x, out, 0.25, rng, 9)
    name, a = fake.calls.pop()
    assert name == "dropout" and a[1:5] == (4, 8, 0, 0.25) and a[6] == 9
    for args, error, match in (
            ((x[:, ::2], out, 0.1, rng), ValueError, "contiguous"),
            ((x, out.float(), 0.1, rng), TypeError, "out has dtype"),
            ((x, out[:3], 0.1, rng), ValueError, "out has shape"),
            ((x.int(), out, 0.1, rng), TypeError, "x has dtype"),
            ((x[0], out, 0.1, rng), ValueError, "2-D"),
            ((x, out, 0.1, None), ValueError, "rng"),
            ((x, out, 0.1, rng.int()), TypeError, "rng has dtype"),
            ((x, out, 0.1, rng[:1]), ValueError, "rng has shape"),
            ((x, out, 0.1, rng, -1), ValueError, "site"),
            ((x, out, 0.1, rng, 1 << 32), ValueError, "site")):
        with pytest.raises(error, match=match):
            ct.dropout(*args)
    assert not fake.calls


def test_layer_norm_binding(fake):
    x = torch.zeros(4, 8, dtype=BF)
    w, stats = torch.zeros(8, dtype=BF), torch.zeros(4)
    ct.layer_norm(x, x, x, x, weight=w, bias=w, mean=stats, rstd=stats)
    ct.layer_norm(None, x, None, x, bias=w.float())
    assert [c[0] for c in fake.calls] == ["layer_norm"] * 2
    fake.calls.clear()
    for kw, error, match in ((dict(weight=w, bias=w.float()), TypeError, "bias has dtype"),
                             (dict(weight=w[:4]), ValueError, "weight has shape"),
                             (dict(weight=3.0), TypeError, "weight must be"),
                             (dict(mean=stats[:3]), ValueError, "mean has shape"),
                             (dict(rstd=stats.half()), TypeError, "rstd has dtype"),
                             (dict(p=0.1), ValueError, "rng")):
        with pytest.raises(error, match=match):
            ct.layer_norm(x, x, x, x, **kw)
    with pytest.raises(TypeError, match="u must be"):
        ct.layer_norm(3, x, x, x)
    with pytest.raises(TypeError, match="y must be"):
        ct.layer_norm(None, x)
    with pytest.raises(ValueError, match="dweight has shape"):
        ct.layer_norm_backward(x, x, x, stats, stats, x, dweight=stats.to(BF))
    with pytest.raises(TypeError, match="dbias has dtype"):
        ct.layer_norm_backward(x, x, x, stats, stats, x, dweight=w, dbias=w.float())
    with pytest.raises(ValueError, match="mean"):
        ct.layer_norm_backward(x, x, x, stats[:2], stats, x)
    with pytest.raises(TypeError, match="mean must be"):
        ct.layer_norm_backward(x, x, x, None, stats, x)
    with pytest.raises(TypeError, match="int32"):
        ct.layer_norm(x.int(), x.int(), x.int(), x.int())
    assert not fake.calls


def test_router_binding(fake):
    x, idx, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=I32), torch.zeros(4, 2)
    counts, loss, mask = torch.zeros(9, dtype=I32), torch.zeros(1), torch.ones(4, dtype=torch.bool)
    ct.moe_router(x, idx, w, counts, loss, mask=mask)
    ct.moe_router(x, idx, w, counts, mask=mask.to(torch.uint8))
    ct.moe_router_backward(w, loss, x, idx, counts, x.clone(), mask=mask)
    assert len(fake.calls) == 3
    fake.calls.clear()
    for args, error, match in (((x, idx.long(), w, counts), TypeError, "expert_idx has dtype"),
                               ((x, idx[:3], w, counts), ValueError, "expert_idx has shape"),
                               ((x, idx, w[:, :1], counts), ValueError, "weights has shape"),
                               ((x, idx, w, counts[:8]), ValueError, "counts has shape"),
                               ((x[0], idx, w, counts), ValueError, "2-D"),
                               ((x.double(), idx, w, counts), TypeError, "logits has dtype")):
        with pytest.raises(error, match=match):
            ct.moe_router(*args)
    for mask in (torch.ones(4), torch.ones(3, dtype=torch.bool)):
        with pytest.raises((TypeError, ValueError), match="mask has"):
            ct.moe_router(x, idx, w, counts, mask=mask)
    with pytest.raises(TypeError, match="dlogits has dtype"):
        ct.moe_router_backward(w, loss, x, idx, counts, x.half())
    assert not fake.calls


def test_embedding_binding(fake):
    idx, table, out = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8), torch.zeros(3, 8)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    ct.embedding(idx, table, out)
    ct.embedding_backward(idx, out.half(), table, ws)
    assert len(fake.calls) == 2
    fake.calls.clear()
    for args, error, match in (((idx.float(), table, out), TypeError, "idx has dtype"),
                               ((idx[None], table, out), ValueError, "1-D"),
                               ((idx, table, out.half()), TypeError, "out has dtype"),
                               ((idx, table, out[:2]), ValueError, "out has shape"),
                               ((idx, table.t(), out), ValueError, "contiguous|out has shape")):
        with pytest.raises(error, match=match):
            ct.embedding(*args)
    for args, error, match in (((idx, out, table.half(), ws), TypeError, "dtable has dtype"),
                               ((idx, out, table[:, :4], ws), ValueError, "columns"),
                               ((idx, out[:2], table, ws), ValueError, "dout has shape"),
                               ((idx, out, table, ws.int()), TypeError, "workspace has dtype")):
        with pytest.raises(error, match=match):
            ct.embedding_backward(*args)
    assert not fake.calls


def test_another_device_is_refused(fake, monkeypatch):
    x, rng = torch.zeros(4, 8, dtype=BF), torch.zeros(2, dtype=torch.int64)
    out = torch.zeros(4, 8, dtype=BF)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1 if t is rng else 0)
    with pytest.raises(ValueError, match="rng is on cuda:1"):
        ct.dropout(x, out, 0.1, rng)
    flag = torch.zeros(1)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1 if t is flag else 0)
    with pytest.raises(ValueError, match="noop_flag is on cuda:1"):
        ct.dropout(x, out, 0.1, rng, noop_flag=flag)
    space = torch.zeros(1 << 16, dtype=torch.uint8)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1 if t is space else 0)
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        ct.embedding_backward(torch.zeros(4, dtype=torch.int64), x, out, space)

    class Stream:
        device_index, cuda_stream = 1, 0
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        ct.dropout(x, out, 0.0, None, stream=Stream())
    assert not fake.calls
