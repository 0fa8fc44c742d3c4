"""The dropout / residual sum / layer norm junction and the dropout alone,
against their 64-bit forms with worst-case bounds of the fp32 arithmetic."""
import numpy as np
import pytest
import torch

import cast_transpose_gb300 as ct
import ops_reference as base
import oracle
import step_reference as ref
from gpu_util import Guarded, f32_bits, scalar

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [(BF, BF, BF), (BF, F32, F32), (HF, HF, HF), (HF, F32, HF), (F32, F32, F32), (BF, BF, F32)]
EPS, SEED, STEP, SITE = 1e-5, 0x123456789ABCDEF0, 0x7FFFFFFFF, 0xFFFFFFFE


def data(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def state(seed=SEED, step=STEP):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


class Case:
    def __init__(self, rows, hidden, dtype=BF, res=BF, param=BF, p=0.1, offset=0.0, u=True,
                 weight=True, bias=True, mean=0.5, eps=EPS, seed=0):
        self.rows, self.hidden, self.dtype, self.rdtype, self.pdtype = rows, hidden, dtype, res, param
        shape = rows, hidden
        self.u = data(shape, dtype, seed + 1, 0.7) if u else None
        self.res = data(shape, res, seed + 2, 2.0, mean)
        self.weight = data((hidden,), param, seed + 3, 0.2, 1 - offset) if weight else None
        self.bias = data((hidden,), param, seed + 4, 0.2) if bias else None
        self.dy, self.dres_out = data(shape, dtype, seed + 6, 0.3), data(shape, res, seed + 7, 0.3)
        self.eps, self.offset, self.p = eps, offset, p
        self.factor = ref.drop_factor(rows, hidden, p, SEED, STEP, SITE)
        self.kw = dict(weight_offset=offset, p=p, site=SITE, rng=state() if p else None,
                       weight=self.weight.cuda() if weight else None)
        self.want = ref.LayerNorm(self.u, self.res, self.weight, self.bias, eps, offset, self.factor)

    def forward(self, in_place=False, fp8=None, shift=0, **more):
        n, shape = self.rows * self.hidden, (self.rows, self.hidden)
        guards = {"mean": Guarded(self.rows, dtype=F32), "rstd": Guarded(self.rows, dtype=F32),
                  "y": Guarded(n, dtype=self.dtype if fp8 is None else torch.uint8, offset=shift)}
        if self.u is not None:
            guards["res_out"] = Guarded(n, dtype=self.rdtype, offset=shift)
        out = {k: g.t.view(shape) if k in ("y", "res_out") else g.t for k, g in guards.items()}
        res = self.res.cuda()
        if in_place:
            out["res_out"] = res
        if fp8 is not None:
            more = dict(scale=scalar(fp8[1]), amax=scalar(0.0), scale_inv=scalar(-1.0), fmt=fp8[0])
        ct.layer_norm(None if self.u is None else self.u.cuda(), res, eps=self.eps,
                      bias=None if self.bias is None else self.bias.cuda(), **self.kw, **out, **more)
        torch.cuda.synchronize()
        for g in guards.values():
            g.check()
        return {**out, **more}

    def check_forward(self, **kw):
        out, w = self.forward(**kw), self.want.forward()
        if self.u is not None:
            base.close(out["res_out"], w.out, base.rounded(w.out, w.out_err, self.rdtype), "res_out")
        base.close(out["mean"], w.mean, w.mean_err + 2 * ref.F * w.mean.abs(), "mean")
        base.close(out["rstd"], w.rstd, w.rstd_err, "rstd")
        if out["y"].dtype != torch.uint8:
            base.close(out["y"], w.y, base.rounded(w.y, w.y_err, self.dtype), "y")
        return out, w

    def backward(self, which=("du", "dweight", "dbias"), dres_out=True, shift=0, noop=None):
        w = self.want.forward()
        kept = (w.out if self.u is not None else self.res.double()).to(self.rdtype)
        mean, rstd = w.mean.float(), w.rstd.float()
        n, shape = self.rows * self.hidden, (self.rows, self.hidden)
        g = {"dres": Guarded(n, dtype=self.rdtype, offset=shift)}
        if "du" in which:
            g["du"] = Guarded(n, dtype=self.dtype, offset=shift)
        for k in ("dweight", "dbias"):
            if k in which:
                g[k] = Guarded(self.hidden, dtype=self.pdtype)
        out = {k: v.t.view(shape) if k[:2] != "db" and k != "dweight" else v.t for k, v in g.items()}
        ws = Guarded(ct.layer_norm_backward_workspace_size(self.rows, self.hidden))
        dr = self.dres_out if dres_out else None
        ct.layer_norm_backward(self.dy.cuda(), None if dr is None else dr.cuda(), kept.cuda(), mean.cuda(),
                               rstd.cuda(), workspace=ws.t, noop_flag=noop, **out, **self.kw)
        torch.cuda.synchronize()
        ws.check()
        for v in g.values():
            v.check()
        return out, w.backward(self.dy, dr, kept, mean, rstd)

    def check_backward(self, **kw):
        got, want = self.backward(**kw)
        types = {"du": self.dtype, "dres": self.rdtype}
        for k, t in got.items():
            value, err = want[k]
            base.close(t, value, base.rounded(value, err, types.get(k, self.pdtype)), k)
        return got


SHAPES = [(1, 8), (1, 4096), (3, 1), (5, 777), (2, 1000), (64, 520), (37, 2048), (130, 4099), (9, 6144),
          (4, 8200), (21, 12288), (3, 12287), (2, 16384), (2, 24584), (3, 32768), (2, 32767), (1000, 264),
          (700, 1032), (650, 777), (400, 6144)]


@pytest.mark.parametrize("rows,hidden", SHAPES)
def test_forward_and_backward(rows, hidden):
    c = Case(rows, hidden)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("rows,hidden", [(7, 1024), (400, 1024), (5, 333), (700, 333), (2, 20000)])
@pytest.mark.parametrize("types", TYPES)
def test_types(rows, hidden, types):
    c = Case(rows, hidden, *types, p=0.3, offset=1.0)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.5, 0.99])
@pytest.mark.parametrize("hidden", [512, 513])
def test_shares(p, hidden):
    c = Case(33, hidden, p=p)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("rows,hidden", [(4, 2048), (500, 2048), (4, 515), (700, 515)])
@pytest.mark.parametrize("kw", [dict(u=False, p=0.0), dict(weight=False), dict(bias=False),
                                dict(weight=False, bias=False, p=0.0)])
def test_without(rows, hidden, kw):
    c = Case(rows, hidden, **kw)
    c.check_forward()
    c.check_backward(dres_out=False)
    c.check_backward(which=())
    c.check_backward(which=("dweight",))
    c.check_backward(which=("dbias", "du"))


@pytest.mark.parametrize("rows,hidden", [(4, 4096), (300, 4096), (4, 777), (600, 777)])
def test_a_mean_far_from_zero(rows, hidden):
    """A row's mean a thousand times its deviation: nothing may cancel."""
    c = Case(rows, hidden, F32, F32, F32, u=False, p=0.0, mean=2000.0)
    out, w = c.check_forward()
    assert (w.rstd_err / w.rstd).max() < 1.2e-1       # that the bound says something
    assert torch.allclose(out["rstd"].cpu().double(), w.rstd, rtol=1e-3)
    c.check_backward()


@pytest.mark.parametrize("hidden", [1, 8, 300, 4096])
def test_a_constant_row(hidden):
    """Variance 0: rstd is 1 / sqrt(eps) and y the bias."""
    c = Case(3, hidden, F32, F32, F32, u=False, p=0.0)
    c.res.fill_(3.0)
    c.want = ref.LayerNorm(None, c.res, c.weight, c.bias, EPS, 0.0, c.factor)
    out = c.forward()
    assert torch.equal(out["mean"].cpu(), torch.full((3,), 3.0))
    assert torch.allclose(out["rstd"].cpu(), torch.full((3,), EPS ** -0.5), rtol=1e-6)
    assert torch.equal(out["y"].cpu(), c.bias.expand(3, -1))


@pytest.mark.parametrize("rows,hidden", [(5, 4096), (500, 4096), (600, 333)])
@pytest.mark.parametrize("shift", [1, 2])
def test_misaligned(rows, hidden, shift):
    c = Case(rows, hidden)
    c.check_forward(shift=shift)
    c.check_backward(shift=shift)


@pytest.mark.parametrize("rows,hidden", [(500, 333), (9, 777)])
def test_inputs_at_odd_addresses(rows, hidden):
    """Views that begin in the middle of 16 bytes, at the ends of their storage."""
    c = Case(rows, hidden)

    def odd(t):
        n = t.numel()
        return torch.cat([t.reshape(-1)[:3], t.reshape(-1)]).cuda()[3:3 + n].view(t.shape)
    out = {k: torch.empty(rows, hidden, dtype=BF, device="cuda") for k in ("res_out", "y")}
    stats = {k: torch.empty(rows, device="cuda") for k in ("mean", "rstd")}
    kw = {**c.kw, "weight": odd(c.weight)}
    ct.layer_norm(odd(c.u), odd(c.res), bias=odd(c.bias), eps=EPS, **kw, **out, **stats)
    w = c.want.forward()
    base.close(out["y"], w.y, base.rounded(w.y, w.y_err, BF), "y")
    g = {k: torch.empty(rows, hidden, dtype=BF, device="cuda") for k in ("dres", "du")}
    ws = torch.empty(ct.layer_norm_backward_workspace_size(rows, hidden), dtype=torch.uint8, device="cuda")
    grads = {k: torch.empty(hidden, dtype=BF, device="cuda") for k in ("dweight", "dbias")}
    kept, mean, rstd = w.out.to(BF), w.mean.float(), w.rstd.float()
    ct.layer_norm_backward(odd(c.dy), odd(c.dres_out), odd(kept), mean.cuda(), rstd.cuda(), workspace=ws,
                           **kw, **g, **grads)
    want = w.backward(c.dy, c.dres_out, kept, mean, rstd)
    for k, t in {**g, **grads}.items():
        base.close(t, want[k][0], base.rounded(*want[k], BF), k)


@pytest.mark.parametrize("rows,hidden", [(6, 4096), (450, 4096), (600, 259)])
def test_in_place(rows, hidden):
    Case(rows, hidden, res=F32).check_forward(in_place=True)


@pytest.mark.parametrize("fmt", [ct.E4M3, ct.E5M2])
@pytest.mark.parametrize("rows,hidden", [(1, 4096), (300, 2048), (600, 777), (2, 12288)])
def test_fp8(rows, hidden, fmt):
    """Codes of y within its bound, amax and scale_inv as the casts give them."""
    c = Case(rows, hidden)
    scale = 60.0 if fmt == ct.E4M3 else 9000.0
    out, w = c.check_forward(fp8=(fmt, scale))
    lo = ((w.y - w.y_err) * scale).float().numpy().ravel()
    hi = ((w.y + w.y_err) * scale).float().numpy().ravel()
    value = out["y"].view(ct.TORCH_FP8[fmt]).float().cpu().numpy().ravel()
    codes = [oracle.fp8_decode(oracle.fp8_encode(v, fmt), fmt) for v in (lo, hi)]
    slack = 2 * ref.F * np.abs(value)
    assert np.all(value >= codes[0] - slack) and np.all(value <= codes[1] + slack)
    most = w.y.abs().max().item()
    assert abs(out["amax"].item() - most) <= w.y_err.max().item() + 2 * ref.F * most
    assert f32_bits(out["scale_inv"].item()) == f32_bits(np.float32(1.0) / np.float32(scale))


@pytest.mark.parametrize("rows,hidden", [(3, 4096), (500, 4096), (500, 515)])
def test_what_is_dropped_is_zero_whatever_it_was(rows, hidden):
    c = Case(rows, hidden, p=0.4)
    gone = c.factor == 0
    c.u[gone] = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=BF).repeat(
        -(-int(gone.sum()) // 3))[:int(gone.sum())]
    c.want = ref.LayerNorm(c.u, c.res, c.weight, c.bias, EPS, 0.0, c.factor)
    out, _ = c.check_forward()
    assert torch.equal(out["res_out"].cpu()[gone], c.res[gone])


@pytest.mark.parametrize("rows,hidden", [(5, 4096), (500, 4096), (500, 515)])
def test_a_row_with_a_nan_spoils_no_other(rows, hidden):
    c = Case(rows, hidden, u=False, p=0.0)
    c.res[1, hidden // 2], c.res[3, 0] = float("nan"), float("inf")
    c.want = ref.LayerNorm(None, c.res, c.weight, c.bias, EPS, 0.0, c.factor)
    out = c.forward()
    y = out["y"].cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(out["rstd"][1]).item()
    assert torch.isnan(y[3]).all()
    others = [r for r in range(rows) if r not in (1, 3)]
    w = c.want.forward()
    base.close(y[others], w.y[others], base.rounded(w.y[others], w.y_err[others], BF), "y")


def test_noop_flag():
    for rows, hidden in ((4, 2048), (500, 2048), (700, 333)):
        c = Case(rows, hidden)
        flag = scalar(1.0)
        out = {k: torch.full((rows, hidden), 7.0, dtype=BF, device="cuda") for k in ("res_out", "y")}
        stats = {k: torch.full((rows,), 7.0, device="cuda") for k in ("mean", "rstd")}
        ct.layer_norm(c.u.cuda(), c.res.cuda(), **out, **stats, **c.kw, noop_flag=flag)
        g = {k: torch.full((rows, hidden), 7.0, dtype=BF, device="cuda") for k in ("dres", "du")}
        p = {k: torch.full((hidden,), 7.0, dtype=BF, device="cuda") for k in ("dweight", "dbias")}
        ws = torch.empty(ct.layer_norm_backward_workspace_size(rows, hidden), dtype=torch.uint8, device="cuda")
        ct.layer_norm_backward(c.dy.cuda(), c.dres_out.cuda(), c.res.cuda(), **stats, **g, **p, workspace=ws,
                               **c.kw, noop_flag=flag)
        for t in (*out.values(), *stats.values(), *g.values(), *p.values()):
            assert (t == 7.0).all()


def test_no_rows():
    H = 520
    empty = torch.empty(0, H, dtype=BF, device="cuda")
    stats = torch.empty(0, device="cuda")
    dw, db = (torch.full((H,), 7.0, dtype=BF, device="cuda") for _ in range(2))
    ct.layer_norm(empty, empty, empty.clone(), empty.clone(), mean=stats, rstd=stats.clone())
    ct.layer_norm_backward(empty, None, empty.clone(), stats, stats.clone(), empty.clone(), dweight=dw, dbias=db)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("rows,hidden", [(400, 2048), (2000, 515)])
def test_the_same_from_call_to_call(rows, hidden):
    c = Case(rows, hidden)
    one, two = c.backward()[0], c.backward()[0]
    for k in one:
        assert torch.equal(one[k], two[k])


# ---- dropout alone
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (5, 4096), (37, 777), (300, 1000), (2, 40001)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_dropout(rows, cols, dtype):
    x = data((rows, cols), dtype, rows + cols)
    for p in (0.1, 0.75):
        factor = ref.drop_factor(rows, cols, p, SEED, STEP, SITE)
        g = Guarded(rows * cols, dtype=dtype)
        out = g.t.view(rows, cols)
        ct.dropout(x.cuda(), out, p, state(), SITE)
        torch.cuda.synchronize()
        g.check()
        want = ref.dropped(x, factor)
        base.close(out, want, base.rounded(want, ref.F * want.abs(), dtype), "out")
        y = x.cuda()
        ct.dropout(y, y, p, state(), SITE)
        assert torch.equal(y, out)


@pytest.mark.parametrize("rows,cols", [(40, 1024), (40, 1021)])
def test_dropout_at_odd_addresses(rows, cols):
    x = data((rows, cols), BF, 5)
    want = ref.dropped(x, ref.drop_factor(rows, cols, 0.3, SEED, STEP, SITE))
    n = rows * cols
    for i in range(1, 8):
        y = torch.cat([x.reshape(-1)[:i], x.reshape(-1)]).cuda()[i:i + n].view(rows, cols)
        for j in (0, i, 8 - i):
            g = Guarded(n, dtype=BF, offset=j)
            ct.dropout(y, g.t.view(rows, cols), 0.3, state(), SITE)
            torch.cuda.synchronize()
            g.check()
            base.close(g.t.view(rows, cols), want, base.rounded(want, ref.F * want.abs(), BF), "out")


def test_dropout_of_nan_and_infinity():
    for cols in (512, 515):
        factor = ref.drop_factor(64, cols, 0.5, SEED, STEP, SITE)
        for v in (float("nan"), float("inf"), -float("inf")):
            x = torch.full((64, cols), v, dtype=BF, device="cuda")
            out = torch.empty_like(x)
            ct.dropout(x, out, 0.5, state(), SITE)
            out = out.cpu()
            assert not out[factor == 0].any()
            kept = out[factor > 0]
            assert torch.isnan(kept).all() if v != v else (kept == v).all()


def test_dropout_of_nothing_is_a_copy():
    x = data((9, 515), BF, 1).cuda()
    out = torch.empty_like(x)
    ct.dropout(x, out, 0.0, None)
    assert torch.equal(out, x)
    ct.dropout(x, out.zero_(), 1e-6, None)
    assert torch.equal(out, x)
    ct.dropout(x, out.zero_(), 0.5, state(), noop_flag=scalar(1.0))
    assert not out.any()


def test_the_junctions_dropout_is_dropout():
    for rows, hidden in ((6, 4096), (500, 4096), (500, 777)):
        u = data((rows, hidden), F32, 3).cuda()
        zero = torch.zeros_like(u)
        both = [torch.empty_like(u) for _ in range(3)]
        ct.layer_norm(u, zero, both[0], both[1], p=0.2, rng=state(), site=5)
        ct.dropout(u, both[2], 0.2, state(), 5)
        assert torch.equal(both[0], both[2])


def test_a_captured_graph_follows_the_step():
    rows, hidden = 300, 2048
    x, rng = data((rows, hidden), BF, 3).cuda(), state(7, 0)
    out = torch.empty_like(x)
    ct.dropout(x, out, 0.5, rng, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ct.dropout(x, out, 0.5, rng, 1)
        rng[1:].add_(1)
    for step in range(3):
        graph.replay()
        want = ref.dropped(x.cpu(), ref.drop_factor(rows, hidden, 0.5, 7, step, 1))
        base.close(out, want, base.rounded(want, ref.F * want.abs(), BF), "out")


def test_rows_past_32_bits():
    """Offsets beyond 2^31 elements: the last rows of a matrix of 4.4 GB."""
    rows, cols = 540000, 4096
    x = torch.ones(rows, cols, dtype=BF, device="cuda")
    ct.dropout(x, x, 0.25, state(), 2)
    group, row = np.meshgrid(np.arange(cols // 8), np.arange(rows - 2, rows))
    words = ref.philox((group, row, np.full_like(row, 2), np.full_like(row, STEP % 2 ** 32)),
                       (SEED % 2 ** 32, SEED >> 32))
    bits = np.stack([h for w in words for h in (w % 65536, w // 65536)], 2).reshape(2, -1)
    assert np.array_equal((x[-2:] > 0).cpu().numpy(), bits >= ref.cut_of(0.25))


@pytest.mark.parametrize("hidden", [4096, 4095])
def test_layer_norm_past_32_bits(hidden):
    """Offsets beyond 2^31 elements: the last rows are those of a small call."""
    rows, last = 540000, 3
    res = torch.empty(rows, hidden, dtype=BF, device="cuda").normal_()
    y, dres = torch.empty_like(res), torch.empty_like(res)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    w = data((hidden,), BF, 1, 0.2, 1.0).cuda()
    ct.layer_norm(None, res, None, y, weight=w, mean=mean, rstd=rstd)
    small = torch.empty(last, hidden, dtype=BF, device="cuda")
    ct.layer_norm(None, res[-last:].clone(), None, small, weight=w)
    one = torch.ones(last, hidden, dtype=torch.float64)
    n = ref.LayerNorm(None, res[-last:].cpu(), w.cpu(), None, EPS, 0.0, one).forward()
    for out in (y[-last:], small):
        base.close(out, n.y, base.rounded(n.y, n.y_err, BF), "y")
    ws = torch.empty(ct.layer_norm_backward_workspace_size(rows, hidden), dtype=torch.uint8, device="cuda")
    dbias = torch.empty(hidden, dtype=BF, device="cuda")
    y.zero_()
    y[-1] = 2.0                                  # the only gradient, of the last row
    ct.layer_norm_backward(y, None, res, mean, rstd, dres, dbias=dbias, workspace=ws, weight=w)
    want = n.backward(y[-last:].cpu(), None, res[-last:].cpu(), mean[-last:].cpu(), rstd[-last:].cpu())["dres"]
    base.close(dres[-last:], want[0], base.rounded(*want, BF), "dres")
    assert not dres[:-1].any() and (dbias == 2.0).all()


def test_two_host_threads():
    """Calls from two threads on streams of their own, a workspace each."""
    import threading
    c = [Case(700, 1032, seed=i) for i in range(2)]
    want = [x.backward()[0] for x in c]
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                got = c[i].backward()[0]
                stream.synchronize()
                wrong.extend(k for k in got if not torch.equal(got[k], want[i][k]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong
