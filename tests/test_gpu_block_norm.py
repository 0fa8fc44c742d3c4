"""The norm / gate / residual / norm junction, forward and backward, against
its 64-bit form with worst-case bounds of the fp32 arithmetic."""
import numpy as np
import pytest
import torch

import cast_transpose_gb300 as ct
import ops_reference as ref
import oracle
from gpu_util import Guarded, f32_bits, scalar

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [(BF, BF, BF), (BF, F32, F32), (HF, HF, HF), (HF, F32, HF), (F32, F32, F32), (BF, BF, F32)]
EPS, ALPHA, BETA = 1e-6, 0.5, 1.25


def data(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


class Case:
    def __init__(self, rows, hidden, dtype=BF, res=BF, param=BF, per_gate=0, offset=0.0, u=True,
                 post=True, pre=True, weights=True, seed=0):
        """per_gate: 0 no gate, -1 one gate row for all, else rows per gate row."""
        self.rows, self.hidden, self.dtype, self.rdtype, self.pdtype = rows, hidden, dtype, res, param
        self.u = data((rows, hidden), dtype, seed + 1, 0.7) if u else None
        self.res = data((rows, hidden), res, seed + 2, 2.0)
        self.w_post = data((hidden,), param, seed + 3, 0.2, 1 - offset) if weights else None
        self.w_pre = data((hidden,), param, seed + 4, 0.2, 1 - offset) if weights else None
        groups = 1 if per_gate < 0 else -(-rows // per_gate) if per_gate else 0
        self.gate = data((groups, hidden), param, seed + 5, 0.8) if groups and u else None
        self.kw = dict(rows_per_gate=per_gate if per_gate > 0 else None, branch_scale=ALPHA,
                       residual_scale=BETA, weight_offset=offset, post_norm=post, pre_norm=pre)
        self.post, self.pre = post and u, pre
        self.dy, self.dres_out = data((rows, hidden), dtype, seed + 6, 0.3), data((rows, hidden), res, seed + 7, 0.3)
        self.want = ref.Norm(self.u, self.res, self.w_post, self.w_pre, self.gate,
                             per_gate if per_gate > 0 else None, EPS, ALPHA, BETA, offset, post, pre)

    def params(self):
        return {k: None if getattr(self, k) is None else getattr(self, k).cuda()
                for k in ("w_post", "w_pre", "gate")}

    def forward(self, in_place=False, fp8=None):
        n = self.rows * self.hidden
        shape = self.rows, self.hidden
        guards = {"rstd_post": Guarded(self.rows, dtype=F32) if self.post else None,
                  "rstd_pre": Guarded(self.rows, dtype=F32) if self.pre else None,
                  "res_out": Guarded(n, dtype=self.rdtype) if self.u is not None else None,
                  "y": Guarded(n, dtype=self.dtype if fp8 is None else torch.uint8) if self.pre else None}
        out = {k: None if g is None else g.t.view(shape) if k in ("res_out", "y") else g.t
               for k, g in guards.items()}
        res = self.res.cuda()
        if in_place:
            out["res_out"] = res
        more = {}
        if fp8 is not None:
            more = dict(scale=scalar(fp8[1]), amax=scalar(0.0), scale_inv=scalar(-1.0), fmt=fp8[0])
        ct.block_norm(None if self.u is None else self.u.cuda(), res, eps=EPS, **self.params(),
                      **out, **self.kw, **more)
        torch.cuda.synchronize()
        for g in guards.values():
            if g is not None:
                g.check()
        return {**out, **more}

    def check_forward(self, out):
        w = self.want.forward()
        if self.u is not None:
            ref.close(out["res_out"], w.out, ref.rounded(w.out, w.out_err, self.rdtype), "res_out")
        if self.post:
            err = w.rstd_post * (w.DEEP + 8 * ref.F)
            ref.close(out["rstd_post"], w.rstd_post, err, "rstd_post")
        if self.pre:
            ref.close(out["rstd_pre"], w.rstd_pre, w.rstd_pre * (w.rstd_err + 4 * ref.F), "rstd_pre")
            if out["y"].dtype != torch.uint8:
                ref.close(out["y"], w.y, ref.rounded(w.y, w.y_err, self.dtype), "y")
        return w

    def backward(self, grads=("dw_post", "dw_pre", "dgate"), dres_out=True):
        w = self.want.forward()
        kept = (w.out if self.u is not None else self.res.double()).to(self.rdtype)
        rp = None if not self.post else w.rstd_post.float()
        rr = None if not self.pre else w.rstd_pre.float()
        n = self.rows * self.hidden
        g = {"dres": Guarded(n, dtype=self.rdtype)}
        if self.u is not None:
            g["du"] = Guarded(n, dtype=self.dtype)
        shapes = {"dres": (self.rows, self.hidden), "du": (self.rows, self.hidden)}
        for k, t, on in (("dw_post", self.w_post, self.post), ("dw_pre", self.w_pre, self.pre),
                         ("dgate", self.gate, True)):
            if t is not None and on and k in grads:
                g[k], shapes[k] = Guarded(t.numel(), dtype=self.pdtype), tuple(t.shape)
        out = {k: v.t.view(shapes[k]) for k, v in g.items()}
        ws = Guarded(ct.block_norm_backward_workspace_size(self.rows, self.hidden))
        cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
        dres_out = self.dres_out if dres_out else None
        ct.block_norm_backward(self.dy.cuda() if self.pre else None, cuda(dres_out), cuda(self.u),
                               cuda(kept), cuda(rp), cuda(rr), workspace=ws.t, **self.params(),
                               **out, **self.kw)
        torch.cuda.synchronize()
        ws.check()
        for v in g.values():
            v.check()
        return out, w.backward(self.dy, dres_out, kept, rp, rr)

    def check_backward(self, **kw):
        got, want = self.backward(**kw)
        types = {"du": self.dtype, "dres": self.rdtype}
        for k, t in got.items():
            value, err = want[k]
            ref.close(t, value, ref.rounded(value, err, types.get(k, self.pdtype)), k)
        return got


SHAPES = [(1, 8), (1, 4096), (3, 1), (5, 777), (2, 1000), (64, 520), (37, 2048), (130, 4099), (9, 6144),
          (4, 8200), (21, 12288), (3, 12287), (2, 16384), (2, 24584), (3, 32768), (2, 32767)]


@pytest.mark.parametrize("dtype,res,param", TYPES)
@pytest.mark.parametrize("rows,hidden", SHAPES)
def test_forward_and_backward(rows, hidden, dtype, res, param):
    c = Case(rows, hidden, dtype, res, param, per_gate=max(1, rows // 3), offset=1.0, seed=rows)
    c.check_forward(c.forward())
    c.check_backward()


@pytest.mark.parametrize("rows,hidden", [(700, 264), (701, 131), (2500, 1024), (1300, 3008), (1217, 6144),
                                         (613, 12288)])
@pytest.mark.parametrize("per_gate", [0, -1, 1, 7, 128, 100000])
def test_many_rows_and_gates(rows, hidden, per_gate):
    """Gate rows of one row, of a few, of more than all: sums that end inside
    a block's rows, and at its edges."""
    c = Case(rows, hidden, BF, BF, F32, per_gate=per_gate, seed=3)
    c.check_forward(c.forward())
    c.check_backward()


@pytest.mark.parametrize("rows,hidden,dtype", [(400, 8192, BF), (500, 16384, BF), (200, 24580, BF),
                                               (170, 32768, BF), (170, 32767, HF), (200, 12288, F32),
                                               (90, 32768, F32), (300, 1, BF), (700, 5, HF), (900, 30, BF)])
def test_long_runs_of_long_and_short_rows(rows, hidden, dtype):
    """Rows over clusters of 2, 4 and 8 blocks, whole and odd, and rows of a
    few elements, in runs of more than one row."""
    c = Case(rows, hidden, dtype, dtype, F32, per_gate=rows // 2, seed=9)
    c.check_forward(c.forward())
    c.check_backward()


@pytest.mark.parametrize("post,pre,u,weights", [(True, False, True, True), (False, True, True, True),
                                                (False, False, True, True), (True, True, False, True),
                                                (True, True, True, False), (False, True, False, False)])
@pytest.mark.parametrize("hidden", [333, 1024, 12288])
def test_parts_left_out(post, pre, u, weights, hidden):
    c = Case(45, hidden, BF, F32, F32, per_gate=10 if weights else 0, post=post, pre=pre, u=u,
             weights=weights)
    c.check_forward(c.forward())
    c.check_backward()
    c.check_backward(grads=("dw_pre",), dres_out=False)
    c.check_backward(grads=("dgate",), dres_out=False)
    c.check_backward(grads=())


@pytest.mark.parametrize("hidden", [96, 777, 6144])
def test_in_place_residual_and_dropped_statistics(hidden):
    c = Case(33, hidden, BF, BF, BF, per_gate=-1)
    apart, in_place = c.forward(), c.forward(in_place=True)
    for k in ("res_out", "y", "rstd_pre"):
        assert torch.equal(apart[k], in_place[k])
    res, y = c.res.cuda(), torch.empty(33, hidden, dtype=BF, device="cuda")
    ct.block_norm(c.u.cuda(), res, res, y, eps=EPS, **c.params(), **c.kw)
    assert torch.equal(res, apart["res_out"]) and torch.equal(y, apart["y"])


@pytest.mark.parametrize("fmt", [ct.E4M3, ct.E5M2])
@pytest.mark.parametrize("rows,hidden", [(1, 4096), (4, 777), (300, 1024), (65, 12288)])
def test_fp8_output(rows, hidden, fmt):
    """The codes are those of some fp32 value within the bound of y; amax and
    scale_inv as in fp8_cast."""
    c = Case(rows, hidden, BF, BF, BF, per_gate=-1)
    scale = np.float32(ct.FP8_MAX[fmt] / 4.0)       # some values saturate
    out = c.forward(fp8=(fmt, float(scale)))
    w = c.check_forward(out)
    lo, hi = (w.y - w.y_err).numpy(), (w.y + w.y_err).numpy()

    def codes(v, grow):
        p = (v * float(scale)) * np.where((v > 0) == grow, 1 + 2.0 ** -22, 1 - 2.0 ** -22)
        return oracle.fp8_decode(oracle.fp8_encode(np.ascontiguousarray(p.astype(np.float32)).reshape(-1),
                                                   fmt), fmt).reshape(v.shape)

    got = oracle.fp8_decode(out["y"].cpu().numpy().reshape(-1), fmt).reshape(lo.shape)
    assert np.all(got >= codes(lo, False)) and np.all(got <= codes(hi, True))
    top = w.y.abs().max().item()
    assert abs(out["amax"].item() - top) <= w.y_err.max().item() + 2 * ref.F * top
    assert f32_bits(out["scale_inv"].item()) == f32_bits(np.float32(1.0) / scale)


def test_rows_of_zeros_infinities_and_nan():
    """A zero row gives zeros (eps > 0); Inf and NaN stay in their rows."""
    c = Case(12, 512, BF, F32, F32, per_gate=-1)
    c.u[1] = 0
    c.res[1] = 0
    clean = c.forward()
    assert not clean["y"][1].any() and not clean["res_out"][1].any()
    c.u[4, 7], c.res[8, 3] = float("nan"), float("inf")
    dirty = c.forward()
    rest = [i for i in range(12) if i not in (4, 8)]
    for k in ("y", "res_out"):
        assert torch.equal(dirty[k][rest], clean[k][rest])
    assert bool(torch.isnan(dirty["y"][4]).all())
    assert bool(torch.isinf(dirty["res_out"][8, 3])) and bool((dirty["y"][8, :3] == 0).all())
    assert bool(torch.isnan(dirty["y"][8, 3]))


def test_no_rows():
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    w = torch.ones(64, device="cuda")
    ct.block_norm(e(0, 64), e(0, 64), e(0, 64), e(0, 64), w_post=w, w_pre=w)
    dw = [torch.full((64,), 3.0, device="cuda") for _ in range(2)]
    size = ct.block_norm_backward_workspace_size(0, 64)
    ct.block_norm_backward(e(0, 64), None, e(0, 64), e(0, 64), e(0), e(0), e(0, 64), e(0, 64),
                           dw_post=dw[0], dw_pre=dw[1], w_post=w, w_pre=w,
                           workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
    assert not dw[0].any() and not dw[1].any()


@pytest.mark.parametrize("shift", [1, 4])
def test_unaligned_buffers(shift):
    c = Case(19, 256, BF, BF, BF, per_gate=8)

    def off(t):
        b = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        b[shift:] = t.reshape(-1).cuda()
        return b[shift:].view(t.shape)

    p = {k: off(v) for k, v in c.params().items()}
    out = {k: off(torch.empty(19, 256, dtype=BF)) for k in ("res_out", "y")}
    rstd = {k: torch.empty(19, device="cuda") for k in ("rstd_post", "rstd_pre")}
    ct.block_norm(off(c.u), off(c.res), eps=EPS, **p, **out, **rstd, **c.kw)
    c.check_forward({**out, **rstd})
    w = c.want
    kept = w.out.to(BF)
    rp, rr = w.rstd_post.float(), w.rstd_pre.float()
    got = {"du": off(torch.empty_like(c.u)), "dres": off(torch.empty_like(c.res)),
           **{"d" + k: off(torch.empty_like(v)) for k, v in p.items()}}
    ws = torch.empty(ct.block_norm_backward_workspace_size(19, 256), dtype=torch.uint8, device="cuda")
    ct.block_norm_backward(off(c.dy), off(c.dres_out), off(c.u), off(kept), rp.cuda(), rr.cuda(),
                           workspace=ws, **p, **got, **c.kw)
    for k, (value, err) in w.backward(c.dy, c.dres_out, kept, rp, rr).items():
        ref.close(got[k], value, ref.rounded(value, err, BF), k)


def test_gradients_against_differences():
    """<gradient, direction> of fp32 inputs against central differences of the
    64-bit forward pass: their error is O(h^2) = 1e-8 and 1e-16 / h."""
    c = Case(24, 160, F32, F32, F32, per_gate=7, offset=1.0)
    got, _ = c.backward()
    h = 1e-4

    def loss(**moved):
        t = {k: moved.get(k, getattr(c, k)) for k in ("u", "res", "w_post", "w_pre", "gate")}
        n = ref.Norm(t["u"], t["res"], t["w_post"], t["w_pre"], t["gate"], 7, EPS, ALPHA, BETA, 1.0)
        n.forward()
        return (n.y * c.dy.double()).sum() + (n.out * c.dres_out.double()).sum()

    names = {"u": "du", "res": "dres", "w_post": "dw_post", "w_pre": "dw_pre", "gate": "dgate"}
    for seed, (k, d) in enumerate(names.items()):
        base = getattr(c, k).double()
        way = data(base.shape, torch.float64, 100 + seed)
        diff = (loss(**{k: base + h * way}) - loss(**{k: base - h * way})) / (2 * h)
        slope = (got[d].double().cpu() * way).sum()
        size = got[d].double().norm().item() * way.norm().item()
        assert abs(diff - slope) <= 1e-5 * size, (k, diff, slope)


def test_noop_flag_same_results_and_graph():
    c = Case(500, 1024, BF, F32, F32, per_gate=60)
    cu = {k: getattr(c, k).cuda() for k in ("u", "res", "dy", "dres_out")}
    p, flag = c.params(), scalar(0.0)
    ws = torch.empty(ct.block_norm_backward_workspace_size(500, 1024), dtype=torch.uint8, device="cuda")
    out = {"res_out": torch.empty_like(cu["res"]), "y": torch.empty_like(cu["u"]),
           "rstd_post": torch.empty(500, device="cuda"), "rstd_pre": torch.empty(500, device="cuda")}
    grad = {"du": torch.empty_like(cu["u"]), "dres": torch.empty_like(cu["res"]),
            **{"d" + k: torch.empty_like(v) for k, v in p.items()}}
    bufs = list(out.values()) + list(grad.values())

    def step(noop):
        ct.block_norm(cu["u"], cu["res"], eps=EPS, **p, **out, **c.kw, noop_flag=noop)
        ct.block_norm_backward(cu["dy"], cu["dres_out"], cu["u"], out["res_out"], out["rstd_post"],
                               out["rstd_pre"], workspace=ws, **p, **grad, **c.kw, noop_flag=noop)

    step(None)
    want = [b.clone() for b in bufs]
    for b in bufs:
        b.fill_(9)
    flag.fill_(1.0)
    step(flag)
    assert all(bool((b == 9).all()) for b in bufs)
    flag.fill_(0.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(flag)
    side.synchronize()
    assert all(torch.equal(b, v) for b, v in zip(bufs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(flag)
    for _ in range(2):
        for b in bufs:
            b.fill_(9)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b, v) for b, v in zip(bufs, want))


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows come out as they do alone."""
    rows, hidden = 180_000, 12288
    assert rows * hidden > 2 ** 31
    c = Case(64, hidden, BF, BF, BF, per_gate=0, seed=5)
    u = torch.zeros(rows, hidden, dtype=BF, device="cuda")
    res = torch.zeros_like(u)
    u[-64:], res[-64:] = c.u.cuda(), c.res.cuda()
    out, y = torch.empty_like(u), torch.empty_like(u)
    rp, rr = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ct.block_norm(u, res, out, y, eps=EPS, rstd_post=rp, rstd_pre=rr, **c.params(), **c.kw)
    alone = c.forward()
    assert torch.equal(out[-64:], alone["res_out"]) and torch.equal(y[-64:], alone["y"])
    assert not out[:-64].any() and not y[:-64].any()
    dy = torch.zeros_like(u)
    dy[-64:] = c.dy.cuda()
    du, dres = torch.empty_like(u), res
    dw = [torch.empty(hidden, dtype=BF, device="cuda") for _ in range(2)]
    ws = torch.empty(ct.block_norm_backward_workspace_size(rows, hidden), dtype=torch.uint8, device="cuda")
    ct.block_norm_backward(dy, None, u, out, rp, rr, du, dres, dw_post=dw[0], dw_pre=dw[1],
                           workspace=ws, **c.params(), **c.kw)
    want = c.want.backward(c.dy, None, alone["res_out"].cpu(), rp[-64:].cpu(), rr[-64:].cpu())
    for t, k in ((du[-64:], "du"), (dres[-64:], "dres"), (dw[0], "dw_post"), (dw[1], "dw_pre")):
        ref.close(t, want[k][0], ref.rounded(want[k][0], want[k][1], BF), k)
    assert not du[:-64].any()


def test_no_wait_gave_up():
    """The kernels' bounded waits set a bit of the diagnostic word when they run out."""
    c = Case(2000, 6144, BF, BF, BF, per_gate=300)
    c.check_backward()
    torch.cuda.synchronize()
    assert ct.device_error() & 1 == 0
