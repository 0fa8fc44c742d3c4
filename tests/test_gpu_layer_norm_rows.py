"""The layer norms' launches of many rows: each form of their kernels, with rows
taken from the launch rule (ct_layer_norm_kernel), so that every block has rows to
spare, against the 64-bit forms.  What the rule gives is asserted."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import cast_transpose_gb300 as ct
import ops_reference as base
import oracle
import step_reference as ref
from cast_transpose_gb300.norms import _pack_layer_config
from gpu_util import f32_bits, scalar
from test_gpu_layer_norm import BF, EPS, F32, HF, Case

pytestmark = pytest.mark.gpu

CODE = {BF: 0, HF: 1, F32: 2}
ALL_TYPES = [(t, r, p) for t in (BF, HF, F32) for r in ((t, F32) if t != F32 else (F32,))
             for p in ((t, F32) if t != F32 else (F32,))]
FIELDS = ("blocks", "vectors", "stages", "shifted", "warp_per_row", "once")
JOIN_WAYS = 32                 # warps of the join, at most, each adding every so many-th part


def plan(rows, hidden, dtype=BF, res=BF, backward=False, given=True):
    out = (ctypes.c_int * 6)()
    config = _pack_layer_config(rows, hidden, 0, 0, 0, 0.0, 0.0, 0.0, 0, CODE[dtype], CODE[res], CODE[dtype])
    assert ct.lib().ct_layer_norm_kernel(config, int(backward), int(given), out) == 0
    return dict(zip(FIELDS, out))


def many_rows(hidden, dtype=BF, res=BF, u=True, down=True, times=5, more=3):
    """Rows for `times` and some of every block, forward and, where it has such a
    launch, backward."""
    blocks = max(plan(1 << 20, hidden, dtype, res, False, u)["blocks"],
                 plan(1 << 20, hidden, dtype, res, True, down)["blocks"])
    assert blocks > 0
    return times * blocks + more


class Rows(Case):
    """A case whose column sums are bounded by what the kernels add up: a block's own
    rows one after the other, then the blocks' sums."""

    def plans(self, down=True):
        types = self.rows, self.hidden, self.dtype, self.rdtype
        return plan(*types, False, self.u is not None), plan(*types, True, down)

    def check_backward(self, which=("du", "dweight", "dbias"), dres_out=True):
        got, want = self.backward(which=which, dres_out=dres_out)
        blocks = self.plans(dres_out)[1]["blocks"]
        deep = self.rows + 6
        if blocks:
            deep = -(-self.rows // blocks) + -(-blocks // 8) + JOIN_WAYS + 6
        types = {"du": self.dtype, "dres": self.rdtype}
        for k, t in got.items():
            value, err = want[k]
            if k in ("dweight", "dbias"):
                err = err * min(1.0, deep / (self.rows + 2))
            base.close(t, value, base.rounded(value, err, types.get(k, self.pdtype)), k)
        return got


def has(got, **want):
    assert {k: got[k] for k in want} == want, got
    assert got["blocks"] > 0


ONE = dict(warp_per_row=1, shifted=0, vectors=2)
WHOLE = dict(warp_per_row=0, shifted=0, vectors=2)
SHIFT = dict(warp_per_row=0, shifted=1, vectors=2, once=0)
FOUR = dict(warp_per_row=0, shifted=0, vectors=4)
ROW = dict(blocks=0)
# hidden, the forward kernel, the backward one
FORMS = [(8, ONE, ONE), (264, ONE, ONE), (512, ONE, ONE),
         (520, WHOLE, dict(ONE, vectors=4)), (1024, WHOLE, dict(ONE, vectors=4)),
         (1032, WHOLE, dict(FOUR, once=1, stages=3)), (2048, WHOLE, dict(FOUR, once=1, stages=3)),
         (4096, dict(WHOLE, stages=4), dict(FOUR, once=0, stages=3)), (6144, WHOLE, dict(FOUR, once=0)),
         (8192, WHOLE, dict(FOUR, once=0, stages=4)), (12288, WHOLE, dict(FOUR, once=0)),
         (1, SHIFT, SHIFT), (3, SHIFT, SHIFT), (7, SHIFT, SHIFT), (333, dict(SHIFT, stages=3), SHIFT),
         (515, SHIFT, SHIFT), (777, SHIFT, SHIFT), (1001, SHIFT, SHIFT), (1025, SHIFT, SHIFT), (2049, SHIFT, SHIFT),
         (4099, SHIFT, SHIFT), (6143, SHIFT, SHIFT), (8185, SHIFT, SHIFT), (9001, SHIFT, ROW)]


@pytest.mark.parametrize("p", [0.1, 0.0])
@pytest.mark.parametrize("hidden,forward,backward", FORMS, ids=[str(f[0]) for f in FORMS])
def test_forms(hidden, forward, backward, p):
    # enough that the backward pass of short shifted rows takes its longer form
    c = Rows(many_rows(hidden, times=7 if forward["shifted"] and hidden < 1024 else 5), hidden, p=p)
    got = c.plans()
    has(got[0], **forward)
    if backward is ROW:
        assert got[1]["blocks"] == 0
    else:
        has(got[1], **backward)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("hidden", [3, 333, 515, 777, 1001, 1017])
@pytest.mark.parametrize("types", [(BF, BF, BF), (HF, F32, F32), (F32, F32, F32)])
def test_shifted_rows_few_to_a_block(hidden, types):
    """The backward pass with one vector per thread."""
    rows = next(r for r in range(152, 20000) if plan(r, hidden, *types[:2], True)["vectors"] == 1)
    for times in (1, 4):
        c = Rows(times * rows + 5, hidden, *types)
        has(c.plans()[1], vectors=1, shifted=1, once=0)
        c.check_backward()
        c.check_backward(dres_out=False, which=("dweight",))


# hidden, u's and res's types, stages of the backward ring beside dres_out's one place
ONCE = [(1032, BF, BF, 3), (2040, HF, HF, 3), (2048, BF, F32, 2), (6144, HF, F32, 2), (5120, BF, F32, 3),
        (8192, BF, F32, 4), (4096, F32, F32, 2), (8192, F32, F32, 3), (12288, BF, F32, 2)]


@pytest.mark.parametrize("hidden,dtype,res,stages", ONCE)
@pytest.mark.parametrize("p", [0.1, 0.0])
def test_dres_out_in_one_place(hidden, dtype, res, stages, p):
    for times, more in ((1, 1), (7, 2)):
        c = Rows(many_rows(hidden, dtype, res, times=times, more=more), hidden, dtype, res, dtype, p=p)
        has(c.plans()[1], once=1, stages=stages, vectors=4)
        c.check_backward()
    c.check_backward(which=())
    assert c.plans(down=False)[1]["once"] == 0
    c.check_backward(dres_out=False)


@pytest.mark.parametrize("hidden", [264, 1024, 2048, 333, 777])
@pytest.mark.parametrize("types", ALL_TYPES)
def test_types(hidden, types):
    """All nine of them, in both passes' kernels."""
    c = Rows(many_rows(hidden, *types[:2], times=2), hidden, *types, p=0.3, offset=1.0)
    for got in c.plans():
        has(got, shifted=int(hidden % 8 != 0))
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("more", [1, 2, 9])
@pytest.mark.parametrize("hidden", [264, 1024, 4096, 7, 777, 4099])
def test_blocks_with_a_row_more(hidden, more):
    for backward in (False, True):
        rows = plan(1 << 20, hidden, backward=backward)["blocks"] + more
        c = Rows(rows, hidden)
        assert c.plans()[backward]["blocks"] > 0 or hidden == 1024 and backward
        c.check_backward() if backward else c.check_forward()


@pytest.mark.parametrize("hidden", [264, 1024, 2048, 515])
@pytest.mark.parametrize("kw", [dict(u=False, p=0.0), dict(weight=False), dict(bias=False),
                                dict(weight=False, bias=False, p=0.0)])
def test_without(hidden, kw):
    c = Rows(many_rows(hidden, u=kw.get("u", True), times=4), hidden, **kw)
    for down in (False, True):
        for got in c.plans(down):
            has(got)
    c.check_forward()
    c.check_backward(dres_out=False)
    c.check_backward(which=())
    c.check_backward(which=("dweight",))
    c.check_backward(which=("dbias", "du"), dres_out=False)


@pytest.mark.parametrize("hidden", [264, 512, 1024, 4096, 12288, 7, 777, 4099])
def test_a_mean_far_from_zero(hidden):
    """A row's mean a thousand times its deviation: nothing may cancel."""
    c = Rows(many_rows(hidden, F32, F32, u=False, times=2), hidden, F32, F32, F32, u=False, p=0.0, mean=2000.0)
    has(c.plans()[0])
    out, w = c.check_forward()
    assert torch.allclose(out["rstd"].cpu().double(), w.rstd, rtol=1e-3)
    c.check_backward()


@pytest.mark.parametrize("hidden", [264, 1024, 777])
def test_constant_rows(hidden):
    """Variance 0: rstd is 1 / sqrt(eps) and y the bias."""
    c = Rows(many_rows(hidden, F32, F32, u=False, times=2), hidden, F32, F32, F32, u=False, p=0.0)
    has(c.plans()[0])
    c.res.fill_(3.0)
    out = c.forward()
    assert (out["mean"] == 3.0).all()
    assert torch.allclose(out["rstd"].cpu(), torch.full((c.rows,), EPS ** -0.5), rtol=1e-6)
    assert torch.equal(out["y"].cpu(), c.bias.expand(c.rows, -1))


@pytest.mark.parametrize("hidden", [264, 1024, 6144, 777, 4099])
def test_a_variance_is_never_below_zero(hidden):
    """Without eps, rows of equal or nearly equal values: 1 / sqrt of a number."""
    rows = many_rows(hidden, F32, F32, u=False, times=2)
    has(plan(rows, hidden, F32, F32, given=False))
    values = torch.tensor([0.1, 3.0, 2000.3, -7.77e-12, 1.3e15])[torch.arange(rows) % 5]
    res = values[:, None].expand(-1, hidden).contiguous().cuda()
    last = torch.arange(hidden, device="cuda") % 97 == 0
    res[rows // 2:] = torch.where(last, torch.nextafter(res, res * 2), res)[rows // 2:]
    y, rstd = torch.empty_like(res), torch.empty(rows, device="cuda")
    ct.layer_norm(None, res, None, y, eps=0.0, rstd=rstd)
    assert (rstd > 0).all()


@pytest.mark.parametrize("hidden", [264, 4096, 259])
def test_in_place(hidden):
    c = Rows(many_rows(hidden, res=F32), hidden, res=F32)
    has(c.plans()[0])
    c.check_forward(in_place=True)


def check_fp8(c, fmt):
    """Codes of y within its bound, amax and scale_inv as the casts give them."""
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


@pytest.mark.parametrize("fmt", [ct.E4M3, ct.E5M2])
@pytest.mark.parametrize("hidden", [264, 2048, 6144, 7, 333, 777])
def test_fp8(hidden, fmt):
    c = Rows(many_rows(hidden, times=2), hidden)
    has(c.plans()[0])
    check_fp8(c, fmt)


@pytest.mark.parametrize("types", [(BF, BF, BF), (BF, F32, BF), (HF, F32, HF), (F32, F32, F32), (BF, BF, F32)])
@pytest.mark.parametrize("rows,hidden", [(3, 2048), (0, 264), (0, 2048), (0, 777)])
def test_fp8_without_a_branch(rows, hidden, types):
    """The first junction of a model; rows 0: a launch of many."""
    launch = many_rows(hidden, *types[:2], u=False, times=2)
    c = Rows(rows or launch, hidden, *types, u=False, p=0.0)
    assert (c.plans()[0]["blocks"] > 0) == (rows == 0)
    check_fp8(c, ct.E4M3)


@pytest.mark.parametrize("hidden", [264, 2048, 777])
def test_amax_of_one_large_value(hidden):
    """In the last row, its last column: by the bits of the largest, a NaN above all."""
    rows = many_rows(hidden, u=False, times=2)
    res = torch.zeros(rows, hidden, dtype=BF, device="cuda")
    res[-1, -1] = 1.0
    y, amax, inv = torch.empty(rows, hidden, dtype=torch.uint8, device="cuda"), scalar(0.5), scalar(-1.0)
    ct.layer_norm(None, res, None, y, scale=scalar(1.0), amax=amax, scale_inv=inv)
    one = torch.ones(1, hidden, dtype=torch.float64)
    w = ref.LayerNorm(None, res[-1:].cpu(), None, None, EPS, 0.0, one).forward()
    assert abs(amax.item() - w.y.max().item()) <= w.y_err.max().item()
    res[-1, 0] = float("nan")
    ct.layer_norm(None, res, None, y, scale=scalar(1.0), amax=amax, scale_inv=inv)
    assert torch.isnan(amax).item() and (y[-1] == 0x7F).all() and not y[:-1].any()


@pytest.mark.parametrize("hidden", [264, 4096, 515])
def test_what_is_dropped_is_zero_whatever_it_was(hidden):
    c = Rows(many_rows(hidden, times=2), hidden, p=0.4)
    has(c.plans()[0])
    gone = c.factor == 0
    c.u[gone] = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=BF).repeat(
        -(-int(gone.sum()) // 3))[:int(gone.sum())]
    c.want = ref.LayerNorm(c.u, c.res, c.weight, c.bias, EPS, 0.0, c.factor)
    out, _ = c.check_forward()
    assert torch.equal(out["res_out"].cpu()[gone], c.res[gone])


@pytest.mark.parametrize("hidden", [264, 1024, 4096, 515])
def test_a_row_with_a_nan_spoils_no_other(hidden):
    c = Rows(many_rows(hidden, u=False, times=2), hidden, u=False, p=0.0)
    bad = [1, 3, c.rows - 1]
    c.res[1, hidden // 2], c.res[3, 0], c.res[-1, -1] = float("nan"), float("inf"), float("nan")
    c.want = ref.LayerNorm(None, c.res, c.weight, c.bias, EPS, 0.0, c.factor)
    y = c.forward()["y"].cpu()
    assert torch.isnan(y[bad]).all()
    others = torch.ones(c.rows, dtype=torch.bool)
    others[bad] = False
    w = c.want.forward()
    base.close(y[others], w.y[others], base.rounded(w.y[others], w.y_err[others], BF), "y")
    # and back: dres alone, the column sums have them all
    c = Rows(c.rows, hidden)
    c.dy[bad] = float("nan")
    got, want = c.backward(which=("du",))
    for k in ("dres", "du"):
        base.close(got[k][others.cuda()], want[k][0][others], base.rounded(*(v[others] for v in want[k]), BF), k)
    assert torch.isnan(got["dres"][bad]).all()


@pytest.mark.parametrize("hidden", [264, 1024, 2048, 333, 777])
def test_noop_flag(hidden):
    rows = many_rows(hidden, times=1)
    c = Rows(rows, hidden)
    out = {k: torch.full((rows, hidden), 7.0, dtype=BF, device="cuda") for k in ("res_out", "y")}
    stats = {k: torch.full((rows,), 7.0, device="cuda") for k in ("mean", "rstd")}
    ct.layer_norm(c.u.cuda(), c.res.cuda(), **out, **stats, **c.kw, noop_flag=scalar(1.0))
    codes, amax, inv = torch.full((rows, hidden), 7, dtype=torch.uint8, device="cuda"), scalar(7.0), scalar(7.0)
    ct.layer_norm(c.u.cuda(), c.res.cuda(), out["res_out"], codes, scale=scalar(1.0), amax=amax, scale_inv=inv, **c.kw,
                  noop_flag=scalar(1.0))
    g = {k: torch.full((rows, hidden), 7.0, dtype=BF, device="cuda") for k in ("dres", "du")}
    p = {k: torch.full((hidden,), 7.0, dtype=BF, device="cuda") for k in ("dweight", "dbias")}
    ws = torch.empty(ct.layer_norm_backward_workspace_size(rows, hidden), dtype=torch.uint8, device="cuda")
    ct.layer_norm_backward(c.dy.cuda(), c.dres_out.cuda(), c.res.cuda(), **stats, **g, **p, workspace=ws, **c.kw,
                           noop_flag=scalar(1.0))
    for t in (*out.values(), *stats.values(), *g.values(), *p.values(), codes, amax, inv):
        assert (t == 7.0).all()


@pytest.mark.parametrize("hidden", [1032, 777])
def test_two_host_threads(hidden):
    """Calls from two threads on streams of their own, a workspace each."""
    c = [Rows(many_rows(hidden, times=2), hidden, seed=i) for i in range(2)]
    want = [(x.forward(), x.backward()[0]) for x in c]
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(3):
                for got, of in zip((c[i].forward(), c[i].backward()[0]), want[i]):
                    stream.synchronize()
                    wrong.extend(k for k in got if not torch.equal(got[k], of[k]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong
