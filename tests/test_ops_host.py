"""Host-side refusals of the expert-movement and block-norm entry points (no
GPU needed): status codes of the C ABI and errors of the binding.  The
pointers passed are never dereferenced."""
import ctypes

import pytest
import torch

import cast_transpose_gb300 as ct
from cast_transpose_gb300.norms import _Config

OK, NULL, SHAPE, ALIGN, FORMAT, ARG, ALIAS, WORKSPACE = range(8)
A, B, C, D, E, F, G, H, I, J, K, M = (0x100000000 * (i + 1) for i in range(12))


@pytest.fixture(scope="module")
def L():
    return ct.lib()


def test_sorted_rows(L):
    assert ct.moe_sorted_rows(8, 4, 64, 1) == 32
    assert ct.moe_sorted_rows(8, 4, 64, 16) == 512           # one slot in each of 32 experts
    assert ct.moe_sorted_rows(100, 2, 3, 16) == 256          # 200 + 3 * 15, rounded up
    assert ct.moe_sorted_rows(0, 4, 64, 16) == 0
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 65, 1, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0),
                (1, 1, 1, 1025), (2 ** 31, 1, 1, 1)):
        assert ct.moe_sorted_rows(*bad) == 0
    # enough for the worst routing, found by trying them all
    for n, experts, align in ((3, 2, 4), (5, 3, 4), (4, 6, 3)):
        def worst(left, kinds):
            if kinds == 0:
                return 0 if left == 0 else -10 ** 9
            return max(-(-c // align) * align + worst(left - c, kinds - 1) for c in range(left + 1))
        assert ct.moe_sorted_rows(n, 1, experts, align) >= worst(n, experts)


def sort(L, idx=A, ib=4, tokens=10, topk=2, experts=4, align=16, rows=128, row_of=B, src=C, off=D,
         counts=E, ws=F, wsb=1 << 30):
    return L.moe_sort(idx, ib, tokens, topk, experts, align, rows, row_of, src, off, counts, ws, wsb,
                      None, None)


def test_sort_rejects(L):
    assert sort(L, ib=2) == FORMAT
    for kw in (dict(topk=0), dict(topk=65), dict(experts=0), dict(experts=1025), dict(align=0),
               dict(align=1025)):
        assert sort(L, **kw) == ARG
    for kw in (dict(tokens=-1), dict(rows=-1), dict(tokens=2 ** 30), dict(rows=2 ** 31)):
        assert sort(L, **kw) == SHAPE
    for kw in (dict(idx=None), dict(row_of=None), dict(src=None), dict(off=None), dict(counts=None)):
        assert sort(L, **kw) == NULL
    assert sort(L, idx=A + 2) == ALIGN
    assert sort(L, idx=A + 4, ib=8) == ALIGN
    assert sort(L, src=C + 1) == ALIGN
    assert sort(L, row_of=A + 16) == ALIAS
    assert sort(L, counts=D) == ALIAS
    need = L.moe_sort_workspace_size(1 << 20, 8, 256)
    if need:
        assert sort(L, tokens=1 << 20, topk=8, experts=256, ws=None) == WORKSPACE
        assert sort(L, tokens=1 << 20, topk=8, experts=256, wsb=need - 1) == WORKSPACE
        assert sort(L, tokens=1 << 20, topk=8, experts=256, ws=F + 4) == ALIGN
    assert L.moe_sort_workspace_size(-1, 8, 256) == 0


def test_dispatch_rejects(L):
    def call(x=A, tokens=10, topk=2, hidden=64, dtype=0, row_of=B, src=C, rows=64, out=D):
        return L.moe_dispatch(x, tokens, topk, hidden, dtype, row_of, src, rows, out, None, None)
    assert call(dtype=3) == FORMAT
    assert call(topk=0) == ARG
    for kw in (dict(tokens=-1), dict(hidden=-1), dict(rows=-1), dict(hidden=1 << 21)):
        assert call(**kw) == SHAPE
    for kw in (dict(x=None), dict(row_of=None), dict(src=None), dict(out=None)):
        assert call(**kw) == NULL
    assert call(x=A + 1) == ALIGN
    assert call(dtype=2, x=A + 2) == ALIGN
    assert call(out=A + 64) == ALIAS
    assert call(out=C) == ALIAS
    assert call(hidden=0) == OK and call(rows=0) == OK


def test_combine_rejects(L):
    def call(ys=A, tokens=10, topk=2, hidden=64, dtype=0, row_of=B, w=C, rows=64, out=D):
        return L.moe_combine(ys, tokens, topk, hidden, dtype, row_of, w, rows, out, None, None)

    def dispatch_backward(dout=A, row_of=B, dx=D, tokens=10):
        return L.moe_dispatch_backward(dout, tokens, 2, 64, 0, row_of, 64, dx, None, None)
    for kw in (dict(ys=None), dict(row_of=None), dict(w=None), dict(out=None)):
        assert call(**kw) == NULL
    assert call(dtype=-1) == FORMAT
    assert call(w=C + 2) == ALIGN
    assert call(out=A) == ALIAS and call(out=C) == ALIAS
    assert call(tokens=0) == OK and call(hidden=0) == OK
    assert dispatch_backward(dout=None) == NULL and dispatch_backward(row_of=None) == NULL
    assert dispatch_backward(dx=A) == ALIAS
    assert dispatch_backward(tokens=0) == OK


def test_combine_backward_rejects(L):
    def call(dout=A, ys=B, row_of=C, src=D, w=E, dys=F, dw=G, tokens=10, rows=64, hidden=64):
        return L.moe_combine_backward(dout, ys, tokens, 2, hidden, 0, row_of, src, w, rows, dys, dw,
                                      None, None)
    assert call(dys=None, dw=None) == NULL
    assert call(ys=None) == NULL                 # needed for dweights
    assert call(src=None) == NULL and call(w=None) == NULL
    assert call(dout=None) == NULL
    assert call(dys=B) == ALIAS and call(dw=E) == ALIAS
    assert call(dw=G + 2) == ALIGN
    assert call(tokens=0, dys=None) == OK and call(tokens=0, rows=0) == OK


def test_fp8_dispatch_rejects(L):
    def call(x=A, topk=2, src=B, rows=64, w=None, s=C, a=D, si=E, q=F, qt=G, fmt=0, hidden=64):
        return L.fp8_moe_dispatch(x, 10, topk, hidden, src, rows, w, s, a, si, q, qt, fmt, None, None)
    assert call(fmt=2) == FORMAT
    assert call(topk=0) == ARG
    assert call(rows=-1) == SHAPE
    for kw in (dict(x=None), dict(src=None), dict(s=None), dict(a=None), dict(si=None), dict(q=None)):
        assert call(**kw) == NULL
    assert call(x=A + 1) == ALIGN and call(a=D + 2) == ALIGN
    assert call(q=A) == ALIAS and call(qt=F + 1) == ALIAS and call(si=C) == ALIAS
    assert call(w=E) == ALIAS
    assert call(rows=0) == OK and call(hidden=0) == OK


def config(rows=4, hidden=64, per_gate=4, w_post=A, w_pre=B, gate=None, eps=1e-6, dtype=0, res=0,
           param=0, flags=3):
    return _Config(rows, hidden, per_gate, w_post, w_pre, gate, eps, 1.0, 1.0, 0.0, dtype, res, param,
                   flags)


def test_block_norm_rejects(L):
    def call(u=C, r=D, ro=E, y=F, p1=G, p2=H, s=None, a=None, si=None, fmt=0, cfg=True, **kw):
        c = ctypes.byref(config(**kw)) if cfg else None
        return L.block_norm(c, u, r, ro, y, p1, p2, s, a, si, fmt, None, None)
    assert call(cfg=False) == NULL
    assert call(dtype=3) == FORMAT
    assert call(dtype=0, res=1) == FORMAT                       # fp16 residual of a bf16 block
    assert call(dtype=2, res=0, param=2) == FORMAT
    assert call(param=1) == FORMAT
    assert call(flags=4) == ARG and call(eps=-1.0) == ARG and call(eps=float("nan")) == ARG
    assert call(gate=M, per_gate=0) == ARG
    assert call(rows=-1) == SHAPE and call(hidden=32769) == SHAPE
    assert call(r=None) == NULL and call(ro=None) == NULL and call(y=None) == NULL
    assert call(u=None) == ARG                                  # res_out without u
    assert call(u=None, ro=None, flags=1) == ARG                # nothing to compute
    assert call(s=I) == NULL and call(s=I, a=J) == NULL         # FP8 without amax, scale_inv
    assert call(s=I, a=J, si=K, fmt=2) == FORMAT
    assert call(u=C + 1) == ALIGN and call(p1=G + 2) == ALIGN and call(w_post=A + 1) == ALIGN
    assert call(y=C) == ALIAS and call(ro=D + 16) == ALIAS and call(y=D) == ALIAS
    assert call(ro=D, y=D) == ALIAS                             # in place, but y over it
    assert call(p2=G) == ALIAS and call(y=A) == ALIAS
    assert call(s=I, a=I, si=K) == ALIAS
    assert call(rows=0) == OK and call(hidden=0) == OK


def test_block_norm_backward_rejects(L):
    need = L.block_norm_backward_workspace_size(4, 64)
    assert L.block_norm_backward_workspace_size(-1, 64) == 0

    def call(dy=C, dro=D, u=E, ro=F, p1=G, p2=H, du=I, dr=J, dw1=K, dw2=K + 4096, dg=None, ws=M,
             wsb=need, cfg=True, **kw):
        c = ctypes.byref(config(**kw)) if cfg else None
        return L.block_norm_backward(c, dy, dro, u, ro, p1, p2, du, dr, dw1, dw2, dg, ws, wsb, None,
                                     None)
    assert call(cfg=False) == NULL
    for kw in (dict(dy=None), dict(ro=None), dict(p1=None), dict(p2=None), dict(du=None),
               dict(dr=None)):
        assert call(**kw) == NULL
    assert call(dg=K + 8192) == ARG                             # dgate without a gate
    assert call(flags=2) == ARG and call(flags=1) == ARG        # dw of a norm left out
    assert call(u=None) == ARG
    assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE
    assert call(ws=M + 4) == ALIGN and call(dw1=K + 1) == ALIGN
    assert call(du=C) == ALIAS and call(dr=D) == ALIAS and call(dw2=K + 16) == ALIAS
    assert call(ws=I) == ALIAS
    assert call(hidden=0) == OK


def test_binding_rejects_before_any_launch():
    bf = torch.bfloat16
    x = torch.zeros(4, 8, dtype=bf)
    with pytest.raises(ValueError):
        ct.MoePlan(-1, 2, 4, device="cpu")
    with pytest.raises(ValueError):
        ct.MoePlan(4, 2, 2000, device="cpu")
    with pytest.raises(ValueError):
        ct.MoePlan(4, 2, 4, device="cpu", row_of=torch.zeros(8, dtype=torch.int32))
    with pytest.raises(ValueError):                     # CPU buffers
        ct.MoePlan(4, 2, 4, device="cpu")
    with pytest.raises(ValueError):
        ct.block_norm(x, x, x.clone(), x.clone())
    with pytest.raises(ValueError):                     # another shape
        ct.block_norm(x[:2], x, x.clone(), x.clone())
    with pytest.raises(TypeError):
        ct.block_norm(x.int(), x, x.clone(), x.clone())
    with pytest.raises(ValueError):
        ct.block_norm_backward(x, None, x, x, None, None, x, x.clone(), dw_pre=x[0])
