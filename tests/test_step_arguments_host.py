"""Arguments that a call says it does not use are not looked at (no GPU needed).
The C calls here end in another refusal, so that nothing is launched; the
pointers passed are never dereferenced."""
import ctypes
import struct

import pytest
import torch

import cast_transpose_gb300 as ct
from test_step_host import A, ALIAS, ALIGN, ARG, B, FORMAT, NULL, SHAPE, config, fake, L, router  # noqa: F401

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
FIELDS = ("rows", "hidden", "weight", "bias", "rng", "eps", "weight_offset", "p", "site", "dtype",
          "res_dtype", "param_dtype")


def unpacked(call):
    return dict(zip(FIELDS, struct.unpack("@2q3P3fI3i4x", call[1][0])))


@pytest.mark.parametrize("p", [1.0, -0.5, float("nan"), 0.1])
def test_the_dropout_of_a_norm_without_a_branch(L, p):  # noqa: F811
    cfg, _ = config(p=p, rng=None)
    assert L.layer_norm(cfg, None, A, None, None, None, None, None, None, None, 0, None, None) == NULL
    assert L.layer_norm_backward(cfg, None, None, A, B, B + 4096, A + 4096, None, None, None, None, 0, None,
                                 None) == NULL


def test_the_dropout_of_a_norm_with_a_branch_is_checked(L):  # noqa: F811
    cfg, _ = config(p=1.0)
    assert L.layer_norm(cfg, A, B, B, None, None, None, None, None, None, 0, None, None) == ARG
    assert L.layer_norm_backward(cfg, None, None, A, B, B + 4096, A + 4096, A + 8192, None, None, None, 0,
                                 None, None) == ARG


def test_the_bindings_dropout_without_a_branch(fake):  # noqa: F811
    x, stats = torch.zeros(4, 8, dtype=BF), torch.zeros(4)
    for more in (dict(p=0.1), dict(p=0.1, site=-1), dict(p=2.0)):
        ct.layer_norm(None, x, None, x, **more)
        ct.layer_norm_backward(x, x, x, stats, stats, x, **more)
        with pytest.raises(ValueError, match="rng|site"):
            ct.layer_norm(x, x, x, x, **more)
        with pytest.raises(ValueError, match="rng|site"):
            ct.layer_norm_backward(x, x, x, stats, stats, x, x.clone(), **more)
    assert len(fake.calls) == 6
    for call in fake.calls:
        got = unpacked(call)
        assert got["p"] == 0.0 and got["rng"] == 0


@pytest.mark.parametrize("eps", [-1.0, float("nan")])
def test_the_backward_pass_has_no_eps(L, eps):  # noqa: F811
    cfg, _ = config(eps=eps)
    assert L.layer_norm_backward(cfg, None, None, A, B, B + 4096, A + 4096, None, None, None, None, 0, None,
                                 None) == NULL
    assert L.layer_norm(cfg, None, A, None, None, None, None, None, None, None, 0, None, None) == ARG


def test_the_generator_of_a_dropout_of_nothing(L):  # noqa: F811
    def call(p, rng, out=A + 2):
        return L.dropout(A, 10, 64, 0, p, rng, 0, out, None, None)
    assert call(0.0, B + 4) == ALIAS and call(1e-6, B + 4) == ALIAS and call(0.0, None) == ALIAS
    assert call(0.1, B + 4) == ALIGN and call(0.1, None) == NULL


@pytest.mark.parametrize("res,param,want", [(F32, BF, (0, 2, 0)), (F32, HF, (1, 2, 1)), (F32, F32, (2, 2, 2)),
                                            (F32, None, (2, 2, 2)), (BF, F32, (0, 0, 2)), (BF, BF, (0, 0, 0)),
                                            (HF, None, (1, 1, 1))])
def test_types_of_an_fp8_norm_without_a_branch(fake, res, param, want):  # noqa: F811
    """Neither u nor y has the data's type: that of 16-bit parameters, else res's."""
    x, y, one = torch.zeros(4, 8, dtype=res), torch.zeros(4, 8, dtype=torch.uint8), torch.ones(1)
    p = None if param is None else torch.zeros(8, dtype=param)
    for kw in (dict(weight=p), dict(bias=p)):
        ct.layer_norm(None, x, None, y, scale=one, amax=one.clone(), scale_inv=one.clone(), **kw)
        got = unpacked(fake.calls.pop())
        assert (got["dtype"], got["res_dtype"], got["param_dtype"]) == want


def test_which_kernel(L):  # noqa: F811
    def kernel(backward=0, given=1, **kw):
        out = (ctypes.c_int * 6)()
        return L.ct_layer_norm_kernel(config(**kw)[0], backward, given, out), list(out)
    assert kernel(rows=4, hidden=4096) == (0, [0] * 6) == kernel(rows=0) == kernel(hidden=0)
    for backward in (0, 1):
        assert kernel(backward, rows=10 ** 6, hidden=32768) == (0, [0] * 6)
        status, (blocks, vectors, stages, shifted, one, once) = kernel(backward, rows=10 ** 6, hidden=777)
        assert status == 0 and blocks > 0 and blocks % 8 == 0 and (vectors, shifted, one, once) == (2, 1, 0, 0)
    assert kernel(rows=10 ** 6, hidden=264)[1][4] == 1
    assert kernel(1, rows=10 ** 6, hidden=2048)[1][5] == 1 and kernel(1, 0, rows=10 ** 6, hidden=2048)[1][5] == 0
    assert kernel(dtype=3)[0] == FORMAT and kernel(rows=-1)[0] == SHAPE
    assert L.ct_layer_norm_kernel(config()[0], 0, 0, None) == NULL
    assert L.ct_layer_norm_kernel(None, 0, 0, (ctypes.c_int * 6)()) == NULL


def test_the_flag_is_a_buffer_like_any_other(L):  # noqa: F811
    """Off its four bytes it is refused, and so is an output over it, which some
    blocks would write before others have read it."""
    far = [0x100000000000 * (i + 1) for i in range(13)]
    norm, _ = config(p=0.0)
    choice, _ = router()
    calls = {
        "dropout": (lambda out, n: L.dropout(far[0], 10, 64, 2, 0.0, None, 0, out, n, None)),
        "layer_norm": (lambda out, n: L.layer_norm(norm, far[0], far[1], far[2], out, None, None, None, None, None, 0,
                                                   n, None)),
        "layer_norm_backward": (lambda out, n: L.layer_norm_backward(
            norm, far[0], None, far[2], far[3], far[4], out, None, None, None, None, 0, n, None)),
        "moe_router": (lambda out, n: L.moe_router(choice, far[0], None, far[1], out, far[3], None, None, 0, n, None)),
        "moe_router_backward": (lambda out, n: L.moe_router_backward(choice, far[0], None, far[1], far[2], far[3], None,
                                                                     out, n, None)),
        "embedding": (lambda out, n: L.embedding(far[0], 8, 10, far[1], 100, 64, 2, 1.0, out, n, None)),
        "embedding_backward": (lambda out, n: L.embedding_backward(far[0], 8, 10, far[1], 100, 64, 2, 1.0, out, 2, 0,
                                                                   None, 0, n, None)),
    }
    for name, call in calls.items():
        assert call(far[5] + 1, far[6] + 2) == ALIGN, name
        assert call(far[0] + 16, far[6] + 2) == ALIGN, name     # which comes before the overlap
        assert call(far[0] + 16, None) == ALIAS, name
        assert call(far[5], far[5]) == ALIAS, name
        assert call(far[5], far[5] + 16) == ALIAS, name
