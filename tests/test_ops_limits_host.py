"""Further host-side checks of the expert-movement and block-norm operators (no
GPU needed): limits, refusals and their messages, the plan's attributes."""
import os
import shutil
import subprocess

import pytest
import torch

import cast_transpose_gb300 as ct

OK, NULL, SHAPE, ALIGN, FORMAT, ARG, ALIAS, WORKSPACE = range(8)
A, B, C, D, E, F, G = (0x100000000 * (i + 1) for i in range(7))


@pytest.fixture(scope="module")
def L():
    return ct.lib()


def test_norm_wait_selftest_rejects(L):
    for blocks, thread, limit in ((0, 0, 10), (3, 0, 10), (16, 0, 10), (2, -1, 10), (2, 64, 10),
                                  (2, 0, 0), (2, 0, 1000001)):
        assert L.ct_selftest_norm_wait(blocks, thread, limit, None) == ARG


class Recorder:
    """In place of the library: sizes from it, other calls kept."""
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in ("moe_sorted_rows", "moe_sort_workspace_size"):
            return getattr(self.real, name)
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def cpu_plan(monkeypatch, L):
    """A plan with CPU buffers, whose calls go to a recorder."""
    import cast_transpose_gb300.moe as moe
    recorder = Recorder(L)
    monkeypatch.setattr(moe, "lib", lambda: recorder)
    monkeypatch.setattr(moe, "_ptr", lambda t, name, dtype, shape: t.data_ptr())
    monkeypatch.setattr(moe, "_dev", lambda t, *rest: t.data_ptr())
    monkeypatch.setattr(moe, "_stream", lambda stream: 0)
    return ct.MoePlan(10000, 4, 8, align=16, device="cpu"), recorder


ATTRIBUTES = ("row_of", "src", "offsets", "counts", "workspace", "tokens", "topk", "experts",
              "align", "rows", "slots")


@pytest.mark.parametrize("name", ATTRIBUTES)
def test_a_plans_sizes_and_buffers_cannot_be_replaced(cpu_plan, name):
    plan, _ = cpu_plan
    before = getattr(plan, name)
    with pytest.raises(AttributeError):
        setattr(plan, name, before)
    assert getattr(plan, name) is before


def test_a_plans_addresses_are_those_of_its_buffers_now(cpu_plan):
    """Also where a buffer's memory has been exchanged since."""
    plan, recorder = cpu_plan
    for t in (plan.row_of, plan.src, plan.offsets, plan.counts, plan.workspace):
        t.set_(torch.zeros_like(t))
    idx, x = torch.zeros(10000, 4, dtype=torch.int32), torch.zeros(10000, 8)
    out, w = torch.zeros(plan.rows, 8), torch.zeros(10000, 4)
    ct.moe_sort(idx, plan)
    ct.moe_dispatch(x, plan, out)
    ct.moe_dispatch_backward(out, plan, x)
    ct.moe_combine(out, plan, w, x)
    ct.moe_combine_backward(x, out, plan, w, out, w)
    one, q = torch.zeros(1), torch.zeros(plan.rows, 8, dtype=torch.uint8)
    ct.fp8_moe_dispatch(x, plan, one, one, one, q)
    row_of, src, offsets, counts, ws = (t.data_ptr() for t in (
        plan.row_of, plan.src, plan.offsets, plan.counts, plan.workspace))
    args = dict(recorder.calls)
    assert args["moe_sort"][7:12] == (row_of, src, offsets, counts, ws)
    assert args["moe_dispatch"][5:7] == (row_of, src)
    assert args["moe_dispatch_backward"][5] == row_of
    assert args["moe_combine"][5] == row_of
    assert args["moe_combine_backward"][6:8] == (row_of, src)
    assert args["fp8_moe_dispatch"][4] == src


MOST = 2 ** 31 - 1


def test_blocks_beyond_a_launch(L):
    """One block per token and one per 32 sorted rows have to fit a grid."""
    def dispatch(tokens, rows):
        return L.moe_dispatch(A, tokens, 1, 1, 0, B, C, rows, D, None, None)

    def backward(tokens, rows, dys=F, dw=G):
        return L.moe_combine_backward(A, B, tokens, 1, 1, 0, C, D, E, rows, dys, dw, None, None)
    for call in (dispatch, backward):
        assert call(MOST, 1) == SHAPE
        assert call(MOST - 1, 33) == SHAPE
        assert call(MOST // 33 * 32 + 33, MOST) == SHAPE
    # nothing is sorted: a block per token alone (here no further than its buffers)
    assert backward(MOST, MOST, dys=None, dw=G + 2) == ALIGN
    assert L.moe_combine(A, MOST, 1, 1, 0, B, C, 1, D + 1, None, None) == ALIGN


def test_limits_of_hidden_and_of_a_sorted_matrix(L):
    def dispatch(hidden, rows):
        return L.moe_dispatch(A, 10, 2, hidden, 0, B, C, rows, D + 1, None, None)

    def cast(hidden, rows):
        return L.fp8_moe_dispatch(A + 1, 10, 2, hidden, B, rows, None, C, D, E, F, None, 0, None, None)
    for call in (dispatch, cast):
        assert call(2 ** 20 + 1, 1) == SHAPE
        assert call(2 ** 20, 2 ** 20 + 1) == SHAPE
        assert call(2 ** 20, 2 ** 20) == ALIGN          # within them


def test_norm_errors_name_the_argument():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="dres"):            # the signature's default
        ct.block_norm_backward(x, None, x, x, None, None, x)
    with pytest.raises(TypeError, match="dy"):              # neither u nor dy: no type
        ct.block_norm_backward(None, None, None, x, None, None, None, x)
    with pytest.raises(TypeError, match="res"):
        ct.block_norm(x, None, x, x)
    with pytest.raises(TypeError, match="u must"):
        ct.block_norm([1.0], x, x, x)
    with pytest.raises(TypeError, match="w_pre"):
        ct.block_norm(x, x, x, x, w_pre=1.0)
    with pytest.raises(ValueError, match="res"):
        ct.block_norm(x, x[0], x, x)
    with pytest.raises(ValueError, match="dres"):
        ct.block_norm_backward(x, None, x, x, None, None, x, x[0])


class Gpu(torch.Tensor):
    """A CPU tensor that says it is on a GPU: as far as the binding's checks go."""
    is_cuda = True


def test_norm_outputs_of_another_kind_are_named():
    x = torch.zeros(4, 8, dtype=torch.bfloat16).as_subclass(Gpu)
    with pytest.raises(TypeError, match="res_out must"):
        ct.block_norm(x, x, 3.0, x)
    with pytest.raises(TypeError, match="du must"):
        ct.block_norm_backward(x, None, x, x, None, None, "du", x)


def test_current_stream_without_torchs_private_names(monkeypatch):
    """The handle comes from two private functions of torch; where a version
    has them no longer, from the public call."""
    class Stream:
        cuda_stream = 0x1234

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream)
    assert ct._stream(None) == 0x1234
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    assert ct._stream(None) == 0x1234
    assert ct._stream(Stream) == 0x1234


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
@pytest.mark.parametrize("unit", ["ct_moe", "ct_moe_cast", "ct_norm", "ct_ops_api"])
def test_a_launch_needs_no_host_memory(unit):
    """An allocation that failed would leave the C entry point as an exception:
    the library's own objects ask for none."""
    path = os.path.join(os.path.dirname(ct.__file__), "_build", unit + ".o")
    wanted = subprocess.run(["nm", "-uC", path], capture_output=True, text=True, check=True).stdout
    assert "operator new" not in wanted and "__throw_length_error" not in wanted


def test_a_refused_data_type_is_called_that(L):
    assert L.moe_dispatch(A, 1, 1, 8, 3, B, C, 1, D, None, None) == FORMAT
    assert "data type" in L.ct_status_string(FORMAT).decode()
