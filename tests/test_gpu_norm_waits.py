"""The norms' bounded waits: a thread that gives up is reported, whichever it
is, and ends the kernel without a fault.  ct_selftest_norm_wait makes one
thread go on as if its wait had run out; what depends on it runs into the
(short) limit."""
import pytest
import torch

import cast_transpose_gb300 as ct

pytestmark = pytest.mark.gpu

LIMIT_US = 50000


def milliseconds(blocks, thread):
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    ct.selftest_norm_wait(blocks, thread, LIMIT_US)
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end)


def norm_still_right():
    """The kernels after it start from their own barriers."""
    u = torch.ones(9, 12288, dtype=torch.bfloat16, device="cuda")
    res, y = torch.zeros_like(u), torch.empty_like(u)
    ct.block_norm(u, res, res, y, eps=0.0)
    assert bool((res == 1).all()) and bool((y == 1).all())


# thread 0 arrives for its block, lane 0 of a warp for the warp (one block) or
# sends to the first block (a cluster)
@pytest.mark.parametrize("blocks", [1, 2, 4, 8])
@pytest.mark.parametrize("thread", [0, 32])
def test_a_thread_that_others_wait_for(blocks, thread):
    ct.device_error(clear=True)
    took = milliseconds(blocks, thread)
    assert ct.device_error(clear=True) == 2
    assert LIMIT_US / 1000 <= took < 100 * LIMIT_US / 1000
    norm_still_right()
    assert ct.device_error() == 0


# lanes that neither arrive nor send: nobody else gives up, and it is known all the same
@pytest.mark.parametrize("blocks", [1, 2, 4, 8])
@pytest.mark.parametrize("thread", [9, 31, 63])
def test_a_thread_that_nobody_waits_for(blocks, thread):
    ct.device_error(clear=True)
    took = milliseconds(blocks, thread)
    assert ct.device_error(clear=True) == 2
    assert took < LIMIT_US / 1000
    norm_still_right()
    assert ct.device_error() == 0
