"""Further host-side checks of the expert-movement and block-norm operators (no
GPU needed): limits, refusals and their messages, the plan's attributes."""
import pytest

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
