"""The stream that a call without one goes to."""
import os
import subprocess
import sys

import pytest
import torch

import cast_transpose_gb300 as ct

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_is_torchs_current_one():
    assert ct._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert ct._stream(None) == side.cuda_stream
    assert ct._stream(None) == torch.cuda.current_stream().cuda_stream
    assert ct._stream(side) == side.cuda_stream


def test_of_a_program_that_has_not_used_the_gpu_yet():
    code = ("import cast_transpose_gb300 as ct\n"
            "ct.selftest_bounded_wait(1000)\n"
            "assert ct.device_error() == 2\n"
            "import torch\n"
            "x = torch.ones(32, 64, dtype=torch.bfloat16, device='cuda')\n"
            "q, qt = ct.empty_outputs(x)\n"
            "s, a, i = (torch.ones(1, device='cuda') for _ in range(3))\n"
            "ct.fp8_cast_transpose(x, s, a, i, q, qt)\n"
            "assert bool((q == 0x38).all()) and bool((qt == 0x38).all())\n")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, timeout=300)
