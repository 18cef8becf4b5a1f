"""The attention operators where a size, a bound or a stream changes what runs:
launch limits, lists that another list replaces, clamped lengths, outputs made
for another stream.  Tolerances as in test_gpu_attn.py."""
import math
import os
import subprocess
import sys

import pytest
import torch

from segmented_gemm_gb300 import attn as A
from segmented_gemm_gb300 import lora as L

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_attn import BF, Prompt, Step, assert_attn, reference  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_plan_of_nearly_the_most_requests():
    """4075 to 4095 requests need more shared memory than a launch has without asking for it, 4074 do not.
    In a process of their own, where no call of 4096 has asked before."""
    code = ("import sys; sys.path[:0] = ['tests', '.']\n"
            "from test_gpu_attn import check_plan\n"
            "for R in (4074, 4075, 4095, 4096):\n"
            "    new, ctx = [r % 5 for r in range(R)], [r % 37 for r in range(R)]\n"
            "    check_plan(new, ctx, 16, 4, list(range(3 * R)), sum(new) + 3, 3 * R, seed=R)\n")
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
