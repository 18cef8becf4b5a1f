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


@pytest.mark.parametrize("D", [64, 128])
def test_clamped_lengths_of_prompts(D):
    """A prompt of n rows clamped to L keys: row i sees the first max(0, L - n + i + 1) keys of its prompt."""
    p = Prompt([50, 300, 0, 131, 700], 4, 2, D, seed=D)
    for most in (130, 299, 1):
        sched = A.lora_attn_schedule(p.cu, None, p.T, most, 4, 2, D, p.ws)
        o, lse = p.run(sched=sched)
        assert L.lora_get_status(p.ws) == A.LORA_DEV_BAD_LENGTH
        parts, t = [], 0
        for n in p.lens:
            q, k, v = (x[t:t + n] for x in p.cpu)
            parts.append(reference(q, k, v, [max(0, min(n, most) - n + i + 1) for i in range(n)], p.scale))
            t += n
        assert_attn(o, lse, *[torch.cat(x) for x in zip(*parts)], f"at most {most}")


def test_clamped_lengths_of_a_cache():
    s = Step([2, 150, 1], [40, 400, 900], 4, 2, 64, 16, seed=13)
    for most in (399, 48, 1):
        sched = A.lora_attn_schedule(s.cu, s.kv_len, s.T, most, 4, 2, 64, s.ws)
        o, lse = s.run(sched=sched)
        assert L.lora_get_status(s.ws) == A.LORA_DEV_BAD_LENGTH
        parts, t = [], 0
        for n, length, k, v in zip(s.new, s.kv, s.keys, s.values):
            lim = [max(0, min(length, most) - n + i + 1) for i in range(n)]
            parts.append(reference(s.q_cpu[t:t + n], k, v, lim, s.scale))
            t += n
        assert_attn(o, lse, *[torch.cat(x) for x in zip(*parts)], f"at most {most}")
