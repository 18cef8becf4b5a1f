"""Attention over the 4-bit cache (include/lora_kv.h) against fp64 to within what
each of its paths rounds, at the places where its shares, rings and joins change."""
import os
import sys

import pytest
import torch

from segmented_gemm_gb300 import lora as L

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_kv4_attn import Step  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_first_tiles_arrive_where_the_shares_were_counted(D):
    """The units before each thread's requests are kept where the first warp's tiles of keys and values arrive.  Short
    requests, so that every CTA's first warp starts its ring at once; many calls in a row, with the same bits."""
    s = Step([1] * 700, [1 + (7 * r) % 37 for r in range(700)], 4, 1, D, 16, seed=D)
    o, lse = s.check()
    for _ in range(50):
        again, lse2 = s.run()
        assert torch.equal(again, o) and torch.equal(lse2, lse)
    assert L.lora_get_status(s.ws) == 0
