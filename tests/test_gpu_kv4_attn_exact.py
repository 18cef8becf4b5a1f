"""Attention over the 4-bit cache (include/lora_kv.h) against fp64 to within what
each of its paths rounds, at the places where its shares, rings and joins change."""
import os
import sys

import pytest
import torch

from segmented_gemm_gb300 import kv as KV
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


@pytest.mark.parametrize("H,Hk,D", [(32, 8, 128), (32, 4, 64)])
def test_a_workspace_of_the_largest_step_unpacks_the_chunks_of_smaller_ones(H, Hk, D):
    """A server has one workspace, by its most tokens and most requests.  A step of one chunk takes the same path over it
    as over one made for the step: the same bits, which the path without unpacking does not give."""
    server = KV.Kv4Workspace(512, 256, H, Hk, D)
    assert server.unpack_tokens > 0
    s = Step([512], [700], H, Hk, D, 16, seed=H)
    assert s.any_wide
    want, lse = s.check()
    s.ws = server
    o, lse2 = s.run()
    assert torch.equal(o, want) and torch.equal(lse2, lse) and L.lora_get_status(server) == 0
    s.ws = KV.Kv4Workspace(512, 1, H, Hk, D, unpack_tokens=0)
    assert not torch.equal(s.check()[0], want)
