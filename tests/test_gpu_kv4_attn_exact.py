"""Attention over the 4-bit cache (include/lora_kv.h) against fp64 to within what
each of its paths rounds, at the places where its shares, rings and joins change."""
import math
import os
import sys

import pytest
import torch

from segmented_gemm_gb300 import kv as KV
from segmented_gemm_gb300 import lora as L

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_gpu_kv4_attn as beside  # noqa: E402
from test_gpu_kv4_attn import Step  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -8


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


def check_exactly(s, what=""):
    """Within what either path rounds.  o goes to bf16 once (U of it).  p goes to fp16: 2^-11 of sum_j p_j |v_j|, and where p is
    below 2^-14, 2^-25 absolutely; a row's largest p is at least 2^7, so its sum is, and the latter is at most 2^-32 max |v|
    a key.  A score's fp32 sum of up to 128 exact products loses at most 2^-20 of the sum of their magnitudes, below 100 (in
    powers of two) at these sizes, and sums of p and of products some 2^-20 of themselves: 2e-4 in all."""
    o, lse = s.run()
    assert L.lora_get_status(s.ws) == 0, what
    ref_o, ref_lse, mass = s.reference()
    vmax = max([float(v.abs().max()) for v in s.values if v.numel()] + [0.0])
    err = (o.double().cpu() - ref_o).abs()
    tol = U * ref_o.abs() + (2.0 ** -11 + 2e-4) * mass + max(s.kv) * 2.0 ** -32 * vmax
    assert torch.isfinite(o).all() and (err <= tol).all(), f"{what}: worst {(err / tol).max():.2f} x tol"
    empty = torch.isinf(ref_lse)
    lse = lse.double().cpu()
    assert torch.equal(lse == -math.inf, empty), what
    assert empty.all() or float((lse - ref_lse)[~empty].abs().max()) <= 2e-4, what


@pytest.mark.parametrize("sharp", [1.0, 8.0])   # 8: scores some 30 above and below a row's first one
@pytest.mark.parametrize("unpack", [0, None])
@pytest.mark.parametrize("H,Hk,D,page", [(32, 8, 128, 16), (16, 2, 64, 32), (24, 3, 96, 64), (32, 4, 40, 16), (128, 1, 80, 128)])
def test_chunks_and_single_tokens_to_what_is_rounded(H, Hk, D, page, unpack, sharp):
    s = Step([1, 200, 0, 5, 33, 1, 130, 2, 64, 90], [300, 450, 77, 5, 33, 1, 600, 129, 64, 20], H, Hk, D, page, seed=H, unpack=unpack)
    s.scale *= sharp
    check_exactly(s)


@pytest.mark.parametrize("sharp", [1.0, 8.0])
@pytest.mark.parametrize("H,Hk,D", [(8, 2, 128), (4, 4, 64), (7, 1, 128), (16, 1, 80), (10, 2, 8), (128, 1, 64)])
def test_few_tokens_to_what_is_rounded(H, Hk, D, sharp):
    s = Step([1, 1, 2, 1, 3, 1, 1, 5, 1, 1], [1, 2, 15, 16, 17, 127, 128, 129, 3000, 33], H, Hk, D, 16, seed=H + D)
    s.scale *= sharp
    check_exactly(s)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,unpack", [(100, None), (100, 0), (1, None)])
def test_weights_keep_eleven_bits(n, unpack, D):
    """Every other key has a weight that rounding to bf16's 8 bits takes down by nearly 2^-8 of it, and the values cancel:
    the outputs are far smaller than what they are sums of, and such a rounding would be most of them."""
    s = Step([n], [n + 901], 64, 8, D, 16, seed=1, unpack=unpack)
    w = 1 + 2.0 ** -8 - 2.0 ** -12
    odd = torch.arange(n + 901) % 2 == 1
    k, v = torch.zeros(2, n + 901, 8, D).to(BF)
    k[odd, :, 0] = 6.0
    v[~odd], v[odd] = -6.0, 6.0
    t = torch.arange(n + 901)
    KV.lora_kv4_store(k.cuda(), v.cuda(), s.cache, (s.table[0].cpu()[t // 16] * 16 + t % 16).int().cuda(), s.ws)
    s.keys, s.values = [k.double()], [v.double()]
    s.q.zero_()
    s.q[..., 0] = 1.0
    s.q_cpu = s.q.double().cpu()
    s.scale = math.log(w) / 6.0
    check_exactly(s)


@pytest.mark.parametrize("H,D,new,kv", [(4, 128, 1, 90000), (4, 64, 1, 90000), (8, 64, 2, 90000), (1, 128, 1, 60005),
                                        (3, 72, 2, 38917), (8, 128, 1, 78000), (4, 128, 1, 9000)])
def test_one_group_over_the_whole_gpu(H, D, new, kv):
    """One key head of one request, in pieces over every CTA there is (from some 78000 keys on; two tiles are the
    least share of a warp), or over some of them, of which the last one has a few warps at work."""
    s = Step([new], [kv], H, 1, D, 16, seed=kv, spare=2)
    check_exactly(s)
    o, lse = s.run()
    again, lse2 = s.run()
    assert torch.equal(o, again) and torch.equal(lse, lse2)


def test_waits_that_give_up_do_so_and_the_next_call_is_right():
    """A budget that no first load can meet.  (Not every call has to run out: one try of a barrier may itself
    suspend for longer than the load takes.)"""
    s = Step([1] * 40, [4000 - 90 * i for i in range(40)], 32, 8, 128, 16, seed=5)
    want, _ = s.run()
    seen = 0
    L.lora_set_wait_budget(1)
    try:
        for _ in range(20):
            s.run()
            seen |= L.lora_get_status(s.ws)
    finally:
        L.lora_set_wait_budget(0)
    assert seen == L.LORA_DEV_TIMEOUT
    o, _ = s.run()
    assert L.lora_get_status(s.ws) == 0 and torch.equal(o, want)


def test_the_operators_in_use_over_the_4_bit_cache(monkeypatch):
    """The serving steps of the test beside this one, its attention held to what fp16 p rounds."""
    def exactly(o, lse, ref_o, ref_lse, mass, vmax, wide, what=""):
        err = (o.double().cpu() - ref_o).abs()
        tol = U * ref_o.abs() + (2.0 ** -11 + 2e-4) * mass + 200 * 2.0 ** -32 * vmax
        assert (err <= tol).all(), f"{what}: worst {(err / tol).max():.2f} x tol"
        assert float((lse.double().cpu() - ref_lse).abs().max()) <= 1e-4, what
    monkeypatch.setattr(beside, "assert_attn4", exactly)
    beside.test_the_operators_in_use(4)


@pytest.mark.parametrize("cfg", [dict(requests=6, layers=1, steps=10), dict(requests=5, layers=2, steps=6, head_dim=128, kv_heads=1)])
def test_serving_example_with_rotation(cfg):
    """Norms and rotation round queries and keys to bf16 (u = 2^-8) once more, so a score moves by up to 4 u times its
    magnitude (4 covers these) and p with it, 16 u; with p, o, QKV, the output projection and the sum 21 u a layer."""
    from test_gpu_attn_serving import _example
    status, errors = _example().serve(rope=True, **cfg)
    assert status == 0 and max(errors) <= 21 * U * cfg["layers"], errors
