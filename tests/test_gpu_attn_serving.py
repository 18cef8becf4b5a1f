"""The attention operators in use: the serving example from one end to the
other, waits that run out, and a work list that does not fit its call."""
import math
import os
import sys

import pytest
import torch

from segmented_gemm_gb300 import attn as A
from segmented_gemm_gb300 import lora as L

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_attn import Step, assert_attn, reference  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _example():
    import importlib.util
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_attention.py")
    spec = importlib.util.spec_from_file_location("serve_attention", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("cfg", [dict(), dict(requests=3, layers=1, heads=4, kv_heads=4, head_dim=128, page=32),
                                 dict(requests=9, steps=5, heads=6, kv_heads=1, head_dim=80, page=8, hidden=384)])
def test_serving_example(cfg):
    """bf16 (u = 2^-8) is rounded to in QKV, p, o, the output projection and the sum, 5 u a layer; QKV's
    rounding moves a score by at most 2 u times its magnitude (4 covers them here), and p with it, 8 u more."""
    status, errors = _example().serve(**cfg)
    assert status == 0
    assert max(errors) <= 13 * 2.0 ** -8 * cfg.get("layers", 2), errors


@pytest.mark.parametrize("budget", [100, 1000, 3000, 10000])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(budget):
    """A budget shorter than a healthy wait: the kernel gives up somewhere,
    says so, and returns.  (Not in every call: one try of a barrier may itself
    suspend for longer than the load that it waits for takes, and only what
    is still waited for after it counts.)  With a new schedule the same
    workspace serves the next call."""
    s = Step([1] * 20 + [300, 7], [2000 - 90 * i for i in range(20)] + [900, 40], 8, 2, 128, 16, seed=5)
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(s.T, 2, 128, generator=g).to(BF).cuda() for _ in range(2))
    statuses = []
    L.lora_set_wait_budget(budget)
    try:
        for _ in range(3):
            s.run()
            statuses.append(L.lora_get_status(s.ws))
            A.lora_attn_prompt(s.q, k, v, s.cu, s.scale, s.ws)
            statuses.append(L.lora_get_status(s.ws))
    finally:
        L.lora_set_wait_budget(0)
    assert all(x in (0, L.LORA_DEV_TIMEOUT) for x in statuses), statuses
    if budget == 100:
        assert L.LORA_DEV_TIMEOUT in statuses, statuses
    s.check("after the timeouts")
    s.check("with a schedule", sched=s.schedule())


def test_a_schedule_of_other_sizes_in_the_workspace_runs_nothing():
    s = Step([1, 40, 3], [50, 700, 3], 8, 2, 64, 16, seed=8)
    big = Step([1, 400, 3], [50, 700, 3], 8, 2, 64, 16, seed=9)
    big.check()
    small = A.lora_attn_schedule(s.cu, s.kv_len, s.T, s.table.shape[1] * s.page, s.H, s.Hk, s.D, big.ws)
    o = torch.full((s.T, s.H, s.D), 7.0, dtype=BF, device="cuda")

    def run():
        o.fill_(7.0)
        A.lora_attn_paged(s.q, s.k_cache, s.v_cache, s.table, s.cu, s.kv_len, s.scale, big.ws, sched=small, o=o)
        return L.lora_get_status(big.ws)
    assert run() == 0
    good = o.clone()
    big.run()                      # builds its own list over the small one
    assert run() == L.LORA_DEV_CHECK
    assert bool((o == 7.0).all())
    A.lora_attn_schedule(s.cu, s.kv_len, s.T, s.table.shape[1] * s.page, s.H, s.Hk, s.D, big.ws)
    assert run() == 0 and torch.equal(o, good)
    big.ws.buf.zero_()             # no list at all
    assert run() == L.LORA_DEV_CHECK


@pytest.mark.parametrize("seed", range(12))
def test_random_steps(seed):
    """Draws over head counts, dimensions, pages and mixes of lengths."""
    g = torch.Generator().manual_seed(1000 + seed)

    def pick(*xs):
        return xs[int(torch.randint(len(xs), (1,), generator=g))]

    def upto(n):
        return int(torch.randint(n + 1, (1,), generator=g))
    Hk, G, D, page = pick(1, 2, 3, 8), pick(1, 2, 4, 5, 8), pick(16, 64, 72, 96, 128), pick(8, 16, 64, 256)
    R = 1 + upto(11)
    new = [pick(0, 1, 1, 1, 2, 5, upto(200)) for _ in range(R)]
    kv = [n + pick(0, upto(40), upto(900)) if pick(True, True, True, False) else upto(n) for n in new]
    if not sum(new):
        new[0], kv[0] = 1, max(1, kv[0])
    s = Step(new, kv, Hk * G, Hk, D, page, seed=seed, order=pick("phsd", "pshd", "hpsd"), q_pad=8 * upto(3))
    s.check(f"{new} {kv} {Hk}x{G} d{D} p{page}")
    s.check("again, with a schedule", sched=s.schedule())


@pytest.mark.parametrize("seed", range(6))
def test_random_prompts(seed):
    g = torch.Generator().manual_seed(2000 + seed)
    Hk, G = (1, 2, 4)[seed % 3], (1, 4, 7)[seed // 2]
    D = (128, 64, 104)[seed % 3]
    lens = [int(torch.randint(0, 260, (1,), generator=g)) for _ in range(5)] + [1]
    T = sum(lens)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    q = torch.randn(T, Hk * G, D, generator=g).to(BF)
    k, v = (torch.randn(T, Hk, D, generator=g).to(BF) for _ in range(2))
    ws = A.AttnWorkspace(T, len(lens), Hk * G, Hk, D)
    lse = torch.empty(T, Hk * G, device="cuda")
    o = A.lora_attn_prompt(q.cuda(), k.cuda(), v.cuda(), cu, D ** -0.5, ws, lse=lse)
    assert L.lora_get_status(ws) == 0
    parts, t = [], 0
    for n in lens:
        parts.append(reference(q[t:t + n].double(), k[t:t + n].double(), v[t:t + n].double(), range(1, n + 1),
                               D ** -0.5))
        t += n
    assert_attn(o, lse, *[torch.cat(x) for x in zip(*parts)], f"{lens}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("first", [-300.0, 300.0, -math.inf])
@pytest.mark.parametrize("n", [1, 40])
def test_first_keys_far_from_the_others(D, first, n):
    """Each row's first visible score (and the first of every tile, so of each
    piece of a split context) far below, far above, or -infinity beside the others."""
    s = Step([n, n], [3000, 500], 4, 1, D, 16, seed=3)
    q = torch.randn(s.T, 4, D, generator=torch.Generator().manual_seed(4)).to(BF)
    q[:, :, 0] = 1.0
    s.q, s.q_cpu, s.scale = q.cuda(), q.double(), 0.25
    kc = s.k_cache.cpu()
    for r, length in enumerate(s.kv):
        for pos in range(0, length, 128):   # scale * q . k = first there
            page, slot = int(s.table[r, pos // 16]), pos % 16
            kc[page, 0, slot] = 0
            kc[page, 0, slot, 0] = first / s.scale
            s.keys[r][pos, 0] = kc[page, 0, slot].double()
    s.k_cache.copy_(kc)
    s.check(f"{first}")
    s.check("with a schedule", sched=s.schedule())


@pytest.mark.parametrize("H,Hk,D", [(8, 2, 128), (8, 1, 64)])
def test_chunks_beside_single_tokens_split_over_the_gpu(H, Hk, D):
    """Pieces of pairs of query tiles and of single ones in one cut list, whose tiles weigh differently."""
    tq = 128 * Hk // H
    new = [1, 2 * tq + 1, 1, tq, 0, tq + 1, 1, 3]
    s = Step(new, [2500, 2 * tq + 2001, 129, tq + 700, 40, tq + 1, 1, 1800], H, Hk, D, 16, seed=D)
    s.check("mixed")
    sched = s.schedule()
    first = s.run(sched=sched)
    again = s.run(sched=sched)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("G,D,new", [(2, 128, 1), (4, 64, 2), (1, 72, 3), (16, 128, 1)])
def test_many_short_contexts(G, D, new):
    """More groups of few rows than the GPU holds several times over: two heads of a request at a time."""
    R, Hk = 90, 8
    n = [new if r % 7 else 0 for r in range(R)]
    s = Step(n, [n[r] + (37 * r) % 290 if r % 11 else 0 for r in range(R)], G * Hk, Hk, D, 16, seed=G)
    s.check("short contexts")
    first = s.run(sched=s.schedule())
    again = s.run(sched=s.schedule())
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
