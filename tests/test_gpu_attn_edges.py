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


def test_a_list_of_the_other_kind_or_bound_runs_nothing():
    s = Step([3] * 40, [3 + 5 * r for r in range(40)], 4, 2, 64, 16, seed=1)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(s.T, 2, 64, generator=g).to(BF).cuda() for _ in range(2))
    sched = s.schedule()
    want, lse0 = s.run(sched=sched)
    assert L.lora_get_status(s.ws) == 0
    A.lora_attn_prompt(s.q, k, v, s.cu, s.scale, s.ws)   # more requests than a short list holds: builds its own
    o, lse = s.run(sched=sched)
    assert L.lora_get_status(s.ws) == L.LORA_DEV_CHECK
    assert torch.isnan(o.float()).all() and torch.isnan(lse).all()
    prompt = A.lora_attn_schedule(s.cu, None, s.T, s.T, 4, 2, 64, s.ws)
    s.schedule()
    A.lora_attn_prompt(s.q, k, v, s.cu, s.scale, s.ws, sched=prompt)
    assert L.lora_get_status(s.ws) == L.LORA_DEV_CHECK
    sched = s.schedule()
    A.lora_attn_schedule(s.cu, s.kv_len, s.T, 100, 4, 2, 64, s.ws)   # clamps the longer requests
    assert L.lora_get_status(s.ws) == A.LORA_DEV_BAD_LENGTH
    s.run(sched=sched)
    assert L.lora_get_status(s.ws) == L.LORA_DEV_CHECK
    o, lse = s.run(sched=s.schedule())
    assert L.lora_get_status(s.ws) == 0 and torch.equal(o, want) and torch.equal(lse, lse0)


def stream_of(t):
    """The stream whose pool the caching allocator took t from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not of the caching allocator")


def test_outputs_made_by_a_call_belong_to_its_stream():
    s = Step([1, 20, 1], [700, 90, 33], 8, 2, 64, 16, seed=15)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(s.T, 2, 64, generator=g).to(BF).cuda() for _ in range(2))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = A.lora_attn_paged(s.q, s.k_cache, s.v_cache, s.table, s.cu, s.kv_len, s.scale, s.ws, stream=side)
    assert stream_of(o) == side.cuda_stream
    o = A.lora_attn_prompt(s.q, k, v, s.cu, s.scale, s.ws, stream=side)
    assert stream_of(o) == side.cuda_stream
    i32 = dict(dtype=torch.int32, device="cuda")
    args = [torch.tensor([1, 2, 3], **i32), torch.tensor([0, 5, 9], **i32), torch.zeros(3, 4, **i32),
            torch.arange(10, **i32), torch.zeros(1, **i32)]
    torch.cuda.synchronize()
    plan = A.lora_kv_plan(*args, 16, 20, s.ws, max_tokens=8, stream=side)
    for t in (plan.cu_new, plan.kv_len, plan.free_head, plan.slot_map, plan.position, plan.lora_id_map):
        assert stream_of(t) == side.cuda_stream
    side.synchronize()
    assert plan.cu_new.tolist() == [0, 1, 3, 6]
    # and, where the call is on the current stream, to that one
    o = A.lora_attn_paged(s.q, s.k_cache, s.v_cache, s.table, s.cu, s.kv_len, s.scale, s.ws)
    assert stream_of(o) == torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()


def test_a_refused_request_keeps_its_context():
    """The serving example's bookkeeping where the free pages run short for a step."""
    from test_gpu_attn_serving import _example
    ex = _example()
    R, hidden = 3, 256
    m = ex.Model(R, 1, hidden, 4, 2, 64, 16, 64, 64, seed=3)
    g = torch.Generator().manual_seed(4)
    xs, ys = [[] for _ in range(R)], [[] for _ in range(R)]

    def step(new, prompts, refused=()):
        x = torch.randn(sum(new), hidden, generator=g).to(BF)
        y = m.step(x.cuda(), new, prompts).cpu()
        at = 0
        for r, n in enumerate(new):
            if r not in refused:
                xs[r].append(x[at:at + n])
                ys[r].append(y[at:at + n])
            at += n
    step([16, 20, 7], True)
    assert m.ctx.tolist() == [16, 20, 7] and L.lora_get_status(m.ws) == 0
    free, m.free = m.free, m.free[:4]          # all four pages are taken
    step([1, 1, 1], False, refused=(0,))       # request 0 needs a fifth
    assert L.lora_get_status(m.ws) == A.LORA_DEV_NO_PAGE
    assert m.ctx.tolist() == [16, 21, 8]
    m.free = free                              # pages came free again
    step([2, 1, 3], False)
    step([1, 1, 1], False)
    assert m.ctx.tolist() == [19, 23, 12] and L.lora_get_status(m.ws) == 0
    for r in range(R):
        got, ref = torch.cat(ys[r]).double(), m.recompute(r, torch.cat(xs[r]))
        assert float((got - ref).norm() / ref.norm()) <= 13 * 2.0 ** -8, r


def work_list(ws):
    """The header of the work list in a workspace: blocks, units, weight of a cut (0: whole groups), heads of a section."""
    return dict(zip(("blocks", "units", "cut", "sec_heads"), ws.buf[768:784].view(torch.int32).tolist()))


def list_of(new, kv, H, Hk, D):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    T, R, i32 = cu[-1], len(new), dict(dtype=torch.int32, device="cuda")
    ws = A.AttnWorkspace(T, R, H, Hk, D)
    A.lora_attn_schedule(torch.tensor(cu, **i32), None if kv is None else torch.tensor(kv, **i32), T,
                         T if kv is None else max(kv), H, Hk, D, ws)
    assert L.lora_get_status(ws) == 0
    return work_list(ws)


@pytest.mark.parametrize("H,Hk,D", [(1, 1, 128), (4, 1, 128), (8, 1, 128), (16, 2, 128), (1, 1, 64), (8, 1, 64)])
def test_groups_of_many_rows_are_cut_only_where_the_join_pays(H, Hk, D):
    """Lists whose cut pieces took 1.2 to 3 times as long to run and join as the whole groups."""
    for T in (1024, 2048):
        assert list_of([T], None, H, Hk, D)["cut"] == 0, T
    if H // Hk < 8:
        assert list_of([256], [4352], H, Hk, D)["cut"] == 0
    assert list_of([1024], [2024], H, Hk, D)["cut"] == 0
    # and ones that take 2 to 5 times as long whole
    assert list_of([1], [3000], H, Hk, D)["cut"] == 1
    assert list_of([1] * 12, [250 * r + 90 for r in range(12)], H, Hk, D)["cut"] == 1
    if H == 1:
        assert list_of([16384], None, H, Hk, D)["cut"] == 2
    else:
        assert list_of([512], [16512], H, Hk, D)["cut"] == 2


@pytest.mark.parametrize("H,Hk,D,lens", [(1, 1, 128, [12000]), (4, 1, 64, [8000]), (2, 2, 64, [50] * 9 + [9000])])
def test_long_prompts_of_few_heads_run_as_with_a_schedule(H, Hk, D, lens):
    """Too long for the list that the attention kernel makes itself, though of few groups: whole groups
    would take 1.2 to 2 times as long as the schedule's cut list, whose results these are to the bit."""
    T, R = sum(lens), len(lens)
    g = torch.Generator(device="cuda").manual_seed(T)
    q = torch.randn(T, H, D, device="cuda", generator=g).to(BF)
    k, v = (torch.randn(T, Hk, D, device="cuda", generator=g).to(BF) for _ in "kv")
    cu = torch.tensor([sum(lens[:i]) for i in range(R + 1)], dtype=torch.int32, device="cuda")
    ws = A.AttnWorkspace(T, R, H, Hk, D)
    o = A.lora_attn_prompt(q, k, v, cu, D ** -0.5, ws)
    sched = A.lora_attn_schedule(cu, None, T, T, H, Hk, D, ws)
    assert work_list(ws)["cut"] == 2
    with_sched = A.lora_attn_prompt(q, k, v, cu, D ** -0.5, ws, sched=sched)
    assert L.lora_get_status(ws) == 0
    assert torch.equal(o, with_sched)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_the_largest_values_that_the_header_promises(n, D):
    """Values of 2^60, under scores that all lie just as far above each tile's first as leaves the row's reference alone."""
    s = Step([n, n], [3000, 500], 4, 1, D, 16, seed=7)
    s.q_cpu = torch.zeros(s.T, 4, D, dtype=torch.float64)
    s.q_cpu[:, :, 0] = 1.0
    s.q, s.scale = s.q_cpu.to(BF).cuda(), 0.25
    kc, vc = s.k_cache.cpu(), s.v_cache.cpu()
    for r, length in enumerate(s.kv):
        for pos in range(length):
            page, slot = int(s.table[r, pos // 16]), pos % 16
            kc[page, 0, slot] = 0
            kc[page, 0, slot, 0] = 0.0 if pos % 128 == 0 else 92.0   # scores 0 and 23: p of 2^33, 2^39 in half a tile
            vc[page, 0, slot] = s.values[r][pos, 0].sign().to(BF) * 2.0 ** 60
            s.keys[r][pos, 0] = kc[page, 0, slot].double()
            s.values[r][pos, 0] = vc[page, 0, slot].double()
    s.k_cache.copy_(kc)
    s.v_cache.copy_(vc)
    s.check("large values")


def test_shapes_that_do_not_fit_are_refused():
    s = Step([2, 3], [40, 50], 4, 2, 64, 16, seed=13)
    k = torch.zeros(5, 2, 64, dtype=BF, device="cuda")
    flat = s.q.flatten(1)                      # a projection's rows, heads not told apart
    for q, kk, v in ((flat, k, k), (s.q, flat, k), (s.q, k, flat), (s.q, k[:4], k[:4]), (s.q[..., :32], k, k),
                     (s.q, k, k[:, :1]), (s.q.float(), k, k)):
        with pytest.raises(ValueError):
            A.lora_attn_prompt(q, kk, v, s.cu, s.scale, s.ws)
    for q in (flat, s.q[..., :32], s.q.float()):
        with pytest.raises(ValueError):
            A.lora_attn_paged(q, s.k_cache, s.v_cache, s.table, s.cu, s.kv_len, s.scale, s.ws)
    for q, kk in ((k[:, 0], k), (k, k[:, 0]), (k[:, :1], k[:, :1]), (k[..., :32], k[..., :32])):
        with pytest.raises(ValueError):
            A.lora_kv_store(q, kk, s.k_cache, s.v_cache, torch.zeros(5, dtype=torch.int32, device="cuda"), s.ws)
    s.check()
