"""The attention's work lists beyond the sizes of the other tests: whole groups
claimed by more units than the GPU has CTAs, sections of heads, thousands of
requests, cut lists of more than a thousand blocks.  Each is run twice in one
workspace (the counters go back to zero) and checked against fp64 in rows
picked over all requests; tolerances as in test_gpu_attn.py."""
import math
import os
import sys

import pytest
import torch

from segmented_gemm_gb300 import attn as A
from segmented_gemm_gb300 import lora as L

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_attn import BF, Step, assert_attn  # noqa: E402
from test_gpu_attn_edges import work_list  # noqa: E402

pytestmark = pytest.mark.gpu


def check_rows(o, lse, q, keys, values, first, n, length, rows, scale):
    """Rows `rows` of a request whose n query rows start at `first`: row i sees max(0, length - n + i + 1) keys."""
    D, G = q.shape[2], q.shape[1] // keys.shape[1]
    i = torch.tensor(rows, device="cuda")
    limit = (length - n + i + 1).clamp(min=0)
    qs = q[first + i].double().unflatten(1, (keys.shape[1], G))
    s = torch.einsum("rhgd,khd->rhgk", qs, keys.double()) * scale
    s = s.masked_fill((torch.arange(length, device="cuda")[None] >= limit[:, None])[:, None, None], -math.inf)
    ref_lse = torch.logsumexp(s, -1)
    p = torch.exp(s - ref_lse.clamp(min=-1e300)[..., None])
    v = values.double()
    shape = (len(rows), q.shape[1], D)
    assert_attn(o[first + i], lse[first + i], torch.einsum("rhgk,khd->rhgd", p, v).reshape(shape).cpu(),
                ref_lse.flatten(1).cpu(), torch.einsum("rhgk,khd->rhgd", p, v.abs()).reshape(shape).cpu(), f"row {first}")


def some_rows(n, many):
    return sorted({0, n - 1, n // 2, *(int(x) for x in torch.randint(n, (many,), generator=torch.Generator().manual_seed(n)))})


def prompts(lens, H, Hk, D, many):
    """Runs the prompts twice; the list that was built, and every check of the outputs."""
    g = torch.Generator(device="cuda").manual_seed(sum(lens))
    T = sum(lens)
    w = torch.randn(T, (H + 2 * Hk) * D, device="cuda", generator=g).to(BF)
    q, k, v = (x.unflatten(1, (-1, D)) for x in (w[:, :H * D], w[:, H * D:(H + Hk) * D], w[:, (H + Hk) * D:]))
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    ws = A.AttnWorkspace(T, len(lens), H, Hk, D)
    out = []
    for _ in range(2):
        o = torch.full((T, H, D), float("nan"), dtype=BF, device="cuda")
        lse = torch.full((T, H), float("nan"), device="cuda")
        A.lora_attn_prompt(q, k, v, cu, D ** -0.5, ws, o=o, lse=lse)
        assert L.lora_get_status(ws) == 0
        out.append((o, lse))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
    at = 0
    for r, n in enumerate(lens):
        if n and (len(lens) < 50 or r % 37 == 0):
            check_rows(o, lse, q, k[at:at + n], v[at:at + n], at, n, n, some_rows(n, many), D ** -0.5)
        at += n
    return work_list(ws)


@pytest.mark.parametrize("D", [64, 128])
def test_whole_groups_of_long_prompts(D):
    # pairs of query tiles one after another in a CTA, their streams' turns among them
    w = prompts([2900, 2200], 16, 8, D, 60)
    assert w["cut"] == 0 and w["units"] == 41 * 8


def test_sections_of_heads():
    # 45000 keys: two heads of 128 fill a section, the last section has one
    w = prompts([3000] * 15, 5, 5, 128, 12)
    assert w["cut"] == 0 and w["sec_heads"] == 2 and w["units"] == 180 * 5


def test_thousands_of_short_prompts():
    w = prompts([1 + (r * 5) % 9 for r in range(1300)], 6, 3, 128, 3)
    assert w["cut"] == 0 and w["blocks"] == 1300


def paged(s, want_cut):
    """Twice the step; every row by its own request's keys."""
    sched = s.schedule()
    w = work_list(s.ws)
    assert (w["cut"] != 0) == want_cut
    first, lse0 = s.run(sched=sched)
    o, lse = s.run(sched=sched)
    assert L.lora_get_status(s.ws) == 0
    assert torch.equal(first, o) and torch.equal(lse0, lse)
    assert_attn(o, lse, *s.reference(), "paged")
    return w


def test_thousands_of_requests():
    new = [(r * 7) % 4 for r in range(1500)]
    w = paged(Step(new, [n + (r * 13) % 60 for r, n in enumerate(new)], 4, 1, 64, 16, seed=1), False)
    assert w["blocks"] == 1125 and w["units"] == 1125


def test_whole_groups_of_chunks():
    # units of one and of two query tiles, claimed by CTAs as they come free
    n, kv = [130, 70, 1, 210, 150, 33, 90, 64, 200, 5, 140], [400, 270, 500, 600, 150, 33, 300, 320, 700, 450, 141]
    w = paged(Step(n, kv, 32, 8, 64, 16, seed=2), False)
    assert w["units"] == w["blocks"] * 8 == 200


def test_units_of_one_head_beyond_the_ctas():
    # an odd number of kv heads: no two heads at a time
    w = paged(Step([1 + r % 3 for r in range(70)], [3 + (r * 31) % 190 for r in range(70)], 9, 3, 72, 8, seed=3), False)
    assert w["units"] == 210


def test_a_cut_list_of_more_than_a_thousand_blocks():
    s = Step([1] * 1101, [20] * 1100 + [20000], 4, 1, 64, 16, seed=4)
    w = paged(s, True)
    assert w["blocks"] == 1101
