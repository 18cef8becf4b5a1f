"""The attention operators (include/lora_attn.h) against plain fp64
implementations: cache plan, cache store, paged and prompt attention.

Tolerance of an output element, from the two bf16 roundings the kernels make
(unit roundoff u = 2^-8): o itself is rounded once, u |o|, and every p_j is
rounded before the second product, which moves o by at most u sum_j p_j |v_j|.
fp32 scores of up to 128 terms and the fp32 sums add less than 2e-4 of
sum_j p_j |v_j| at these magnitudes.  lse is fp32 throughout: 1e-4 absolute
covers the scores' accumulation (128 terms, |terms| summing to below 64)."""
import math

import numpy as np
import pytest
import torch

from segmented_gemm_gb300 import attn as A
from segmented_gemm_gb300 import lora as L

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
BF = torch.bfloat16


# --- helpers -----------------------------------------------------------------

def reference(q, keys, values, limits, scale):
    """One request: q [n, H, D], keys/values [len, Hk, D] (fp64), limits [n].
    Returns o, lse and the tolerance's sum_j p_j |v_j|."""
    n, H, D = q.shape
    Hk = keys.shape[1] if keys.numel() else 1
    o, mass = torch.zeros(n, H, D, dtype=torch.float64), torch.zeros(n, H, D, dtype=torch.float64)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64)
    for h in range(H):
        kv = h // (H // Hk)
        for i in range(n):
            m = int(limits[i])
            if m <= 0:
                continue
            s = keys[:m, kv] @ q[i, h] * scale
            lse[i, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[i, h])
            o[i, h] = p @ values[:m, kv]
            mass[i, h] = p @ values[:m, kv].abs()
    return o, lse, mass


def assert_attn(o, lse, ref_o, ref_lse, mass, what=""):
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.isfinite(o).all(), f"{what}: non-finite outputs"
    err = (o - ref_o).abs()
    tol = U * ref_o.abs() + (U + 2e-4) * mass + 1e-30
    assert (err <= tol).all(), f"{what}: {(err > tol).sum()} of {err.numel()} off, worst {(err / tol).max():.2f} x tol"
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty), f"{what}: empty rows"
    d = (lse - ref_lse)[~empty].abs()
    assert d.numel() == 0 or float(d.max()) <= 1e-4, f"{what}: lse off by {float(d.max()):.2e}"


class Step:
    """A step over a paged cache: requests with new and cached tokens, random
    pages, and NaN in every slot that no request holds."""

    def __init__(self, new, kv, H, Hk, D, page, seed=0, order="phsd", q_pad=0, spare=4):
        g = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.H, self.Hk, self.D, self.page = new, kv, H, Hk, D, page
        R, T = len(new), sum(new)
        pages = [-(-x // page) for x in kv]
        width = max(pages + [1]) + 1
        self.num_pages = sum(pages) + spare
        perm = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        table = torch.full((R, width), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(pages):
            table[r, :n] = perm[at:at + n]
            at += n
        shape = dict(zip("phsd", (self.num_pages, Hk, page, D)))
        kc = torch.full([shape[c] for c in order], float("nan"), dtype=BF)
        vc = kc.clone()
        axes = [order.index(c) for c in "phsd"]
        self.keys, self.values = [], []
        kv_k, kv_v = kc.permute(axes), vc.permute(axes)
        for r, n in enumerate(kv):
            k = torch.randn(n, Hk, D, generator=g).to(BF)
            v = torch.randn(n, Hk, D, generator=g).to(BF)
            self.keys.append(k.double())
            self.values.append(v.double())
            for p in range(n):
                kv_k[table[r, p // page], :, p % page] = k[p]
                kv_v[table[r, p // page], :, p % page] = v[p]
        self.table = table.cuda()
        self.k_cache, self.v_cache = kc.cuda().permute(axes), vc.cuda().permute(axes)
        wide = torch.randn(T, H * D + q_pad, generator=g).to(BF)
        self.q_cpu = wide[:, :H * D].reshape(T, H, D).double()
        self.q = wide.cuda()[:, :H * D].unflatten(1, (H, D))
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        self.T, self.R = T, R
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device="cuda")
        self.scale = 1.0 / math.sqrt(D)
        self.ws = A.AttnWorkspace(T, R, H, Hk, D)

    def run(self, sched=None, **kw):
        o = torch.full((self.T, self.H, self.D), float("nan"), dtype=BF, device="cuda")
        lse = torch.full((self.T, self.H), float("nan"), dtype=torch.float32, device="cuda")
        A.lora_attn_paged(self.q, self.k_cache, self.v_cache, self.table, self.cu, self.kv_len, self.scale, self.ws,
                          sched=sched, o=o, lse=lse, **kw)
        return o, lse

    def schedule(self):
        return A.lora_attn_schedule(self.cu, self.kv_len, self.T, self.table.shape[1] * self.page, self.H, self.Hk,
                                    self.D, self.ws)

    def reference(self):
        parts, t = [], 0
        for n, length, k, v in zip(self.new, self.kv, self.keys, self.values):
            lim = [max(0, length - n + i + 1) for i in range(n)]
            parts.append(reference(self.q_cpu[t:t + n], k, v, lim, self.scale))
            t += n
        return [torch.cat(x) for x in zip(*parts)]

    def check(self, what="", **kw):
        o, lse = self.run(**kw)
        assert L.lora_get_status(self.ws) == 0, what
        assert_attn(o, lse, *self.reference(), what)


# --- paged attention -----------------------------------------------------------

@pytest.mark.parametrize("H,Hk,D,page", [(8, 2, 128, 16), (4, 4, 64, 32), (7, 1, 128, 64), (16, 1, 80, 16),
                                         (10, 2, 8, 8), (6, 2, 40, 128), (4, 1, 120, 256), (1, 1, 128, 16),
                                         (12, 4, 72, 4096)])
def test_single_tokens(H, Hk, D, page):
    Step([1] * 9, [1, 2, 15, 16, 17, 127, 128, 129, 700], H, Hk, D, page, seed=H + D).check(f"{H}/{Hk} d{D} p{page}")


@pytest.mark.parametrize("H,Hk,D,page", [(8, 2, 128, 16), (14, 2, 64, 32), (3, 3, 96, 64)])
def test_chunks_and_single_tokens_mixed(H, Hk, D, page):
    Step([5, 0, 1, 130, 33, 0, 64, 3], [300, 40, 513, 130, 161, 0, 64, 1000], H, Hk, D, page, seed=3).check()


@pytest.mark.parametrize("n", [31, 32, 33, 63, 64, 65, 127, 129, 200])
def test_chunk_lengths_around_the_tiles(n):
    Step([n], [n + 150], 4, 1, 64, 16, seed=n).check(f"chunk {n}")


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 16, 24, 65, 128])
def test_group_sizes(group):
    Step([3, 1], [200, 129], group, 1, 64, 16, seed=group).check(f"group {group}")


@pytest.mark.parametrize("order", ["phsd", "pshd", "hpsd"])
def test_cache_orders_and_strided_queries(order):
    Step([1, 40, 2], [77, 300, 2], 8, 4, 64, 16, seed=5, order=order, q_pad=64).check(order)


def test_rows_without_keys_are_zero():
    # a request refused by the plan has rows but no keys; one with fewer keys
    # than rows leaves its first rows empty
    s = Step([3, 6, 2], [0, 4, 50], 4, 2, 64, 16, seed=6)
    s.check()
    o, lse = s.run()
    assert torch.equal(o[:5].float(), torch.zeros_like(o[:5].float()))
    assert torch.isinf(lse[:5]).all()


@pytest.mark.parametrize("kv,H,Hk", [(20000, 4, 1), (9001, 8, 8), (33333, 16, 1)])
def test_long_context_split_over_the_gpu(kv, H, Hk):
    # few rows against a long context: the key axis is split and joined
    Step([2], [kv], H, Hk, 64, 64, seed=kv).check(f"kv {kv}")


def test_ragged_decode_batch():
    rng = np.random.RandomState(2)
    kv = [int(x) for x in rng.randint(1, 3000, 24)]
    Step([1] * 24, kv, 8, 2, 128, 16, seed=8).check()


def test_schedule_serves_several_layers_and_calls_repeat_exactly():
    s = Step([1, 17, 1, 1], [900, 400, 5000, 31], 8, 2, 128, 16, seed=9)
    sched = s.schedule()
    o1, l1 = s.run(sched=sched)
    o2, l2 = s.run(sched=sched)
    o3, l3 = s.run()
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    assert torch.equal(o1, o3) and torch.equal(l1, l3)
    s.check(sched=s.schedule())


def test_large_scores_do_not_overflow():
    s = Step([1, 70], [600, 300], 4, 2, 64, 16, seed=10)
    s.q = s.q * 16           # scores of several hundred: the running maximum moves a lot
    s.q_cpu = s.q.double().cpu()
    o, lse = s.run()
    ref_o, ref_lse, mass = s.reference()
    # scores up to |s| ~ 400 carry fp32 errors of about 400 * 2^-21 = 2e-4, which scale p
    assert torch.isfinite(o.float()).all()
    err = (o.double().cpu() - ref_o).abs()
    assert (err <= U * ref_o.abs() + (U + 2e-3) * mass + 1e-30).all()
    assert float((lse.double().cpu() - ref_lse).abs().max()) <= 2e-3


def test_an_infinite_score_in_a_masked_place_does_not_leak():
    s = Step([4], [90], 2, 1, 64, 16, seed=11)
    # the key of the last token, which only the last row sees
    page, line = int(s.table[0, 89 // 16]), 89 % 16
    s.k_cache[page, :, line] = float("inf")
    o, _ = s.run()
    ref_o, _, mass = s.reference()
    err = (o.double().cpu() - ref_o).abs()[:3]
    assert (err <= U * ref_o[:3].abs() + (U + 2e-4) * mass[:3]).all()


def test_a_page_outside_the_cache_reads_as_zeros():
    s = Step([1, 1], [100, 50], 4, 2, 64, 16, seed=12)
    for bad in (-1, s.num_pages, 2 ** 31 - 1):
        t = s.table.clone()
        t[0, 2] = bad
        keep, s.table = s.table, t
        o, lse = s.run()
        s.table = keep
        assert L.lora_get_status(s.ws) == A.LORA_DEV_BAD_PAGE
        k, v = s.keys[0].clone(), s.values[0].clone()
        k[32:48] = 0
        v[32:48] = 0
        r0 = reference(s.q_cpu[:1], k, v, [100], s.scale)
        r1 = reference(s.q_cpu[1:], s.keys[1], s.values[1], [50], s.scale)
        assert_attn(o, lse, *[torch.cat(x) for x in zip(r0, r1)])


def test_lengths_out_of_range_are_clamped_and_flagged():
    s = Step([2, 3], [40, 50], 4, 2, 64, 16, seed=13)
    s.run()
    assert L.lora_get_status(s.ws) == 0
    for cu, kv in (([0, 2, 9], [40, 50]), ([-3, 2, 5], [40, 50]), ([0, 4, 2], [40, 50]), ([0, 2, 5], [-1, 50]),
                   ([0, 2, 5], [40, 10 ** 9])):
        s.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s.kv_len = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s.run()
        assert L.lora_get_status(s.ws) & A.LORA_DEV_BAD_LENGTH, (cu, kv)


def test_rows_of_no_request_stay_untouched():
    s = Step([2, 3], [40, 50], 4, 2, 64, 16, seed=14)
    s.cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    o, lse = s.run()
    assert torch.isnan(o[4:].float()).all() and torch.isnan(lse[4:]).all()
    assert torch.isfinite(o[:4].float()).all()


def test_offsets_past_32_bits():
    # two pages of interest at the ends of a cache of more than 2^31 elements
    H, Hk, D, page = 2, 1, 128, 16
    num = (1 << 31) // (page * D) + 64
    kc = torch.empty(num, Hk, page, D, dtype=BF, device="cuda")
    vc = torch.empty_like(kc)
    g = torch.Generator().manual_seed(1)
    k = torch.randn(32, Hk, D, generator=g).to(BF)
    v = torch.randn(32, Hk, D, generator=g).to(BF)
    q = torch.randn(1, H, D, generator=g).to(BF)
    table = torch.tensor([[num - 1, 0]], dtype=torch.int32, device="cuda")
    ws = A.AttnWorkspace(32, 1, H, Hk, D)
    slot = torch.cat([(num - 1) * page + torch.arange(16), torch.arange(16)]).to(torch.int32).cuda()
    A.lora_kv_store(k.cuda(), v.cuda(), kc, vc, slot, ws)
    assert torch.equal(kc[num - 1, 0].cpu(), k[:16, 0]) and torch.equal(vc[0, 0].cpu(), v[16:, 0])
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    kv = torch.tensor([32], dtype=torch.int32, device="cuda")
    ws = A.AttnWorkspace(1, 1, H, Hk, D)
    lse = torch.empty(1, H, dtype=torch.float32, device="cuda")
    o = A.lora_attn_paged(q.cuda(), kc, vc, table, cu, kv, 0.1, ws, lse=lse)
    assert L.lora_get_status(ws) == 0
    assert_attn(o, lse, *reference(q.double(), k.double(), v.double(), [32], 0.1))


def test_on_another_stream_and_in_a_graph():
    s = Step([1, 20, 1], [700, 90, 33], 8, 2, 64, 16, seed=15)
    want, lse0 = s.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got, _ = s.run()
    side.synchronize()
    assert torch.equal(got, want)
    got, _ = s.run(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    o, lse = torch.zeros_like(want), torch.zeros_like(lse0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sched = s.schedule()
        for _ in range(3):
            A.lora_attn_paged(s.q, s.k_cache, s.v_cache, s.table, s.cu, s.kv_len, s.scale, s.ws, sched=sched, o=o, lse=lse)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, lse0)


def test_debug_library_agrees():
    s = Step([1, 20, 1], [700, 90, 33], 8, 2, 64, 16, seed=16)
    want, _ = s.run()
    L.use_debug_library(True)
    try:
        got, _ = s.run()
        assert L.lora_get_status(s.ws) == 0
    finally:
        L.use_debug_library(False)
    assert torch.equal(got, want)


# --- prompts -------------------------------------------------------------------

class Prompt:
    def __init__(self, lens, H, Hk, D, seed=0, merged=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.Hk, self.D = lens, H, Hk, D
        T = self.T = sum(lens)
        if merged:
            w = torch.randn(T, (H + 2 * Hk) * D, generator=g).to(BF)
            parts = [w[:, :H * D], w[:, H * D:(H + Hk) * D], w[:, (H + Hk) * D:]]
            self.cpu = [x.reshape(T, -1, D).double() for x in parts]
            wd = w.cuda()
            self.dev = [wd[:, :H * D].unflatten(1, (H, D)), wd[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D)),
                        wd[:, (H + Hk) * D:].unflatten(1, (Hk, D))]
        else:   # head-major tensors: the token stride is the smaller one
            t = [torch.randn(n, T, D, generator=g).to(BF) for n in (H, Hk, Hk)]
            self.cpu = [x.transpose(0, 1).double() for x in t]
            self.dev = [x.cuda().transpose(0, 1) for x in t]
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.scale = 1.0 / math.sqrt(D)
        self.ws = A.AttnWorkspace(T, len(lens), H, Hk, D)

    def run(self, **kw):
        o = torch.full((self.T, self.H, self.D), float("nan"), dtype=BF, device="cuda")
        lse = torch.full((self.T, self.H), float("nan"), dtype=torch.float32, device="cuda")
        A.lora_attn_prompt(*self.dev, self.cu, self.scale, self.ws, o=o, lse=lse, **kw)
        return o, lse

    def reference(self, rows=None):
        parts, t = [], 0
        for n in self.lens:
            q, k, v = (x[t:t + n] for x in self.cpu)
            parts.append(reference(q, k, v, range(1, n + 1), self.scale))
            t += n
        return [torch.cat(x) for x in zip(*parts)]

    def check(self, what="", **kw):
        o, lse = self.run(**kw)
        assert L.lora_get_status(self.ws) == 0, what
        assert_attn(o, lse, *self.reference(), what)


@pytest.mark.parametrize("lens", [[1], [2], [77], [128], [129], [1, 1, 1], [64, 0, 65, 1, 127, 128, 3], [300, 5]])
@pytest.mark.parametrize("H,Hk,D", [(8, 2, 128), (2, 2, 64), (7, 1, 80)])
def test_prompts(lens, H, Hk, D):
    Prompt(lens, H, Hk, D, seed=sum(lens)).check(f"{lens} {H}/{Hk} d{D}")


def test_prompt_head_major_and_one_long():
    Prompt([190, 33], 4, 2, 64, seed=1, merged=False).check("head-major")
    Prompt([700], 2, 1, 128, seed=2).check("700")


def test_prompt_longer_against_fp64_on_the_device():
    # 2500 and 1300 tokens: every block of the schedule, checked whole
    p = Prompt([2500, 1300], 8, 2, 128, seed=3)
    o, lse = p.run()
    assert L.lora_get_status(p.ws) == 0
    t = 0
    for n in p.lens:
        q, k, v = (x[t:t + n].cuda() for x in p.cpu)
        hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        for h in range(p.H):
            s = (q[:, h] @ k[:, h // 4].T * p.scale).masked_fill(hidden, -math.inf)
            w = torch.softmax(s, -1)
            assert_attn(o[t:t + n, h:h + 1], lse[t:t + n, h:h + 1], (w @ v[:, h // 4])[:, None].cpu(),
                        torch.logsumexp(s, -1)[:, None].cpu(), (w @ v[:, h // 4].abs())[:, None].cpu(), f"head {h}")
        t += n


def test_a_neighbour_prompt_full_of_nan_does_not_leak():
    p = Prompt([50, 70, 40], 4, 2, 64, seed=4)
    ref = p.reference()
    for x in p.dev:
        x[50:120] = float("nan")
    o, lse = p.run()
    keep = torch.cat([torch.arange(50), torch.arange(120, 160)])
    assert_attn(o.cpu()[keep], lse.cpu()[keep], *[x[keep] for x in ref])


def test_prompt_and_paged_agree():
    p = Prompt([200], 8, 2, 64, seed=5)
    o1, l1 = p.run()
    page = 16
    num = -(-200 // page)
    kc = torch.zeros(num, 2, page, 64, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    slots = torch.arange(200, dtype=torch.int32, device="cuda")
    A.lora_kv_store(p.dev[1], p.dev[2], kc, vc, slots, p.ws)
    table = torch.arange(num, dtype=torch.int32, device="cuda")[None]
    l2 = torch.empty_like(l1)
    o2 = A.lora_attn_paged(p.dev[0], kc, vc, table, p.cu, torch.tensor([200], dtype=torch.int32, device="cuda"), p.scale,
                           p.ws, lse=l2)
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


# --- plan and store ------------------------------------------------------------

def plan_reference(new, ctx, table, free, head, page, num_pages, T, adapters):
    table = table.clone()
    width = table.shape[1]
    cap, status = width * page, 0
    cu, kv, slot, pos, ids = [0], [], [], [], []
    taken, wanted = 0, 0
    for r in range(len(new)):
        c = min(max(ctx[r], 0), cap)
        n = min(max(new[r], 0), cap - c)
        if (c, n) != (ctx[r], new[r]):
            status |= A.LORA_DEV_BAD_LENGTH
        if cu[-1] + n > T:
            n, status = T - cu[-1], status | A.LORA_DEV_BAD_LENGTH
        need = -(-(c + n) // page) - -(-c // page)
        ok = need == 0 or wanted + need <= len(free) - head
        if ok:
            for j in range(need):
                table[r, -(-c // page) + j] = free[head + wanted + j]
            taken += need
        else:
            status |= A.LORA_DEV_NO_PAGE
        wanted += need
        for p in range(c, c + n):
            pg = int(table[r, p // page]) if ok else -1
            if ok and not 0 <= pg < num_pages:
                status |= A.LORA_DEV_BAD_PAGE
                pg = -1
            slot.append(pg * page + p % page if pg >= 0 else -1)
            pos.append(p)
            ids.append(adapters[r])
        cu.append(cu[-1] + n)
        kv.append(c + n if ok else 0)
    pad = [-1] * (T - len(slot))
    return table, cu, kv, slot + pad, pos + pad, ids + pad, head + taken, status


def check_plan(new, ctx, page, width, free, T, num_pages, head=0, seed=0, table=None):
    g = torch.Generator().manual_seed(seed)
    R = len(new)
    if table is None:
        table = torch.randint(0, num_pages, (R, width), generator=g, dtype=torch.int32)
    adapters = torch.randint(-1, 9, (R,), generator=g, dtype=torch.int32)
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = A.AttnWorkspace(T, R)
    td = table.cuda()
    args = [torch.tensor(new, **i32), torch.tensor(ctx, **i32), td, torch.tensor(free, **i32), torch.tensor([head], **i32)]
    want = plan_reference(new, ctx, table, free, head, page, num_pages, T, adapters.tolist())
    for _ in range(2):   # the same inputs again: the same result
        out = A.lora_kv_plan(*args, page, num_pages, ws, req_adapter=adapters.cuda(), max_tokens=T)
        assert L.lora_get_status(ws) == want[7]
        assert torch.equal(td.cpu(), want[0])
        got = (out.cu_new, out.kv_len, out.slot_map, out.position, out.lora_id_map, out.free_head)
        for name, a, b in zip(("cu", "kv_len", "slot", "position", "ids", "head"), got, (*want[1:6], [want[6]])):
            assert a.cpu().tolist() == list(b), name


@pytest.mark.parametrize("page", [8, 16, 128, 4096])
@pytest.mark.parametrize("R", [1, 3, 255, 256, 257, 1500, 4096])
def test_plan(R, page):
    rng = np.random.RandomState(R + page)
    new = [int(x) for x in rng.randint(0, 20, R)]
    ctx = [int(x) for x in rng.choice([0, 1, page - 1, page, page + 1, 3 * page + 5], R)]
    free = [int(x) for x in rng.permutation(20 * R + 50)[:sum(new) + 7]]
    check_plan(new, ctx, page, 30 // page + 8, free, sum(new) + 5, 20 * R + 50, seed=R)


def test_plan_free_list_runs_short():
    new, ctx = [3, 20, 1, 0, 40, 1, 1], [16, 0, 5, 16, 16, 16, 7]
    for n_free in range(0, 8):
        check_plan(new, ctx, 16, 6, list(range(n_free)), sum(new), 50, seed=n_free)
    check_plan(new, ctx, 16, 6, list(range(9)), sum(new), 50, head=4)


def test_plan_clamps_lengths_and_flags_pages():
    check_plan([5, 9, 4], [0, 100, -3], 16, 3, list(range(30)), 30, 40)          # past the table, negative
    check_plan([-2, 60, 4], [0, 10, 3], 16, 3, list(range(30)), 30, 40)
    check_plan([10, 10, 10], [0, 3, 3], 16, 3, list(range(30)), 14, 40)          # more tokens than there is room for
    check_plan([2, 2], [16, 0], 16, 3, [99, 7, 8], 4, 40)                        # a free page that is none
    t = torch.tensor([[-1, 5, 5], [3, 1, 1]], dtype=torch.int32)
    check_plan([2, 2], [4, 4], 16, 3, [7, 8], 4, 40, table=t)                    # a table entry that is none
    check_plan([0, 0], [4, 4], 16, 3, [], 0, 40)                                 # nothing to do, nothing free


@pytest.mark.parametrize("Hk,D,page", [(8, 128, 16), (1, 8, 8), (3, 80, 64)])
@pytest.mark.parametrize("T", [1, 33, 1000])
def test_store(Hk, D, page, T):
    g = torch.Generator().manual_seed(T)
    num = -(-T // page) + 3
    w = torch.randn(T, 2 * Hk * D + 16, generator=g).to(BF).cuda()
    k, v = w[:, :Hk * D].unflatten(1, (Hk, D)), w[:, Hk * D:2 * Hk * D].unflatten(1, (Hk, D))
    kc = torch.randn(num, Hk, page, D, generator=g).to(BF).cuda()
    vc = torch.randn(num, Hk, page, D, generator=g).to(BF).cuda()
    slot = torch.randperm(num * page, generator=g)[:T].to(torch.int32)
    slot[::5] = -1
    want_k, want_v = kc.clone(), vc.clone()
    for t, s in enumerate(slot.tolist()):
        if s >= 0:
            want_k[s // page, :, s % page] = k[t]
            want_v[s // page, :, s % page] = v[t]
    ws = A.AttnWorkspace(T, 1)
    A.lora_kv_store(k, v, kc, vc, slot.cuda(), ws)
    assert L.lora_get_status(ws) == 0
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    slot[0] = num * page
    A.lora_kv_store(k, v, kc, vc, slot.cuda(), ws)
    assert L.lora_get_status(ws) == A.LORA_DEV_BAD_PAGE
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_store_into_a_token_major_cache():
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(20, 2, 64, generator=g).to(BF).cuda() for _ in range(2))
    kc, vc = (torch.zeros(4, 16, 2, 64, dtype=BF, device="cuda").permute(0, 2, 1, 3) for _ in range(2))
    ws = A.AttnWorkspace(20, 1)
    A.lora_kv_store(k, v, kc, vc, torch.arange(5, 25, dtype=torch.int32, device="cuda"), ws)
    assert torch.equal(kc.permute(0, 2, 1, 3).reshape(64, 2, 64)[5:25], k)
    assert torch.equal(vc.permute(0, 2, 1, 3).reshape(64, 2, 64)[5:25], v)
