"""Attention over the 4-bit cache (include/lora_kv.h) against a plain fp64
implementation over the values that the cache stands for, and the cache
operators in use together.

Tolerance of an output element: o is rounded to bf16 once (u = 2^-8 of it); p is
rounded to fp16 (2^-11) or, for wide requests, to bf16 (u) before the second product,
which moves o by at most that times sum_j p_j |v_j|.  Scores of up to 128 terms
and the sums are fp32: less than 2e-4 of sum_j p_j |v_j| at these magnitudes.  p below
2^-14 of the reference score's lose bits in fp16, 2^-25 absolutely: at most 2^-25 times the
keys' number over the sum of p (at least 1) of max |v|, below 1e-4 of it for 3000 keys.
lse is fp32 throughout: 1e-4."""
import math
import os
import sys

import pytest
import torch

from segmented_gemm_gb300 import attn as A
from segmented_gemm_gb300 import kv as KV
from segmented_gemm_gb300 import lora as L

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import kv_reference as ref  # noqa: E402
from test_gpu_attn import reference  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -8


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def assert_attn4(o, lse, ref_o, ref_lse, mass, vmax, wide, what=""):
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.isfinite(o).all(), f"{what}: non-finite outputs"
    tol = U * ref_o.abs() + ((U if wide else 2.0 ** -11) + 2e-4) * mass + 1e-4 * vmax + 1e-30
    err = (o - ref_o).abs()
    assert (err <= tol).all(), f"{what}: {(err > tol).sum()} of {err.numel()} off, worst {(err / tol).max():.2f} x tol"
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty), f"{what}: empty rows"
    d = (lse - ref_lse)[~empty].abs()
    assert d.numel() == 0 or float(d.max()) <= 1e-4, f"{what}: lse off by {float(d.max()):.2e}"


def near(got, want, vmax):
    """Two results for the same row out of different batches: where groups are cut differs with the batch, so
    they are compared by twice the tolerance (sum_j p_j |v_j| is at most max |v|)."""
    got, want = got.double(), want.double()
    return ((got - want).abs() <= 2 * (U * want.abs() + (2.0 ** -11 + 3e-4) * vmax)).all()


class Step:
    """A step over a 4-bit cache: random pages, random keys and values written by lora_kv4_store, and NaN (scales
    of all ones) in every slot that no request holds."""

    def __init__(self, new, kv, H, Hk, D, page, seed=0, q_pad=0, spare=4, unpack=None, scale_q=1.0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.H, self.Hk, self.D, self.page = new, kv, H, Hk, D, page
        R, T = len(new), sum(new)
        used = [-(-x // page) for x in kv]
        width = max(used + [1]) + 1
        self.num_pages = sum(used) + spare
        perm = torch.randperm(self.num_pages, generator=g).int()
        table = torch.full((R, width), -1, dtype=torch.int32)
        at, slots = 0, []
        for r, n in enumerate(used):
            table[r, :n] = perm[at:at + n]
            at += n
            p = torch.arange(kv[r])
            slots.append(table[r][p // page] * page + p % page)
        self.ws = KV.Kv4Workspace(T, R, H, Hk, D, unpack_tokens=unpack)
        data = torch.full((self.num_pages, Hk, KV.lora_kv4_block_size(page, D)), 255, dtype=torch.uint8, device="cuda")
        self.cache = KV.Kv4Cache(data, page, D)
        n = sum(kv)
        k, v = (torch.randn(n, Hk, D, generator=g).to(BF).cuda() for _ in range(2))
        slots = torch.cat(slots).int().cuda()
        KV.lora_kv4_store(k, v, self.cache, slots, self.ws)
        k, v = (x.double().cpu() for x in KV.lora_kv4_load(self.cache, slots, self.ws))
        self.keys, self.values = list(k.split(kv)), list(v.split(kv))
        self.table = table.cuda()
        wide = (scale_q * torch.randn(T, H * D + q_pad, generator=g)).to(BF)
        self.q_cpu = wide[:, :H * D].reshape(T, H, D).double()
        self.q = wide.cuda()[:, :H * D].unflatten(1, (H, D))
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        self.T, self.R = T, R
        self.cu, self.kv_len = i32(cu), i32(kv)
        self.scale = 1.0 / math.sqrt(D) / scale_q
        rows = 160 if D <= 64 else 96
        self.any_wide = self.ws.unpack_tokens > 0 and T * H >= 6400 and any(x * H // Hk > rows for x in new)

    def run(self):
        o = torch.full((self.T, self.H, self.D), float("nan"), dtype=BF, device="cuda")
        lse = torch.full((self.T, self.H), float("nan"), dtype=torch.float32, device="cuda")
        KV.lora_kv4_attn(self.q, self.cache, self.table, self.cu, self.kv_len, self.scale, self.ws, o=o, lse=lse)
        return o, lse

    def reference(self):
        parts, t = [], 0
        for n, length, k, v in zip(self.new, self.kv, self.keys, self.values):
            lim = [max(0, length - n + i + 1) for i in range(n)]
            parts.append(reference(self.q_cpu[t:t + n], k, v, lim, self.scale))
            t += n
        return [torch.cat(x) for x in zip(*parts)]

    def check(self, what=""):
        o, lse = self.run()
        assert L.lora_get_status(self.ws) == 0, what
        vmax = max([float(v.abs().max()) for v in self.values if v.numel()] + [0.0])
        assert_attn4(o, lse, *self.reference(), vmax, self.any_wide, what)
        again, lse2 = self.run()      # the same bits, whatever the timing
        assert torch.equal(again, o) and torch.equal(lse2, lse)
        return o, lse


@pytest.mark.parametrize("H,Hk,D,page", [(8, 2, 128, 16), (4, 4, 64, 32), (7, 1, 128, 64), (16, 1, 80, 16),
                                         (10, 2, 8, 16), (6, 2, 40, 128), (4, 1, 120, 256), (1, 1, 128, 16),
                                         (12, 4, 72, 4096), (128, 1, 64, 16), (20, 2, 64, 16)])
def test_single_tokens(H, Hk, D, page):
    Step([1] * 10, [1, 2, 15, 16, 17, 127, 128, 129, 700, 33], H, Hk, D, page, seed=H + D).check(f"{H}/{Hk} d{D} p{page}")


@pytest.mark.parametrize("unpack", [0, None, 512])   # never, all, only the first ones fit
@pytest.mark.parametrize("H,Hk,D,page", [(8, 2, 128, 16), (14, 2, 64, 32), (3, 3, 96, 64),
                                         (16, 4, 128, 16), (32, 2, 64, 32), (18, 3, 96, 64)])   # these have wide requests
def test_chunks_and_single_tokens_mixed(H, Hk, D, page, unpack):
    new, kv = [1, 200, 0, 5, 33, 1, 130, 2, 64], [300, 450, 77, 5, 33, 1, 600, 129, 64]
    Step(new, kv, H, Hk, D, page, seed=H, unpack=unpack, q_pad=16).check(f"{H}/{Hk} d{D} unpack {unpack}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk", [(12, 3), (80, 20)])
@pytest.mark.parametrize("n", [2, 3, 8, 9, 24, 25, 41])
def test_a_few_tokens_a_request(n, H, Hk, D):
    # around the most rows that a request may have and not be wide, and blocks that end inside a token's heads
    Step([n, 1, n, 0, n], [n, 90, 400, 20, n + 130], H, Hk, D, 16, seed=n).check(f"{n} tokens")


def test_rows_that_see_nothing():
    # more new tokens than keys, none at all, and a request that got no pages
    for H, Hk in ((4, 2), (64, 4)):
        s = Step([5, 3, 1, 4, 120], [2, 0, 0, 4, 7], H, Hk, 128, 16, seed=3)
        o, lse = s.check()
        assert (o[:3] == 0).all() and torch.isinf(lse[:3]).all() and (o[5:9] == 0).all()
        assert s.any_wide == (H == 64)
    s = Step([5, 3, 1, 4, 120], [2, 0, 0, 4, 7], 4, 2, 128, 16, seed=3, unpack=0)
    s.check()


@pytest.mark.parametrize("R,page", [(257, 16), (1000, 16), (4096, 16)])
def test_many_requests(R, page):
    g = torch.Generator().manual_seed(R)
    new = torch.randint(0, 2, (R,), generator=g).tolist()
    kv = [int(x) if n else int(x) // 2 for n, x in zip(new, torch.randint(1, 40, (R,), generator=g))]
    Step(new, kv, 4, 2, 64, page, seed=R).check()


def test_one_long_request():
    # a single group of few rows over all CTAs, pieces of one joined over the whole GPU
    Step([1], [3000], 2, 1, 128, 16, seed=1).check()
    Step([2], [3000], 8, 2, 64, 16, seed=2).check()


def test_queries_of_any_size():
    # a row's queries are scaled by a power of two into fp16 on the way
    for e in (1e-30, 1e-3, 1e4, 1e25):
        Step([1, 2, 1], [40, 130, 17], 8, 2, 128, 16, seed=5, scale_q=e).check(f"queries of {e}")
    s = Step([1, 2, 1], [40, 130, 17], 8, 2, 64, 16, seed=5)
    s.q[1, 3] = 0
    s.q_cpu[1, 3] = 0
    s.check("a row of zeros")


@pytest.mark.parametrize("H,unpack", [(8, 0), (8, None), (128, None)])
def test_nans_and_infinities_stay_in_their_rows(H, unpack):
    s = Step([3, 1, 60], [90, 40, 200], H, max(2, H // 8), 128, 16, seed=9, unpack=unpack)
    assert s.any_wide == (H == 128)
    want, _ = s.run()
    s.q[1, 5, 7] = float("nan")
    s.q[3, 0, 0] = float("inf")
    got, _ = s.run()
    assert L.lora_get_status(s.ws) == 0
    assert got[1, 5].isnan().all() and not torch.equal(got[3, 0], want[3, 0])
    for t, h in ((1, 5), (3, 0)):
        got[t, h] = want[t, h]
    assert torch.equal(got, want)


def test_rows_of_no_request_and_lengths_out_of_range():
    for H, unpack in ((8, 0), (8, None), (128, None)):
        s = Step([1, 60, 2], [50, 90, 20], H, max(2, H // 8), 128, 16, seed=2, unpack=unpack)
        o = torch.full((s.T, H, 128), 3.0, dtype=BF, device="cuda")
        want, _ = s.run()
        s.cu[3], s.cu[0] = s.T - 2, 1          # the first row and the last two belong to nobody now
        KV.lora_kv4_attn(s.q, s.cache, s.table, s.cu, s.kv_len, s.scale, s.ws, o=o)
        assert L.lora_get_status(s.ws) == 0
        assert (o[0] == 3).all() and (o[-2:] == 3).all()
        assert near(o[1:61], want[1:61], 6.0)
    s = Step([1, 1], [50, 20], 4, 2, 64, 16, seed=2)
    want, _ = s.run()
    s.kv_len[0] = 10 ** 6                      # clamped to the table's row, whose last entry is -1: a page of zeros
    s.cu[2] = 7
    o, _ = s.run()
    assert L.lora_get_status(s.ws) == A.LORA_DEV_BAD_LENGTH | A.LORA_DEV_BAD_PAGE
    assert near(o[1], want[1], 6.0)            # (row 0 sees the unwritten slots of its last page, NaN here)
    s.kv_len[0] = -5
    o, lse = s.run()
    assert L.lora_get_status(s.ws) == A.LORA_DEV_BAD_LENGTH
    assert (o[0] == 0).all() and torch.isinf(lse[0]).all() and near(o[1], want[1], 6.0)


@pytest.mark.parametrize("H,unpack", [(8, 0), (8, None), (128, None)])
def test_pages_outside_the_cache_read_as_zeros(H, unpack):
    s = Step([1, 64], [60, 130], H, max(2, H // 8), 128, 16, seed=4, unpack=unpack)
    for r, j, page in ((0, 1, s.num_pages), (1, 3, -1), (1, 8, 1 << 30)):
        s.table[r, j] = page
        s.keys[r][16 * j:16 * j + 16] = 0
        s.values[r][16 * j:16 * j + 16] = 0
    o, lse = s.run()
    assert L.lora_get_status(s.ws) == A.LORA_DEV_BAD_PAGE
    vmax = max(float(v.abs().max()) for v in s.values)
    assert_attn4(o, lse, *s.reference(), vmax, s.any_wide)


@pytest.mark.parametrize("H", [8, 96])
def test_strides_streams_and_captured_calls(H):
    s = Step([1, 70, 1], [500, 300, 9], H, max(2, H // 8), 64, 32, seed=6, q_pad=64)
    assert s.any_wide == (H == 96)
    want, lse0 = s.run()
    # o as rows of a wider tensor, heads apart; the table's rows apart; another stream
    o = torch.full((s.T, H, 3, 64), 2.0, dtype=BF, device="cuda")
    table = torch.full((3, s.table.shape[1] + 5), 12345, dtype=torch.int32, device="cuda")
    table[:, :s.table.shape[1]] = s.table
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    KV.lora_kv4_attn(s.q, s.cache, table[:, :s.table.shape[1]], s.cu, s.kv_len, s.scale, s.ws, o=o[:, :, 1], stream=stream)
    stream.synchronize()
    assert torch.equal(o[:, :, 1], want) and (o[:, :, 0] == 2).all() and (o[:, :, 2] == 2).all()
    # two captured graphs over one workspace, replayed in turn
    t = Step([1, 2], [90, 700], H, max(2, H // 8), 64, 32, seed=7)
    t.ws = s.ws
    want_t, _ = t.run()
    out = [torch.empty_like(want), torch.empty_like(want_t)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, x, y in zip(graphs, (s, t), out):
        with torch.cuda.graph(g):
            KV.lora_kv4_attn(x.q, x.cache, x.table, x.cu, x.kv_len, x.scale, s.ws, o=y)
    for _ in range(5):
        for y in out:
            y.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want) and torch.equal(out[1], want_t)
    # the lengths of a captured call are read at each replay
    s.kv_len[0] = 17
    graphs[0].replay()
    o2, _ = s.run()
    assert torch.equal(out[0], o2) and not torch.equal(o2[0], want[0]) and near(o2[1:], want[1:], 6.0)
    assert L.lora_get_status(s.ws) == 0


def test_a_cache_past_32_bit_offsets():
    # 5 GB: page numbers whose bytes lie past 2^32
    Hk, D, page = 8, 128, 64
    block = KV.lora_kv4_block_size(page, D)
    pages = (5 << 30) // (Hk * block)
    cache = KV.Kv4Cache(torch.empty(pages, Hk, block, dtype=torch.uint8, device="cuda"), page, D)
    g = torch.Generator().manual_seed(1)
    n = 150
    table = torch.tensor([[pages - 1, 2, pages - 2], [pages // 2, pages - 3, 0]], dtype=torch.int32)
    k, v = (torch.randn(2 * n, Hk, D, generator=g).to(BF) for _ in range(2))
    pos = torch.arange(n)
    slots = torch.cat([table[r][pos // page] * page + pos % page for r in range(2)]).int().cuda()
    ws = KV.Kv4Workspace(2, 2, 16, Hk, D)
    KV.lora_kv4_store(k.cuda(), v.cuda(), cache, slots, ws)
    k, v = (x.double().cpu() for x in KV.lora_kv4_load(cache, slots, ws))
    q = torch.randn(2, 16, D, generator=g).to(BF)
    lse = torch.empty(2, 16, device="cuda")
    o = KV.lora_kv4_attn(q.cuda(), cache, table.cuda(), i32([0, 1, 2]), i32([n, n]), 0.1, ws, lse=lse)
    assert L.lora_get_status(ws) == 0
    parts = [reference(q[r:r + 1].double(), k[r * n:r * n + n], v[r * n:r * n + n], [n], 0.1) for r in range(2)]
    assert_attn4(o, lse, *[torch.cat(x) for x in zip(*parts)], float(v.abs().max()), False)


@pytest.mark.parametrize("budget", [100, 3000])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(budget):
    s = Step([1] * 20 + [300, 7], [2000 - 90 * i for i in range(20)] + [900, 40], 32, 8, 128, 16, seed=5)
    want, _ = s.run()
    statuses = []
    L.lora_set_wait_budget(budget)
    try:
        for _ in range(3):
            s.run()
            statuses.append(L.lora_get_status(s.ws))
    finally:
        L.lora_set_wait_budget(0)
    assert all(x in (0, L.LORA_DEV_TIMEOUT) for x in statuses), statuses
    o, _ = s.run()
    assert L.lora_get_status(s.ws) == 0 and torch.equal(o, want)


def test_workspace_of_a_large_step_serves_smaller_ones():
    ws = KV.Kv4Workspace(600, 40, 16, 4, 128, unpack_tokens=2048)
    for new, kv in (([1] * 40, list(range(1, 41))), ([600], [700]), ([1, 64], [9, 300]), ([3], [3]), ([200, 200], [200, 900])):
        s = Step(new, kv, 16, 4, 128, 16, seed=len(new), unpack=2048)
        s.ws = ws
        s.check(str(new))
    for kw in (dict(o=torch.empty(1, 8, 64, dtype=BF, device="cuda")), dict(lse=torch.empty(3, 8, device="cuda"))):
        with pytest.raises(ValueError):
            KV.lora_kv4_attn(s.q, s.cache, s.table, s.cu, s.kv_len, s.scale, ws, **kw)
    with pytest.raises(L.LoraError):
        KV.lora_kv4_attn(s.q, s.cache, s.table, s.cu, s.kv_len, -1.0, ws)
    with pytest.raises(L.LoraError):   # a workspace made for a smaller step
        small = KV.Kv4Workspace(1, 1, 8, 2, 128)
        small.unpack_tokens = 2048
        KV.lora_kv4_attn(s.q, s.cache, s.table, s.cu, s.kv_len, s.scale, small)


@pytest.mark.parametrize("H", [8, 128])
def test_debug_library_gives_the_same(H):
    s = Step([1, 60, 2], [300, 90, 20], H, max(2, H // 8), 128, 16, seed=12)
    assert s.any_wide == (H == 128)
    want, _ = s.run()
    L.use_debug_library(True)
    try:
        got, _ = s.run()
        assert L.lora_get_status(s.ws) == 0
    finally:
        L.use_debug_library(False)
    assert torch.equal(got, want)


@pytest.mark.parametrize("bits", [16, 4])
def test_the_operators_in_use(bits):
    """Steps of a served layer: plan, rotation (into the cache, or to rows and then the 4-bit cache), attention;
    between steps rows are dropped, forked and the cache compacted.  At each step the attention is compared with fp64
    over every row's whole history, as it went into the cache."""
    H, Hk, D, page, R, width, pages = 8, 2, 128, 16, 6, 12, 60
    g = torch.Generator().manual_seed(bits)
    ws, wsp = KV.Kv4Workspace(400, R, H, Hk, D), KV.PagesWorkspace(pages)
    aws = A.AttnWorkspace(400, R, H, Hk, D)
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    free, head = torch.randperm(pages, generator=g).int().cuda(), i32([0])
    ctx, counts = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    inv = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float()
    wq, wk = ((1 + 0.1 * torch.randn(D, generator=g)).to(BF) for _ in range(2))
    cache4 = KV.Kv4Cache.zeros(pages, Hk, page, D)
    kc, vc = (torch.zeros(pages, Hk, page, D, dtype=BF, device="cuda") for _ in range(2))
    history = [[] for _ in range(R)]        # each row's (key, value) as stored, fp64
    books = dict(ctx_len=ctx, block_table=table, ref=counts, free_pages=free, page_size=page, ws=wsp)
    scale = D ** -0.5
    for step, new in enumerate([[40, 17, 0, 33, 64, 1], [1] * 6, [1, 2, 60, 1, 0, 1], [1] * 6, [3, 1, 1, 1, 1, 0], [1] * 6]):
        T = sum(new)
        plan = A.lora_kv_plan(i32(new), ctx, table, free, head, page, pages, aws, max_tokens=T + 3)
        head = plan.free_head
        qkv = torch.randn(T + 3, (H + 2 * Hk) * D, generator=g).to(BF)
        heads = qkv.cuda().unflatten(1, (H + 2 * Hk, D))
        q, k, v = heads[:, :H], heads[:, H:H + Hk], heads[:, H + Hk:]
        # the plan's positions of -1 behind the last token: those rows are passed over
        args = dict(q_weight=wq.cuda(), k_weight=wk.cuda())
        q_out = torch.full((T + 3, H, D), 7.0, dtype=BF, device="cuda")
        k_out = torch.full((T + 3, Hk, D), 7.0, dtype=BF, device="cuda")
        if bits == 16:
            KV.lora_qk_rope(q, k, plan.position, inv.cuda(), ws, v=v, k_cache=kc, v_cache=vc, slot_map=plan.slot_map,
                            q_out=q_out, k_out=k_out, **args)
        else:
            KV.lora_qk_rope(q, k, plan.position, inv.cuda(), ws, q_out=q_out, k_out=k_out, **args)
            KV.lora_kv4_store(k_out, v, cache4, plan.slot_map, ws)
        assert (q_out[T:] == 7).all() and (k_out[T:] == 7).all()
        pos = plan.position[:T].cpu()
        y, size = ref.rope(qkv[:T, :H * D].unflatten(1, (H, D)), wq, 1e-6, pos, inv, False)
        assert ((q_out[:T].double().cpu() - y).abs() <= U * y.abs() + 2e-6 * size).all()
        y, size = ref.rope(qkv[:T, H * D:(H + Hk) * D].unflatten(1, (Hk, D)), wk, 1e-6, pos, inv, False)
        assert ((k_out[:T].double().cpu() - y).abs() <= U * y.abs() + 2e-6 * size).all()
        lse = torch.empty(T, H, device="cuda")
        if bits == 16:
            o = A.lora_attn_paged(q_out[:T], kc, vc, table, plan.cu_new, plan.kv_len, scale, aws, lse=lse)
        else:
            o = KV.lora_kv4_attn(q_out[:T], cache4, table, plan.cu_new, plan.kv_len, scale, ws, lse=lse)
        ks, vs = k_out[:T].cpu(), v[:T].cpu()
        if bits == 4:
            ks, vs = (ref.dequantise(*ref.quantise(x))[..., :D] for x in (ks, vs))
        at, parts = 0, []
        for r, n in enumerate(new):
            history[r] += [(ks[t].double(), vs[t].double()) for t in range(at, at + n)]
            if n:
                keys, values = (torch.stack(x) for x in zip(*history[r]))
                lim = [len(history[r]) - n + i + 1 for i in range(n)]
                parts.append(reference(q_out[at:at + n].double().cpu(), keys, values, lim, scale))
            at += n
        assert_attn4(o, lse, *[torch.cat(x) for x in zip(*parts)], float(vs.abs().max()), True, f"step {step}")
        ctx.copy_(plan.kv_len)
        # two rows are dropped and continue others; then the cache is cut
        drop = [(2 * step) % R, (2 * step + 1) % R]
        parents = [(drop[1] + 1) % R] * 2
        KV.lora_kv_release(i32(drop), free_head=head, **books)
        src, dst = KV.lora_kv_fork(i32(parents), i32(drop), free_head=head, **books)
        for a, b in zip(parents, drop):
            history[b] = list(history[a])
        for _ in range(2):
            if bits == 16:
                KV.lora_kv_copy(src, dst, kc, vc, wsp)
            else:
                KV.lora_kv4_copy(src, dst, cache4, wsp)
            src, dst = KV.lora_kv_compact(free_head=head, limit=40 + 3 * (step % 3), **books)
        if bits == 16:
            KV.lora_kv_copy(src, dst, kc, vc, wsp)
        else:
            KV.lora_kv4_copy(src, dst, cache4, wsp)
        assert ctx.tolist() == [len(h) for h in history]
        assert L.lora_get_status(ws) == 0 and L.lora_get_status(wsp) == 0 and L.lora_get_status(aws) == 0


@pytest.mark.parametrize("cfg", [dict(rope=True), dict(bits=4), dict(rope=True, bits=4, head_dim=128, kv_heads=1, page=32)])
def test_serving_example_runs_with_the_cache_operators(cfg):
    from test_gpu_attn_serving import _example
    status, errors = _example().serve(requests=4, layers=1, steps=5, **cfg)
    assert status == 0 and all(math.isfinite(e) for e in errors)


def test_rows_that_start_on_16_bytes_only():
    # the cache's writes and reads take 32 bytes at once where they can
    wide = torch.randn(20, 2, 3 * 64 + 8, device="cuda").to(BF)
    a, b = KV.Kv4Cache.zeros(2, 2, 16, 64), KV.Kv4Cache.zeros(2, 2, 16, 64)
    ws, slots = A.AttnWorkspace(1, 1), torch.arange(20, dtype=torch.int32, device="cuda")
    k, v = wide[..., 8:72], wide[..., 72:136]
    KV.lora_kv4_store(k, v, a, slots, ws)
    KV.lora_kv4_store(k.contiguous(), v.contiguous(), b, slots, ws)
    assert torch.equal(a.data, b.data)
    out = torch.full_like(wide, 3.0)
    KV.lora_kv4_load(a, slots, ws, k=out[..., 8:72], v=out[..., 136:200])
    k1, v1 = KV.lora_kv4_load(a, slots, ws)
    assert torch.equal(out[..., 8:72], k1) and torch.equal(out[..., 136:200], v1)
    assert (out[..., :8] == 3).all() and (out[..., 72:136] == 3).all()


def test_many_small_weights_beside_a_large_one():
    """2^20 keys whose weights are 2^-25.5 of the first one's: together 2 % of it, each below what fp16 has beside 1.
    Pages repeat, and there are enough groups that a warp has most of one.  With n = 2^16 tiles, adding equal numbers
    in fp32 loses up to n / 2 * 2^-23 of o (truncated in a product) and as much of l; o itself is rounded by U, p by 2^-11,
    and x = 25.5 by 2^-22 of itself.  l is summed by lanes, an eighth of the keys each; in the one that has the
    first key, its 1 absorbs what is added one by one: 2^-25.5 is below half of fp32's last place there, 2^-24."""
    R, Hk, D, page, N = 320, 8, 128, 4096, 1 << 20
    k = torch.zeros(2 * page, Hk, D, dtype=BF, device="cuda")
    v = torch.full_like(k, 6.0)              # a scale of 1: exact
    k[0, :, 0], v[0] = 6.0, 0.0
    cache = KV.Kv4Cache.zeros(2, Hk, page, D)
    ws = KV.Kv4Workspace(R, R, Hk, Hk, D)
    KV.lora_kv4_store(k, v, cache, torch.arange(2 * page, dtype=torch.int32, device="cuda"), ws)
    table = torch.ones(R, N // page, dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    q = torch.zeros(R, Hk, D, dtype=BF, device="cuda")
    q[..., 0] = 2.0
    lse = torch.empty(R, Hk, device="cuda")
    o = KV.lora_kv4_attn(q, cache, table, i32(list(range(R + 1))), i32([N] * R), 25.5 / 12 * math.log(2.0), ws, lse=lse)
    rest = (N - 1) * 2.0 ** -25.5
    want = 6.0 * rest / (1.0 + rest)
    tol = (U + 2.0 ** -11 + 2 * 2.0 ** 15 * 2.0 ** -23 + 2.0 ** -16) * want
    assert float((o.double() - want).abs().max()) <= tol
    want = 25.5 * math.log(2.0) + math.log1p(rest)
    assert float((lse.double() - want).abs().max()) <= rest / 8 + 2 * 2.0 ** -8 * rest + 25 * 2.0 ** -22
