"""Rotation, the 4-bit cache's writes and reads, and the calls on pages
(include/lora_kv.h) against plain implementations in 64 bits.

Rotation: fp32 arithmetic, one rounding to bf16 (half a step, 2^-8 of the
value).  Before it, an angle's fp32 form is off by 2^-25 turns (2e-7), cosine and sine
by 2^-23, norm, weight and products by a few 2^-24: 2e-6 of the operands covers
them.  Everything else is exact: codes, scales and copies are compared bit by bit."""
import os
import random
import sys

import pytest
import torch

from segmented_gemm_gb300 import attn as A
from segmented_gemm_gb300 import kv as KV
from segmented_gemm_gb300 import lora as L

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import kv_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -8


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def ws():
    return A.AttnWorkspace(1, 1)


# --- rotation ----------------------------------------------------------------

def rope_inputs(T, H, Hk, D, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(T, (H + 2 * Hk) * D + pad, generator=g).to(BF)
    cut = lambda x: (x[:, :H * D].unflatten(1, (H, D)), x[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D)),  # noqa: E731
                     x[:, (H + Hk) * D:(H + 2 * Hk) * D].unflatten(1, (Hk, D)))
    weights = [(1 + 0.3 * torch.randn(D, generator=g)).to(BF) for _ in range(2)]
    return cut(wide), cut(wide.cuda()), weights


def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float() if rot else None


def assert_rope(got, x, w, position, inv, interleaved, eps=1e-6, rows=None):
    y, size = ref.rope(x, w, eps, position, inv, interleaved)
    got = got.double().cpu()
    if rows is not None:
        y, size, got = y[rows], size[rows], got[rows]
    err, tol = (got - y).abs(), U * y.abs() + 2e-6 * size + 1e-30
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.numel()} off, worst {(err / tol).max():.2f} x tol"


@pytest.mark.parametrize("T", [1, 3, 37, 304, 305, 650])
@pytest.mark.parametrize("H,Hk,D,rot,inter,norms", [
    (32, 8, 128, 128, False, "qk"), (4, 1, 64, 64, True, "qk"), (7, 1, 80, 40, False, ""), (6, 2, 96, 96, True, "q"),
    (5, 5, 72, 8, False, "k"), (3, 3, 8, 8, False, "qk"), (2, 1, 40, 0, False, "qk"), (16, 2, 120, 64, True, ""),
])
def test_rotation_to_rows(ws, T, H, Hk, D, rot, inter, norms):
    (q, k, _), (qd, kd, _), (wq, wk) = rope_inputs(T, H, Hk, D, T + D, pad=8)
    g = torch.Generator().manual_seed(T)
    position = torch.randint(0, 100000, (T,), generator=g)
    inv = freqs(rot)
    wq, wk = wq if "q" in norms else None, wk if "k" in norms else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    qo, ko = KV.lora_qk_rope(qd, kd, i32(position.tolist()), dev(inv), ws, dev(wq), dev(wk), interleaved=inter)
    assert L.lora_get_status(ws) == 0
    assert_rope(qo, q, wq, position, inv, inter)
    assert_rope(ko, k, wk, position, inv, inter)
    # in place: the same bits
    q2, k2 = KV.lora_qk_rope(qd, kd, i32(position.tolist()), dev(inv), ws, dev(wq), dev(wk), interleaved=inter, q_out=qd,
                             k_out=kd)
    assert q2 is qd and torch.equal(qd, qo) and torch.equal(kd, ko)


@pytest.mark.parametrize("per_sm,more", [(3, 0), (3, 1), (48, -1), (48, 5), (96, 3)])
def test_rotation_around_the_splits(ws, per_sm, more):
    """Numbers of tokens around which the tokens of a CTA change, and where the last CTA has few."""
    T = per_sm * torch.cuda.get_device_properties(0).multi_processor_count + more
    (q, k, _), (qd, kd, _), (wq, wk) = rope_inputs(T, 3, 1, 24, per_sm)
    position = torch.randint(0, 100000, (T,), generator=torch.Generator().manual_seed(T))
    position[-2] = -1
    qo, ko = torch.full_like(qd, 5.0), torch.full_like(kd, 5.0)
    KV.lora_qk_rope(qd, kd, i32(position.tolist()), freqs(16).cuda(), ws, wq.cuda(), wk.cuda(), q_out=qo, k_out=ko)
    on = position >= 0
    assert_rope(qo, q, wq, position, freqs(16), False, rows=on)
    assert_rope(ko, k, wk, position, freqs(16), False, rows=on)
    assert (qo[-2] == 5).all() and (ko[-2] == 5).all()


@pytest.mark.parametrize("order", ["phsd", "pshd"])
@pytest.mark.parametrize("T,H,Hk,D,page,k_rows", [(1, 8, 2, 128, 16, False), (50, 4, 4, 64, 8, True),
                                                  (700, 6, 2, 80, 64, False)])
def test_rotation_into_the_cache(ws, order, T, H, Hk, D, page, k_rows):
    (q, k, v), (qd, kd, vd), (wq, wk) = rope_inputs(T, H, Hk, D, 7 * T)
    pages = -(-T // page) + 2
    g = torch.Generator().manual_seed(T)
    slot = torch.randperm(pages * page, generator=g)[:T].int()
    position = torch.randint(0, 5000, (T,), generator=g).int()
    slot[T // 2:T // 2 + 1] = -1 if T > 1 else slot[0]      # one that is not stored, but rotated
    if T > 10:
        position[3] = -1                                    # one that is passed over
    shape = dict(zip("phsd", (pages, Hk, page, D)))
    axes = [order.index(c) for c in "phsd"]
    kc = torch.full([shape[c] for c in order], 9.0, dtype=BF, device="cuda").permute(axes)
    vc = torch.full([shape[c] for c in order], 9.0, dtype=BF, device="cuda").permute(axes)
    q_out = torch.full((T, H, D), 5.0, dtype=BF, device="cuda")
    k_out = torch.full((T, Hk, D), 5.0, dtype=BF, device="cuda") if k_rows else None
    KV.lora_qk_rope(qd, kd, position.cuda(), freqs(D).cuda(), ws, wq.cuda(), wk.cuda(), eps=1e-5, v=vd, k_cache=kc,
                    v_cache=vc, slot_map=slot.cuda(), q_out=q_out, k_out=k_out)
    assert L.lora_get_status(ws) == 0
    on = position >= 0
    assert_rope(q_out, q, wq, position, freqs(D), False, 1e-5, rows=on)
    assert (q_out.cpu()[~on] == 5).all()
    if k_rows:
        assert_rope(k_out, k, wk, position, freqs(D), False, 1e-5, rows=on)
        assert (k_out.cpu()[~on] == 5).all()
    flat_k, flat_v = (c.cpu().transpose(1, 2).reshape(pages * page, Hk, D) for c in (kc, vc))
    stored = on & (slot >= 0)
    at = slot[stored].long()
    got = torch.zeros(T, Hk, D, dtype=BF)
    got[stored] = flat_k[at]
    assert_rope(got, k, wk, position, freqs(D), False, 1e-5, rows=stored)
    assert torch.equal(flat_v[at], v[stored])
    left = torch.ones(pages * page, dtype=torch.bool)
    left[at] = False
    assert (flat_k[left] == 9).all() and (flat_v[left] == 9).all()


def test_far_positions_and_odd_frequencies(ws):
    # positions to the last 31-bit one: the angle is exact modulo a turn, where fp32 products would be off by turns
    position = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 31 - 1, 10 ** 9 + 7, 999999937])
    inv = torch.tensor([1.0, -0.3, 6.25, 1e-7, 1e-38, 1e-45, 0.0, 123.456], dtype=torch.float32)
    T = position.numel()
    (q, k, _), (qd, kd, _), _ = rope_inputs(T, 3, 1, 16, 3)
    qo, ko = KV.lora_qk_rope(qd, kd, i32(position.tolist()), inv.cuda(), ws)
    # the reference in exact integers: fp64 products of 2^31 and these frequencies keep 2^-22 turns at least
    from fractions import Fraction
    from math import floor
    two_pi = Fraction(628318530717958647692528676655900576839433879875021, 10 ** 50)
    turn = torch.tensor([[float((Fraction(float(f)) / two_pi * int(p)) - floor(Fraction(float(f)) / two_pi * int(p)))
                          for f in inv] for p in position], dtype=torch.float64) * 2 * torch.pi
    for x, got in ((q, qo), (k, ko)):
        x = x.double()
        a, b = x[..., :8], x[..., 8:]
        c, s = torch.cos(turn)[:, None], torch.sin(turn)[:, None]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
        size = torch.cat([a.abs() + b.abs()] * 2, -1)
        assert ((got.double().cpu() - y).abs() <= U * y.abs() + 2e-6 * size).all()


def test_a_row_of_nans_or_zeros_stays_alone(ws):
    (q, k, _), (qd, kd, _), (wq, wk) = rope_inputs(40, 4, 2, 64, 1)
    want, _ = KV.lora_qk_rope(qd, kd, i32(list(range(40))), freqs(64).cuda(), ws, wq.cuda(), wk.cuda())
    qd[7, 2] = float("nan")
    qd[9, 1] = 0
    qd[11, 0, 3] = float("inf")
    got, _ = KV.lora_qk_rope(qd, kd, i32(list(range(40))), freqs(64).cuda(), ws, wq.cuda(), wk.cuda())
    assert got[7, 2].isnan().all() and (got[9, 1] == 0).all() and got[11, 0].isnan().any()
    for t, h in ((7, 2), (9, 1), (11, 0)):
        got[t, h] = want[t, h]
    assert torch.equal(got, want)


def test_infinities_beside_what_is_rotated(ws):
    # elements that are not rotated keep their own, and pairs that are do not reach beyond themselves
    for D, rot, inter in ((128, 64, False), (128, 64, True), (64, 0, False), (80, 40, False)):
        (_, _, _), (q, k, _), _ = rope_inputs(5, 2, 1, D, 4)
        pos, inv = i32([0, 3, 5, 70, 1000]), None if rot == 0 else freqs(rot).cuda()
        want, _ = KV.lora_qk_rope(q, k, pos, inv, ws, interleaved=inter)
        q[1, 0, D - 1], q[2, 1, D - 8], q[3, 1, rot] = float("inf"), -float("inf"), float("nan")
        got, _ = KV.lora_qk_rope(q, k, pos, inv, ws, interleaved=inter)
        for t, h, d in ((1, 0, D - 1), (2, 1, D - 8), (3, 1, rot)):
            assert torch.equal(got[t, h, d].isnan(), q[t, h, d].isnan()) and (got[t, h, d].isnan() or got[t, h, d] == q[t, h, d])
            got[t, h, d] = want[t, h, d]
        assert torch.equal(got, want)


def test_slots_outside_the_cache_are_reported(ws):
    (_, _, _), (q, k, v), _ = rope_inputs(6, 2, 1, 64, 2)
    kc, vc = (torch.zeros(2, 1, 16, 64, dtype=BF, device="cuda") for _ in range(2))
    KV.lora_qk_rope(q, k, i32([0, 1, 2, 3, 4, -1]), None, ws, v=v, k_cache=kc, v_cache=vc, slot_map=i32([5, 32, -7, -1, 31, 99]))
    assert L.lora_get_status(ws) == A.LORA_DEV_BAD_PAGE
    assert torch.equal(kc[0, 0, 5], k[0, 0]) and torch.equal(vc[1, 0, 15], v[4, 0])
    assert int((kc != 0).any(-1).sum()) == 2
    # a bad slot of a token that is passed over is nobody's fault
    KV.lora_qk_rope(q, k, i32([-1] * 6), None, ws, v=v, k_cache=kc, v_cache=vc, slot_map=i32([99] * 6))
    assert L.lora_get_status(ws) == 0


def test_binding_of_the_rotation_refuses_what_does_not_fit(ws):
    (_, _, _), (q, k, v), (wq, _) = rope_inputs(4, 2, 1, 64, 2)
    pos, cache = i32([0, 1, 2, 3]), torch.zeros(2, 1, 16, 64, dtype=BF, device="cuda")
    for kw in (dict(k_cache=cache), dict(k_cache=cache, v_cache=cache, v=v), dict(q_weight=wq.float().cuda()),
               dict(q_weight=wq[:32].cuda()), dict(q_out=q[:, :1]), dict(k_out=v[:2]),
               dict(k_cache=cache[..., :32], v_cache=cache[..., :32], v=v, slot_map=pos)):
        with pytest.raises(ValueError):
            KV.lora_qk_rope(q, k, pos, None, ws, **kw)
    with pytest.raises(ValueError):
        KV.lora_qk_rope(q, k[:3], pos, None, ws)
    with pytest.raises(ValueError):
        KV.lora_qk_rope(q, k, pos[:2], None, ws)
    with pytest.raises(ValueError):
        KV.lora_qk_rope(q, k, pos, freqs(64).double().cuda(), ws)
    with pytest.raises(L.LoraError):
        KV.lora_qk_rope(q, k, pos, freqs(64)[:6].cuda(), ws)               # 12 rotated elements
    with pytest.raises(L.LoraError):
        KV.lora_qk_rope(q, k, pos, freqs(128).cuda(), ws)                  # more than the row has
    empty, _ = KV.lora_qk_rope(q[:0], k[:0], pos[:0], None, ws)
    assert empty.shape == (0, 2, 64)


# --- the 4-bit cache: writes and reads -------------------------------------------

def odd_rows(n, Hk, D, seed):
    """Rows of many sizes, with ties, zeros, subnormal numbers, infinities, NaN and what saturates among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, Hk, D, generator=g) * torch.exp2(torch.randint(-20, 17, (n, Hk, 1), generator=g).float())
    flat = x.view(n * Hk, D)
    for i in range(0, n * Hk, 7):      # multiples of half steps of a scale: ties
        s = (1 + float(torch.randint(0, 8, (1,), generator=g)) / 8) * 2.0 ** float(torch.randint(-6, 6, (1,), generator=g))
        flat[i] = s * torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6])[torch.randint(0, 8, (D,), generator=g)]
        flat[i] *= torch.where(torch.rand(D, generator=g) < .5, -1.0, 1.0)
    special = [0.0, -0.0, 1e-40, -1e-30, 1e-5, 61440.0, 65504.0, 1e30, float("inf"), -float("inf"), float("nan"), 2.0 ** -16]
    for i, v in enumerate(special):
        flat[(3 + 5 * i) % (n * Hk), (5 * i) % D] = v
    flat[1 % (n * Hk)] = 0
    return x.to(BF)


@pytest.mark.parametrize("D", [8, 64, 72, 80, 128])
@pytest.mark.parametrize("Hk,page,n", [(1, 16, 1), (3, 16, 45), (8, 64, 130), (2, 4096, 300)])
def test_codes_and_scales_are_those_of_the_definition(ws, D, Hk, page, n):
    pages = -(-n // page) + 1
    g = torch.Generator().manual_seed(D + n)
    slot = torch.randperm(pages * page, generator=g)[:n].int()
    if n > 4:
        slot[2] = -1
    k, v = odd_rows(n, Hk, D, D + n), odd_rows(n, Hk, D, D + n + 1)
    wide = torch.cat([k, v, k], -1).cuda()                       # strided views
    data = torch.full((pages, Hk, KV.lora_kv4_block_size(page, D)), 170, dtype=torch.uint8, device="cuda")
    cache = KV.Kv4Cache(data, page, D)
    KV.lora_kv4_store(wide[..., :D], wide[..., D:2 * D], cache, slot.cuda(), ws)
    assert L.lora_get_status(ws) == 0
    want = torch.full((pages, Hk, page // 16, 18 * ref.padded(D)), 170, dtype=torch.uint8)
    for t in range(n):
        if slot[t] < 0:
            continue
        for h in range(Hk):
            ref.put(want[slot[t] // page, h, slot[t] % page // 16], int(slot[t]) % 16, k[t, h], v[t, h])
    assert torch.equal(data.cpu().view_as(want), want)
    # and back
    ko, vo = KV.lora_kv4_load(cache, slot.cuda(), ws)
    assert L.lora_get_status(ws) == 0
    for got, x in ((ko, k), (vo, v)):
        y = ref.dequantise(*ref.quantise(x))[..., :D]
        y[slot < 0] = 0
        got = got.double().cpu()
        assert torch.equal(got.isnan(), y.isnan()) and torch.equal(got.nan_to_num(), y.nan_to_num())


def test_reading_back_other_slots_and_parts(ws):
    k, v = (torch.randn(40, 2, 64, device="cuda").to(BF) for _ in range(2))
    cache = KV.Kv4Cache.zeros(4, 2, 16, 64)
    KV.lora_kv4_store(k, v, cache, torch.arange(40, dtype=torch.int32, device="cuda"), ws)
    rows = i32([5, 5, -1, 63, 39, 0, 64, -2])
    out = torch.full((8, 2, 3, 64), 7.0, dtype=BF, device="cuda")   # strided outputs
    KV.lora_kv4_load(cache, rows, ws, k=out[:, :, 0], v=out[:, :, 2])
    assert L.lora_get_status(ws) == A.LORA_DEV_BAD_PAGE
    assert (out[:, :, 1] == 7).all() and torch.equal(out[0], out[1]) and (out[0, :, 0] != 0).any()
    for i in (2, 3, 6, 7):                                          # none, never written, outside
        assert (out[i, :, 0] == 0).all() and (out[i, :, 2] == 0).all()
    lib = KV._lib()
    only = torch.empty(8, 2, 64, dtype=BF, device="cuda")           # keys alone, values alone
    for a, b, j in ((only.data_ptr(), None, 0), (None, only.data_ptr(), 2)):
        assert lib.lora_kv4_load(cache.packed, rows.data_ptr(), 8, a, b, 128, 64, 128, 64, ws.addr, ws.nbytes, None) == 0
        torch.cuda.synchronize()
        assert torch.equal(only, out[:, :, j])
    L.lora_get_status(ws)


def test_4_bit_slots_outside_the_cache_are_skipped(ws):
    k = torch.randn(4, 1, 128, device="cuda").to(BF)
    cache = KV.Kv4Cache.zeros(2, 1, 16, 128)
    KV.lora_kv4_store(k, k, cache, i32([32, -5, -1, 3]), ws)
    assert L.lora_get_status(ws) == A.LORA_DEV_BAD_PAGE
    assert int((cache.data.view(2, 1, -1) != 0).sum()) > 0 and (cache.data[1] == 0).all()


def test_4_bit_cache_views_and_refusals(ws):
    # pages of two layers in one allocation, heads outermost: any order whose blocks are contiguous
    data = torch.zeros(3, 5, 2, 2304, dtype=torch.uint8, device="cuda")
    k, v = (torch.randn(30, 3, 128, device="cuda").to(BF) for _ in range(2))
    a = KV.Kv4Cache(data[:, :, 1].transpose(0, 1), 16, 128)
    b = KV.Kv4Cache.zeros(5, 3, 16, 128)
    slots = torch.arange(3, 33, dtype=torch.int32, device="cuda")
    for c in (a, b):
        KV.lora_kv4_store(k, v, c, slots, ws)
    assert torch.equal(a.data, b.data) and (data[:, :, 0] == 0).all()
    for bad in (data[..., :2300].transpose(0, 1), data[:, :, :, ::2], data.int(), data[:0]):
        with pytest.raises(ValueError):
            KV.Kv4Cache(bad[:, :, 0] if bad.ndim == 4 and bad.shape[0] else bad, 16, 128)
    with pytest.raises(ValueError):
        KV.Kv4Cache(data[:, :, 0], 8, 128)
    with pytest.raises(ValueError):
        KV.lora_kv4_store(k[..., :64], v[..., :64], b, slots, ws)
    with pytest.raises(ValueError):
        KV.lora_kv4_load(b, slots, ws, k=k[:3])


# --- pages -----------------------------------------------------------------------

def device_state(s, stride=None):
    table = torch.tensor(s.table, dtype=torch.int32)
    if stride:
        wide = torch.full((table.shape[0], stride), 777, dtype=torch.int32)
        wide[:, :table.shape[1]] = table
        table = wide.cuda()[:, :table.shape[1]]
    return dict(ctx_len=i32(s.ctx), block_table=table.cuda(), ref=i32(s.ref), free_pages=i32(s.free), free_head=i32([s.head]),
                page_size=s.page)


def assert_state(d, s, what=""):
    for name, want in (("ctx_len", s.ctx), ("block_table", s.table), ("ref", s.ref), ("free_pages", s.free),
                       ("free_head", [s.head])):
        assert d[name].tolist() == want, f"{what}: {name}"


@pytest.mark.parametrize("rows,width,page,pages", [(6, 5, 8, 40), (40, 9, 16, 200), (300, 30, 16, 5000), (9, 3, 4096, 30)])
def test_random_steps_keep_the_books(rows, width, page, pages):
    """Growing by lora_kv_plan, releasing, forking and compacting in random order, in step with plain loops."""
    rng = random.Random(rows)
    s = ref.Pages([[-1] * width for _ in range(rows)], [0] * rows, [0] * pages, rng.sample(range(pages), pages), 0, page)
    d = device_state(s, stride=width + 3)
    ws, aws = KV.PagesWorkspace(pages), A.AttnWorkspace(rows * width * page, rows)
    for step in range(25):
        # every request grows a little, if it can
        new = [rng.choice([0, 0, 1, page, 3 * page]) for _ in range(rows)]
        new = [min(n, width * page - c) for n, c in zip(new, s.ctx)]
        d["free_head"] = A.lora_kv_plan(i32(new), d["ctx_len"], d["block_table"], d["free_pages"], d["free_head"], page, pages,
                                        aws, max_tokens=sum(new) + 1).free_head
        for r, n in enumerate(new):
            have = s.held(r)
            need = -(-(s.ctx[r] + n) // page) - have
            if need == 0 or s.head + need <= pages:
                s.table[r][have:have + need] = s.free[s.head:s.head + need]
                s.head += need
                s.ctx[r] += n
            elif need:
                break                                   # the first it cannot serve and all later that need a page
        else:
            r = rows
        for q in range(r + 1, rows):
            if -(-(s.ctx[q] + new[q]) // page) == s.held(q):
                s.ctx[q] += new[q]
        d["ctx_len"].copy_(i32(s.ctx))
        L.lora_get_status(aws)
        assert_state(d, s, f"step {step}: plan")
        dropped = rng.sample(range(rows), rng.randrange(1, max(2, rows // 2)))
        s.release(dropped)
        KV.lora_kv_release(i32(dropped), ws=ws, **d)
        assert L.lora_get_status(ws) == 0
        assert_state(d, s, f"step {step}: release")
        parents = [rng.choice([r for r in range(rows) if r not in dropped] or [0]) for _ in dropped]
        if set(parents) & set(dropped):
            continue
        pairs = s.fork(parents, dropped)
        src, dst = KV.lora_kv_fork(i32(parents), i32(dropped), ws=ws, **d)
        status = L.lora_get_status(ws)
        assert status == (A.LORA_DEV_NO_PAGE if any(s.ctx[c] != s.ctx[p] for p, c in zip(parents, dropped)) else 0)
        assert list(zip(src.tolist(), dst.tolist())) == pairs
        assert_state(d, s, f"step {step}: fork")
        limit, most = rng.randrange(pages + 1), rng.choice([0, 3, pages])
        if step % 2:     # into other arrays
            out = {k: torch.full_like(d[n], -9) for k, n in (("ref_out", "ref"), ("free_out", "free_pages"), ("head_out", "free_head"))}
            out["table_out"] = torch.full((rows, width + 3), 777, dtype=torch.int32, device="cuda")[:, :width]
            before = {k: v.clone() for k, v in d.items() if k != "page_size"}
        else:
            out = {}
        src, dst = KV.lora_kv_compact(limit=limit, ws=ws, max_copies=most, **d, **out)
        assert L.lora_get_status(ws) == 0
        if out:
            for k, v in before.items():
                assert torch.equal(d[k], v), k
            d.update(block_table=out["table_out"], ref=out["ref_out"], free_pages=out["free_out"], free_head=out["head_out"])
        pairs = s.compact(limit, most)
        assert list(zip(src.tolist(), dst.tolist())) == pairs
        assert_state(d, s, f"step {step}: compact to {limit}")
        holders = [0] * pages
        for r in range(rows):
            for p in s.table[r][:s.held(r)]:
                holders[p] += 1
        assert s.ref == [max(0, h - 1) for h in holders] and sorted(s.free[s.head:]) == [p for p in range(pages) if not holders[p]]


def small(head=4):
    """Two rows of 20 and 32 tokens in pages of 8, and two empty rows."""
    return ref.Pages([[5, 3, 9, -1], [1, 2, 4, 6], [-1] * 4, [-1] * 4], [20, 32, 0, 0], [0] * 12, [7, 0, 8, 10, 11], head - 4, 8)


def test_release_of_rows_named_twice_or_unknown():
    s = small()
    s.ref[3], s.ref[9] = 1, 2
    s.free, s.head = [0, 0, 0, 0, 0, 0, 0, 7, 8], 7
    d, ws = device_state(s), KV.PagesWorkspace(12)
    s.release([0, 1, 0])
    KV.lora_kv_release(i32([0, -1, 1, 0, 4]), ws=ws, **d)
    assert L.lora_get_status(ws) == KV.LORA_DEV_BAD_ROW
    assert_state(d, s)
    assert s.free[2:7] == [1, 2, 4, 5, 6] and s.ref[9] == 1
    # again: nothing is held any more
    KV.lora_kv_release(i32([0, 1]), ws=ws, **d)
    assert L.lora_get_status(ws) == 0
    assert_state(d, s)


def test_release_into_a_list_without_room_and_bad_states():
    s = small()
    s.head = 2
    d, ws = device_state(s), KV.PagesWorkspace(12)
    s.release([1])                                   # four pages, two places
    KV.lora_kv_release(i32([1]), ws=ws, **d)
    assert L.lora_get_status(ws) == A.LORA_DEV_NO_PAGE
    assert_state(d, s)
    assert s.head == 0 and s.free[:2] == [1, 2]
    s = small()
    s.ctx[0], s.table[0][1], s.head = 99, 12, 4      # longer than its row, a page outside, one that was never taken
    s.table[0][3] = -1
    d = device_state(s)
    KV.lora_kv_release(i32([0]), ws=ws, **d)
    assert L.lora_get_status(ws) == A.LORA_DEV_BAD_LENGTH | A.LORA_DEV_BAD_PAGE
    s.release([0])
    assert_state(d, s)


def test_forks_that_cannot_be():
    s = small()
    s.free, s.head = [7, 0], 0
    parents, children = [0, 0, 1, 9, 0, 2, 0], [2, 2, 3, 1, -1, 0, 3]
    # the second names a child again, 9 and -1 are no rows, 0 and 2 are parents, 3 is named again
    d, ws = device_state(s), KV.PagesWorkspace(12)
    pairs = s.fork(parents, children)
    src, dst = KV.lora_kv_fork(i32(parents), i32(children), ws=ws, **d)
    assert L.lora_get_status(ws) == KV.LORA_DEV_BAD_ROW
    assert list(zip(src.tolist(), dst.tolist())) == pairs
    assert_state(d, s)


def test_forks_run_out_of_pages():
    s = small()
    s.free, s.head = [7, 0, 10], 2
    s.table += [[-1] * 4 for _ in range(4)]
    s.ctx += [0] * 4
    d, ws = device_state(s), KV.PagesWorkspace(12)
    parents, children = [0, 0, 1, 0, 1], [2, 3, 4, 5, 6]     # the second and fourth need a page that is not there
    pairs = s.fork(parents, children)
    src, dst = KV.lora_kv_fork(i32(parents), i32(children), ws=ws, **d)
    assert L.lora_get_status(ws) == A.LORA_DEV_NO_PAGE
    assert list(zip(src.tolist(), dst.tolist())) == pairs and pairs[0] == (9, 10) and pairs[1] == (-1, -1)
    assert_state(d, s)
    assert s.ctx[2:7] == [20, 0, 32, 0, 32]
    # full pages alone need none; a parent without tokens gives a child without
    KV.lora_kv_release(i32([2, 3, 4, 5, 6]), ws=ws, **d)
    s.release([2, 3, 4, 5, 6])
    s.fork([1, 7], [2, 3])
    KV.lora_kv_fork(i32([1, 7]), i32([2, 3]), ws=ws, **d)
    assert L.lora_get_status(ws) == 0
    assert_state(d, s)


def test_forks_onto_bad_pages():
    """A page of the list outside the cache is nobody's: the child's entry is -1, never what stood there before."""
    s = small()
    s.free, s.head = [99, -1, 10], 0
    s.table += [[7] * 4 for _ in range(3)]
    s.ctx += [0] * 3
    d, ws = device_state(s), KV.PagesWorkspace(12)
    src, dst = KV.lora_kv_fork(i32([0, 0, 0]), i32([4, 5, 6]), ws=ws, **d)
    assert L.lora_get_status(ws) == A.LORA_DEV_BAD_PAGE
    old = s.table[0][2]
    assert list(zip(src.tolist(), dst.tolist())) == [(-1, -1), (-1, -1), (old, 10)]
    assert [t[2] for t in d["block_table"].tolist()[4:]] == [-1, -1, 10] and d["free_head"].item() == 3
    assert d["ctx_len"].tolist()[4:] == [20] * 3
    # so is the parent's unfinished page
    s = small()
    s.table[0][2] = 12
    d = device_state(s)
    src, dst = KV.lora_kv_fork(i32([0]), i32([2]), ws=ws, **d)
    assert L.lora_get_status(ws) == A.LORA_DEV_BAD_PAGE and (src.item(), dst.item()) == (-1, -1)
    assert d["block_table"].tolist()[2][2] == s.free[s.head] and d["free_head"].item() == s.head + 1


def test_compaction_of_bad_states():
    s = small()
    s.free, s.head = [7, 0, 9, 0, 99, -4], 0              # a held page, one twice, two outside
    s.table[1][3] = 50
    d, ws = device_state(s), KV.PagesWorkspace(12)
    src, dst = KV.lora_kv_compact(limit=5, ws=ws, max_copies=4, **d)
    assert L.lora_get_status(ws) == A.LORA_DEV_BAD_PAGE
    assert s.compact(5, 4) == list(zip(src.tolist(), dst.tolist())) == [(5, 0), (-1, -1), (-1, -1), (-1, -1)]
    assert_state(d, s)
    # limits beyond the cache and of nothing, and no room for pairs
    for limit, most in ((0, 4), (12, 4), (1 << 30, 4), (3, 0)):
        KV.lora_kv_compact(limit=limit, ws=ws, max_copies=most, **d)
        s.compact(limit, most)
        L.lora_get_status(ws)
        assert_state(d, s, str(limit))


@pytest.mark.parametrize("order", ["phsd", "pshd", "hpsd", "shpd"])
@pytest.mark.parametrize("Hk,page,D", [(1, 8, 8), (3, 16, 72), (8, 32, 128)])
def test_page_copies(ws, order, Hk, page, D):
    shape = dict(zip("phsd", (50, Hk, page, D)))
    axes = [order.index(c) for c in "phsd"]
    kc, vc = (torch.randn([shape[c] for c in order], device="cuda").to(BF).permute(axes) for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    src, dst = [3, -1, 49, 7, 3, -1, 0], [10, -1, 11, 12, 13, -1, 48]
    KV.lora_kv_copy(i32(src), i32(dst), kc, vc, ws)
    assert L.lora_get_status(ws) == 0
    for a, b in zip(src, dst):
        if a >= 0:
            k0[b], v0[b] = k0[a], v0[a]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    KV.lora_kv_copy(i32([50, 2, -2, 5]), i32([1, 50, 4, -1]), kc, vc, ws)
    assert L.lora_get_status(ws) == A.LORA_DEV_BAD_PAGE
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_page_copies_of_4_bit_caches(ws):
    data = torch.randint(0, 256, (3, 40, 2, 2304), dtype=torch.uint8, device="cuda")
    for view in (data[:, :, 0].transpose(0, 1), data.view(40, 6, 2304)):
        c = KV.Kv4Cache(view, 16, 128)
        want = view.clone()
        want[7], want[8] = want[3].clone(), want[39].clone()
        KV.lora_kv4_copy(i32([3, -1, 39]), i32([7, -1, 8]), c, ws)
        assert L.lora_get_status(ws) == 0 and torch.equal(view, want)
    KV.lora_kv4_copy(i32([1] * 5000), i32([-1] * 5000), c, ws)
    assert L.lora_get_status(ws) == A.LORA_DEV_BAD_PAGE and torch.equal(view, want)


def test_copies_of_many_pairs_mostly_none(ws):
    kc, vc = (torch.randn(3000, 2, 16, 64, device="cuda").to(BF) for _ in range(2))
    rng = random.Random(4)
    src, dst = [-1] * 20000, [-1] * 20000
    pages = rng.sample(range(3000), 2000)
    for i, at in enumerate(rng.sample(range(20000), 1000)):
        src[at], dst[at] = pages[i], pages[1000 + i]
    k0 = kc.clone()
    KV.lora_kv_copy(i32(src), i32(dst), kc, vc, ws)
    k0[torch.tensor(pages[1000:])] = k0[torch.tensor(pages[:1000])]
    assert torch.equal(kc, k0)


def test_many_pages_and_rows():
    """More pages than one CTA counts, as many rows as there may be, all of them released at once."""
    rows, width, pages, page = 4096, 40, 200000, 16
    g = torch.Generator().manual_seed(3)
    ctx = torch.randint(0, width * page + 1, (rows,), generator=g)
    held = (ctx + page - 1) // page
    order = torch.randperm(pages, generator=g).int()
    first = torch.cumsum(held, 0) - held
    col = torch.arange(width)[None, :]
    table = torch.where(col < held[:, None], order[(first[:, None] + col).clamp(max=pages - 1)], -1).int()
    total = int(held.sum())
    d = dict(ctx_len=ctx.int().cuda(), block_table=table.cuda(), ref=torch.zeros(pages, dtype=torch.int32, device="cuda"),
             free_pages=torch.cat([torch.full((total,), -1, dtype=torch.int32), order[total:]]).cuda(), free_head=i32([total]),
             page_size=page)
    ws = KV.PagesWorkspace(pages)
    limit = (total + pages) // 2
    src, dst = KV.lora_kv_compact(limit=limit, ws=ws, **d)
    n = int((src >= 0).sum())
    assert L.lora_get_status(ws) == 0 and n == int((order[:total] >= limit).sum())
    assert int(d["block_table"].max()) < limit and int(d["free_head"]) == total
    used = torch.sort(d["block_table"][d["block_table"] >= 0]).values
    assert torch.equal(torch.sort(torch.cat([used, d["free_pages"][total:]])).values, torch.arange(pages, device="cuda").int())
    KV.lora_kv_release(torch.arange(rows, dtype=torch.int32, device="cuda").flip(0).contiguous(), ws=ws, **d)
    assert L.lora_get_status(ws) == 0
    assert int(d["free_head"]) == 0 and int(d["ctx_len"].max()) == 0 and int(d["ref"].abs().max()) == 0
    assert torch.equal(d["free_pages"][:total], used)


@pytest.mark.parametrize("pages,rows,width", [(32768, 256, 128), (32769, 256, 128), (32768, 256, 129), (32768, 4, 1024), (32768, 16, 1025)])
def test_compaction_that_moves_half_of_all_pages(pages, rows, width):
    """Every held page has to move: around the most pages and entries that one launch takes."""
    page, half = 16, pages // 2
    rng = random.Random(pages + rows)
    used = min(half, rows * width)
    order = rng.sample(range(half, pages), used)
    table, ctx, at = [], [], 0
    for r in range(rows):
        n = min(width, used - at) if r % 2 == 0 else 0
        table.append(order[at:at + n] + [-1] * (width - n))
        ctx.append(n * page)
        at += n
    for r in range(1, rows, 2):
        n = min(width, used - at)
        table[r], ctx[r], at = order[at:at + n] + [-1] * (width - n), n * page, at + n
    held = set(order)
    free = [p for p in range(pages) if p not in held]
    rng.shuffle(free)
    s = ref.Pages(table, ctx, [rng.randrange(3) if p in held else 0 for p in range(pages)], [-1] * used + free, used, page)
    d, ws = device_state(s), KV.PagesWorkspace(pages)
    src, dst = KV.lora_kv_compact(limit=half, ws=ws, **d)
    assert L.lora_get_status(ws) == 0
    pairs = s.compact(half, len(s.free))
    assert list(zip(src.tolist(), dst.tolist())) == pairs and sum(a >= 0 for a, _ in pairs) == used
    assert_state(d, s)
