"""Measured cases of the serving attention operators.

Four operators work together around the LoRA projections of an attention
layer: `lora_kv_plan` (block tables, slot map, positions and the step's
lora_id_map from the requests' lengths), `lora_kv_store` (the new tokens' keys
and values into the paged cache), `lora_attn_paged` (attention of the new
tokens over that cache, single tokens and chunks alike) and `lora_attn_prompt`
(causal attention over whole packed prompts).

Where `own` is false, `run` computes them from elementary torch operations in
32 bits; where it is true, it calls the library.  Tensors are bf16 as
everywhere in the library; q, k and v are views of one merged QKV projection's
rows, the form `lora_linear` leaves them in.
"""
import math
import random

import numpy as np
import torch

own = False

BF16 = torch.bfloat16


# --- the cases ---------------------------------------------------------------

def listed():
    # 32 query and 8 key/value heads of 128 are the head layout of the merged
    # QKV projection (K = 4096, N = 4096 + 1024 + 1024) that the library's own
    # benchmark runs.
    h = dict(heads=32, kv_heads=8, dim=128)
    return [
        # bookkeeping of one decode step: a full batch, one new token each
        dict(name="plan_decode", op="plan", reqs=256, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=8192, page=16, lens=1),
        # bookkeeping of a mixed step: many requests, idle ones, chunks of prompts
        dict(name="plan_mixed", op="plan", reqs=777, new_lo=0, new_hi=96, ctx_lo=0, ctx_hi=30000, page=16, lens=2),
        # the 32 new rows of the library's decode step
        dict(name="store_decode", op="store", reqs=32, new_lo=1, new_hi=1, ctx_lo=10, ctx_hi=500, page=16, lens=3, **h),
        # the rows of a prefill step of 8 K tokens or so
        dict(name="store_prefill", op="store", reqs=29, new_lo=64, new_hi=512, ctx_lo=0, ctx_hi=100, page=16, lens=4, **h),
        # one request, one token: the latency of an interactive user
        dict(name="paged_one", op="paged", reqs=1, new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=1000, page=16, lens=5, **h),
        # the decode step of 32 requests with contexts of all lengths
        dict(name="paged_decode", op="paged", reqs=32, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=8000, page=16, lens=6, **h),
        # a large decode batch with long contexts: the cache is read once, several GB of it
        dict(name="paged_decode_large", op="paged", reqs=128, new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=16000, page=16,
             lens=7, **h),
        # a few drafted tokens a request are verified at once; seven heads share a key head
        dict(name="paged_verify", op="paged", reqs=48, new_lo=0, new_hi=5, ctx_lo=300, ctx_hi=6000, page=32, lens=8,
             heads=28, kv_heads=4, dim=128),
        # chunks of long prompts over what is cached of them, and decoding requests beside them
        dict(name="paged_chunk", op="paged", reqs=6, new_lo=1, new_hi=700, ctx_lo=500, ctx_hi=9000, page=64, lens=9,
             heads=32, kv_heads=4, dim=64),
        # one short prompt: latency again
        dict(name="prompt_short", op="prompt", reqs=1, new_lo=77, new_hi=77, lens=10, **h),
        # the library's prefill step: 16 requests of 16 to 128 tokens
        dict(name="prompt_packed", op="prompt", reqs=16, new_lo=16, new_hi=128, lens=11, **h),
        # one long prompt
        dict(name="prompt_long", op="prompt", reqs=1, new_lo=16384, new_hi=16384, lens=12, **h),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (1, 2, 4, 5, 7, 8, 16) if g * kv <= 40])
    return dict(heads=group * kv, kv_heads=kv, dim=rng.choice([64, 80, 128, 128]))


def draw(rng):
    op = rng.choice(["plan", "store", "paged", "paged", "paged", "prompt", "prompt"])
    c = dict(op=op, lens=rng.randrange(1 << 20))
    if op == "prompt":
        total = _log(rng, 20, 16384)
        c["reqs"] = min(_log(rng, 1, 40), total)
        mean = total / c["reqs"]
        # near-equal or very unequal lengths
        f = rng.choice([0.02, 0.5, 0.9])
        c["new_lo"], c["new_hi"] = max(1, int(f * mean)), max(1, int((2 - f) * mean))
        c.update(_draw_heads(rng))
        while c["reqs"] * c["heads"] * c["new_hi"] ** 2 > 32 * 16384 ** 2:   # the padded plain form stays affordable
            c["new_hi"] = c["new_hi"] * 3 // 4
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
        return c
    c["page"] = rng.choice([16, 16, 32, 64, 128])
    c["ctx_lo"] = rng.choice([0, 1, _log(rng, 2, 1000)])
    c["ctx_hi"] = c["ctx_lo"] + _log(rng, 10, 15000)
    if op == "plan":
        c["reqs"] = _log(rng, 1, 1024)
        c["new_hi"] = rng.choice([1, 1, _log(rng, 2, 200)])
        c["new_lo"] = rng.choice([0, c["new_hi"]])
        return c
    c.update(_draw_heads(rng))
    if op == "store":
        c["reqs"] = _log(rng, 1, 256)
        c["new_hi"] = rng.choice([1, _log(rng, 2, 8192 // c["reqs"] + 2)])
        c["new_lo"] = rng.choice([1, c["new_hi"]])
        c["ctx_hi"] = min(c["ctx_hi"], c["ctx_lo"] + 500)
        return c
    c["reqs"] = _log(rng, 1, 160)
    c["new_hi"] = rng.choice([1, 1, _log(rng, 2, 12), _log(rng, 13, 1000)])
    c["new_lo"] = rng.choice([0, 1, c["new_hi"]])
    # the plain form pads to the longest: its scores and its gathered cache stay affordable
    while (c["reqs"] * c["heads"] * c["new_hi"] * (c["ctx_hi"] + c["new_hi"]) > 4e9 or
           c["reqs"] * c["kv_heads"] * c["dim"] * (c["ctx_hi"] + c["new_hi"]) > 128 * 8 * 128 * 16000):
        c["reqs"] = max(1, c["reqs"] * 3 // 4)
        c["ctx_hi"] = max(c["ctx_lo"], c["ctx_hi"] * 7 // 8)
        if c["reqs"] == 1:
            c["new_hi"] = max(1, c["new_hi"] * 3 // 4)
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
    return c


def _lengths(c):
    """(new tokens, cached tokens) of every request; a case's lengths are its own, whatever the seed."""
    r = random.Random(c["lens"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["reqs"])]
    if sum(new) == 0:
        new[0] = 1
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["reqs"])] if "ctx_lo" in c else [0] * c["reqs"]
    return new, ctx


def _cdiv(a, b):
    return -(-a // b)


# --- inputs ------------------------------------------------------------------

def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new, ctx = _lengths(c)
    R, T, op = c["reqs"], sum(new), c["op"]
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = dict(op=op, case=c, T=T, cu=torch.tensor(cu, **i32), max_new=max(new))
    if op != "plan":
        H, Hk, D = c["heads"], c["kv_heads"], c["dim"]
        qkv = torch.randn(T, (H + 2 * Hk) * D, device="cuda", generator=g).to(BF16)   # the merged projection's rows
        s["q"] = qkv[:, :H * D].view(T, H, D)
        s["k"] = qkv[:, H * D:(H + Hk) * D].view(T, Hk, D)
        s["v"] = qkv[:, (H + Hk) * D:].view(T, Hk, D)
        s["scale"] = 1.0 / math.sqrt(D)
    if op in ("paged", "prompt"):
        s["o"] = torch.empty(T, H, D, dtype=BF16, device="cuda")
        s["lse"] = torch.empty(T, H, dtype=torch.float32, device="cuda")
    if op != "prompt":
        P = c["page"]
        s["page"] = P
        total = [a + b for a, b in zip(new, ctx)]
        have = [_cdiv(a, P) for a in ctx]                    # pages each request holds before the step
        used = [_cdiv(a, P) for a in total]
        width = max(used) + 3
        pages = sum(used) + 5
        order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        s["kv_len"] = torch.tensor(total, **i32)
        s["ctx"], s["new"] = torch.tensor(ctx, **i32), torch.tensor(new, **i32)
        s["pages"], s["max_kv"] = pages, max(total)
        # the page of (request, column): requests' pages drawn from `order` in turn
        first = np.concatenate([[0], np.cumsum(have if op == "plan" else used)])
        col = np.arange(width)[None, :]
        held = np.array(have if op == "plan" else used)[:, None]
        idx = torch.from_numpy(np.where(col < held, first[:-1, None] + col, -1)).cuda()
        s["table"] = torch.where(idx >= 0, order[idx.clamp(min=0)], torch.full_like(idx, -1, dtype=torch.int32)).to(torch.int32)
        if op == "plan":
            s["free"] = order[int(first[-1]):].contiguous()  # the rest is free, handed out in this order
            s["head"] = torch.zeros(1, **i32)
            s["adapter"] = torch.randint(-1, 20, (R,), device="cuda", generator=g, dtype=torch.int32)
        else:
            kc = torch.randn(pages, Hk, P, D, device="cuda", generator=g, dtype=BF16)
            vc = torch.randn(pages, Hk, P, D, device="cuda", generator=g, dtype=BF16)
            s["k_cache"], s["v_cache"] = kc, vc
            if op == "store":
                pos = np.concatenate([np.arange(a, a + n) for a, n in zip(ctx, new)])
                req = np.repeat(np.arange(R), new)
                page = s["table"][torch.from_numpy(req).cuda(), torch.from_numpy(pos // P).cuda()]
                s["slot"] = (page * P + torch.from_numpy(pos % P).cuda()).to(torch.int32)
    if own:   # the workspace and the step's outputs and schedule that a serving program keeps for all its layers
        from segmented_gemm_gb300 import attn as A
        if op == "plan":
            s["ws"] = A.AttnWorkspace(T, R)
            s["plan"] = A.KvPlan(T, R)
        elif op == "store":
            s["ws"] = A.AttnWorkspace(T, R)
        else:
            s["ws"] = A.AttnWorkspace(T, R, H, Hk, D)
            if op == "paged":
                s["sched"] = A.lora_attn_schedule(s["cu"], s["kv_len"], T, width * P, H, Hk, D, s["ws"])
    return s


# --- one pass ----------------------------------------------------------------

def run(s):
    op = s["op"]
    if own:
        from segmented_gemm_gb300 import attn as A
        if op == "plan":
            p = A.lora_kv_plan(s["new"], s["ctx"], s["table"], s["free"], s["head"], s["page"], s["pages"], s["ws"],
                               req_adapter=s["adapter"], out=s["plan"])
            return dict(table=s["table"], cu=p.cu_new, kv_len=p.kv_len, slot=p.slot_map, position=p.position,
                        ids=p.lora_id_map, head=p.free_head)
        if op == "store":
            A.lora_kv_store(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slot"], s["ws"])
            return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
        if op == "paged":
            A.lora_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"], s["scale"],
                              s["ws"], sched=s["sched"], o=s["o"], lse=s["lse"])
            return dict(o=s["o"], lse=s["lse"])
        A.lora_attn_prompt(s["q"], s["k"], s["v"], s["cu"], s["scale"], s["ws"], o=s["o"], lse=s["lse"])
        return dict(o=s["o"], lse=s["lse"])
    if op == "plan":
        return _plain_plan(s)
    if op == "store":
        slot = s["slot"].long()
        s["k_cache"][slot // s["page"], :, slot % s["page"]] = s["k"]
        s["v_cache"][slot // s["page"], :, slot % s["page"]] = s["v"]
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    # both attentions: requests padded to the longest, the packed rows gathered into them
    dev, R = s["cu"].device, s["case"]["reqs"]
    cu = s["cu"].long()
    at = torch.arange(s["max_new"], device=dev)
    n = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + at[None, :]).clamp(max=s["T"] - 1)                     # [R, Lq]
    if op == "prompt":
        k, v = s["k"][row].float(), s["v"][row].float()                           # [R, Lk, Hk, D]
        kv_len = n
    else:
        P = s["page"]
        t = s["table"][:, :_cdiv(s["max_kv"], P)].long().clamp(min=0)
        k = s["k_cache"][t].float().transpose(2, 3).flatten(1, 2)                 # [R, pages, Hk, P, D] -> [R, Lk, Hk, D]
        v = s["v_cache"][t].float().transpose(2, 3).flatten(1, 2)
        kv_len = s["kv_len"].long()
    Hk, D = k.shape[2], k.shape[3]
    G, Lq, Lk = s["q"].shape[1] // Hk, s["max_new"], k.shape[1]
    q = s["q"][row].float().view(R, Lq, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(R, Hk, G * Lq, D)
    p = torch.matmul(q, k.permute(0, 2, 3, 1)).view(R, Hk, G, Lq, Lk)
    p.mul_(s["scale"])
    limit = (kv_len - n)[:, None] + at[None, :] + 1                               # keys each row sees
    seen = torch.arange(Lk, device=dev)[None, None, :] < limit[:, :, None]        # [R, Lq, Lk]
    p.masked_fill_(~seen[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True).clamp(min=-3e38)                                 # a row that sees nothing: zeros
    p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, Hk, G * Lq, Lk), v.transpose(1, 2)).view(R, Hk, G, Lq, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))
    # back to the packed rows
    req = torch.repeat_interleave(torch.arange(R, device=dev), n, output_size=s["T"])
    local = torch.arange(s["T"], device=dev) - cu[req]
    o = o.permute(0, 3, 1, 2, 4).reshape(R, Lq, Hk * G, D)[req, local]
    lse = lse.permute(0, 3, 1, 2, 4).reshape(R, Lq, Hk * G)[req, local]
    return dict(o=o.to(BF16), lse=lse)


def _plain_plan(s):
    dev, P, T = s["new"].device, s["page"], s["T"]
    new, ctx = s["new"].long(), s["ctx"].long()
    total = new + ctx
    have, used = (ctx + P - 1) // P, (total + P - 1) // P
    need = used - have
    before = torch.cumsum(need, 0) - need
    left = s["free"].numel() - s["head"].long()
    ok = (need == 0) | (before + need <= left)
    col = torch.arange(s["table"].shape[1], device=dev)[None, :]
    take = (s["head"].long() + before[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    fresh = (col >= have[:, None]) & (col < used[:, None]) & ok[:, None]
    table = torch.where(fresh, s["free"][take], s["table"])
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(new, 0)])
    t = torch.arange(T, device=dev)
    req = torch.searchsorted(cu, t, right=True) - 1
    pos = ctx[req] + t - cu[req]
    page = table[req, pos // P].long()
    slot = torch.where(ok[req], page * P + pos % P, torch.full_like(pos, -1))
    head = s["head"] + torch.where(ok, need, torch.zeros_like(need)).sum()
    i = torch.int32
    return dict(table=table, cu=cu.to(i), kv_len=torch.where(ok, total, torch.zeros_like(total)).to(i), slot=slot.to(i),
                position=pos.to(i), ids=s["adapter"][req], head=head.to(i))


# --- what a pass cannot do without -------------------------------------------

def work(c):
    new, ctx = _lengths(c)
    T, R = sum(new), c["reqs"]
    if c["op"] == "plan":
        fresh = sum(_cdiv(a + b, c["page"]) - _cdiv(b, c["page"]) for a, b in zip(new, ctx))
        # lengths and adapters in, cu and kv_len out; free pages in, table entries out; slot, position, id a token
        return dict(bytes=4 * (5 * R + 2 * fresh + 3 * T), flops=0)
    H, Hk, D = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "store":
        return dict(bytes=T * (4 * Hk * D * 2 + 4), flops=0)
    kv = [(a + b) if a else 0 for a, b in zip(new, ctx)]      # a request without new tokens is not read
    pairs = sum(n * x + n * (n + 1) // 2 for n, x in zip(new, ctx))
    table = sum(_cdiv(x, c["page"]) for x in kv) * 4 if c["op"] == "paged" else 0
    return dict(bytes=2 * T * H * D * 2 + T * H * 4 + sum(kv) * Hk * D * 2 * 2 + table, flops=4 * D * H * pairs)


# --- the definition in 64 bits -----------------------------------------------

def exact(c, seed):
    new, ctx = _lengths(c)
    s = prepare(c, seed)
    if c["op"] == "store":
        kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
        for t, slot in enumerate(s["slot"].tolist()):
            kc[slot // s["page"], :, slot % s["page"]] = s["k"][t]
            vc[slot // s["page"], :, slot % s["page"]] = s["v"][t]
        return dict(k_cache=kc.double(), v_cache=vc.double())
    if c["op"] == "plan":
        return _exact_plan(s, new, ctx)
    H, Hk, D = c["heads"], c["kv_heads"], c["dim"]
    o = torch.zeros(s["T"], H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], H), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for r, (n, x) in enumerate(zip(new, ctx)):
        if n == 0:
            continue
        if c["op"] == "prompt":
            k, v = s["k"][t0:t0 + n].double(), s["v"][t0:t0 + n].double()
        else:
            where = np.arange(n + x)
            page = s["table"][r][torch.from_numpy(where // s["page"]).cuda()].long()
            line = torch.from_numpy(where % s["page"]).cuda()
            k, v = s["k_cache"][page, :, line].double(), s["v_cache"][page, :, line].double()
        for b in range(0, n, 512):                            # blocks of queries against the keys that they see
            e = min(n, b + 512)
            keys = x + e
            hidden = torch.arange(keys, device="cuda")[None, :] > x + torch.arange(b, e, device="cuda")[:, None]
            for h in range(Hk):
                cols = slice(h * (H // Hk), (h + 1) * (H // Hk))
                q = s["q"][t0 + b:t0 + e, cols].double()
                sc = torch.einsum("qgd,kd->qgk", q, k[:keys, h]) * s["scale"]
                sc = sc.masked_fill(hidden[:, None], -math.inf)
                lse[t0 + b:t0 + e, cols] = torch.logsumexp(sc, -1)
                o[t0 + b:t0 + e, cols] = torch.einsum("qgk,kd->qgd", torch.softmax(sc, -1), v[:keys, h])
        t0 += n
    return dict(o=o, lse=lse)


def _exact_plan(s, new, ctx):
    P = s["page"]
    table, free, adapter = s["table"].cpu().numpy().copy(), s["free"].cpu().tolist(), s["adapter"].cpu().tolist()
    slot, position, ids, cu, kv = [], [], [], [0], []
    taken = 0
    for r, (n, x) in enumerate(zip(new, ctx)):
        for j in range(_cdiv(x, P), _cdiv(x + n, P)):
            table[r, j] = free[taken]
            taken += 1
        for p in range(x, x + n):
            slot.append(int(table[r, p // P]) * P + p % P)
            position.append(p)
            ids.append(adapter[r])
        cu.append(cu[-1] + n)
        kv.append(x + n)
    to = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return dict(table=torch.from_numpy(table), cu=to(cu), kv_len=to(kv), slot=to(slot), position=to(position),
                ids=to(ids), head=to([taken]))
