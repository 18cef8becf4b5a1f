"""Measured cases of the cache operators that stand around the serving attention.

Three groups: `lora_qk_rope` (norms of queries and keys for each head and the
rotation by position, with the keys' and values' way into the paged cache in
the same pass); the cache held in 4 bits (`lora_kv4_store`, `lora_kv4_load`,
`lora_kv4_attn`); and the pages themselves (`lora_kv_release`, `lora_kv_fork`,
`lora_kv_copy`, `lora_kv_compact`).

Where `own` is false, `run` computes them from elementary torch operations in
32 bits (angles of positions in 64); where it is true, it calls the library.
Tensors are bf16 as everywhere in the library; q, k and v are views of one
merged QKV projection's rows, the form `lora_linear` leaves them in.
"""
import math
import random

import numpy as np
import torch

own = False

BF16 = torch.bfloat16
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # what the low three bits of a 4-bit code stand for


# --- the cases ---------------------------------------------------------------

def listed():
    # 32 query and 8 key/value heads of 128: the merged QKV projection that the library's own benchmark runs
    h = dict(heads=32, kv_heads=8, dim=128)
    return [
        # the 32 rows of the library's decode step, of a model with norms of its queries and keys
        dict(name="rope_decode", op="rope", tokens=32, far=9000, rot=128, norm=True, pairs=False, cache=True, page=16, **h),
        # the rows of a prefill step of 8 K tokens, into the cache
        dict(name="rope_prefill", op="rope", tokens=8100, far=130000, rot=128, norm=True, pairs=False, cache=True,
             page=16, **h),
        # the decode step's keys and values into the 4-bit cache, and the cache read back
        dict(name="quant_decode", op="quant", tokens=32, slots=1024, page=16, **h),
        # a prefill step's
        dict(name="quant_prefill", op="quant", tokens=7300, slots=8192, page=16, **h),
        # one request, one token: the latency of an interactive user
        dict(name="attn4_one", op="attn4", reqs=1, new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=1000, page=16, lens=5, **h),
        # the decode step of 32 requests with contexts of all lengths
        dict(name="attn4_decode", op="attn4", reqs=32, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=8000, page=16, lens=6, **h),
        # a large decode batch with long contexts: over a GB of cache
        dict(name="attn4_decode_large", op="attn4", reqs=128, new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=16000, page=16,
             lens=7, **h),
        # chunks of long prompts over what is cached of them, and decoding requests beside them
        dict(name="attn4_chunk", op="attn4", reqs=6, new_lo=1, new_hi=700, ctx_lo=500, ctx_hi=9000, page=64, lens=9,
             heads=32, kv_heads=4, dim=64),
        # one prompt continued eight times
        dict(name="branch_few", op="branch", parents=1, copies=8, ctx_lo=777, ctx_hi=777, page=16, lens=10, **h),
        # a beam step over a batch: the dropped rows' pages come back, the kept ones are continued in their place
        dict(name="branch_many", op="branch", parents=64, copies=3, ctx_lo=100, ctx_hi=3000, page=32, lens=11, **h),
        # a small cache with holes
        dict(name="compact_small", op="compact", reqs=5, ctx_lo=10, ctx_hi=400, page=16, spare=0.5, limit=0.7, lens=12, **h),
        # a batch's cache is cut to the size that it needs
        dict(name="compact_large", op="compact", reqs=90, ctx_lo=100, ctx_hi=2500, page=32, spare=1.0, limit=0.55,
             lens=13, **h),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (1, 2, 4, 5, 7, 8, 16) if g * kv <= 40])
    return dict(heads=group * kv, kv_heads=kv, dim=rng.choice([64, 80, 128, 128]))


def draw(rng):
    op = rng.choice(["rope", "quant", "attn4", "attn4", "attn4", "branch", "compact"])
    c = dict(op=op, page=rng.choice([16, 16, 32, 64, 128]))
    c.update(_draw_heads(rng))
    if op == "rope":
        c["tokens"] = _log(rng, 1, 8192)
        c["far"] = rng.choice([1000, 40000, 1000000])
        c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2])
        c["norm"], c["pairs"], c["cache"] = rng.random() < 0.6, rng.random() < 0.3, rng.random() < 0.6
        return c
    if op == "quant":
        c["tokens"] = _log(rng, 1, 8192)
        c["slots"] = -(-(c["tokens"] + _log(rng, 1, 1000)) // c["page"]) * c["page"]
        return c
    c["lens"] = rng.randrange(1 << 20)
    if op == "branch":
        c["parents"], c["copies"] = _log(rng, 1, 64), rng.choice([1, 2, 3, 4])
        c["ctx_lo"] = _log(rng, 1, 500)
        c["ctx_hi"] = c["ctx_lo"] + _log(rng, 1, 2500)
        return c
    if op == "compact":
        c["reqs"] = _log(rng, 1, 90)
        c["ctx_lo"] = _log(rng, 1, 500)
        c["ctx_hi"] = c["ctx_lo"] + _log(rng, 1, 2000)
        c["spare"] = rng.choice([0.1, 0.5, 1.0])
        c["limit"] = rng.uniform(0.3, 1.0)
        return c
    c["ctx_lo"] = rng.choice([0, 1, _log(rng, 2, 1000)])
    c["ctx_hi"] = c["ctx_lo"] + _log(rng, 10, 15000)
    c["reqs"] = _log(rng, 1, 160)
    c["new_hi"] = rng.choice([1, 1, 1, _log(rng, 2, 12), _log(rng, 13, 700)])
    c["new_lo"] = rng.choice([0, 1, c["new_hi"]])
    # the plain form pads to the longest: its scores and its gathered cache stay affordable
    while (c["reqs"] * c["heads"] * c["new_hi"] * (c["ctx_hi"] + c["new_hi"]) > 2e9 or
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
    n = c["parents"] if c["op"] == "branch" else c["reqs"]
    new = [r.randint(c.get("new_lo", 0), c.get("new_hi", 0)) for _ in range(n)]
    if c["op"] == "attn4" and sum(new) == 0:
        new[0] = 1
    return new, [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(n)]


def _cdiv(a, b):
    return -(-a // b)


def _padded(D):
    """Elements of a head's row in the 4-bit cache."""
    return 64 if D <= 64 else 128


def _limit(c, held, pages):
    """A compacted cache's pages: between what its rows hold and what there is."""
    return held + int((1 - c["limit"]) * (pages - held))


# --- inputs ------------------------------------------------------------------

def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    op, H, Hk, D, P = c["op"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    s = dict(op=op, case=c, page=P, H=H, Hk=Hk, D=D)
    rand = lambda lo, hi, shape: torch.randint(lo, hi, shape, device="cuda", generator=g, dtype=torch.int32)  # noqa: E731

    if op in ("rope", "quant", "attn4"):
        if op == "attn4":
            new, ctx = _lengths(c)
            T = sum(new)
        else:
            T = c["tokens"]
        qkv = torch.randn(T, (H + 2 * Hk) * D, device="cuda", generator=g).to(BF16)   # the merged projection's rows
        s["T"], s["q"] = T, qkv[:, :H * D].view(T, H, D)
        s["k"] = qkv[:, H * D:(H + Hk) * D].view(T, Hk, D)
        s["v"] = qkv[:, (H + Hk) * D:].view(T, Hk, D)
    if op == "rope":
        s["pos"] = rand(0, c["far"], (T,))
        s["freq"] = (10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).float().cuda()
        s["qw"] = s["kw"] = None
        if c["norm"]:
            s["qw"] = (1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(BF16)
            s["kw"] = (1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(BF16)
        s["q_out"] = torch.empty(T, H, D, dtype=BF16, device="cuda")
        if c["cache"]:
            pages = _cdiv(T, P) + 3
            s["slot"] = torch.randperm(pages * P, device="cuda", generator=g)[:T].to(torch.int32)
            s["k_cache"] = torch.zeros(pages, Hk, P, D, dtype=BF16, device="cuda")
            s["v_cache"] = torch.zeros(pages, Hk, P, D, dtype=BF16, device="cuda")
        else:
            s["k_out"] = torch.empty(T, Hk, D, dtype=BF16, device="cuda")
    elif op == "quant":
        # rows of different sizes, as layers' keys and values have
        size = torch.exp2(torch.randint(-4, 4, (T, 1, 1), device="cuda", generator=g).float())
        s["k"], s["v"] = (s["k"] * size).to(BF16), (s["v"] * size).to(BF16)
        s["slot"] = torch.randperm(c["slots"], device="cuda", generator=g)[:T].to(torch.int32)
        s["all"] = torch.arange(c["slots"], **i32)
        s["cache"] = torch.zeros(c["slots"] // P, Hk, P // 16, 18 * _padded(D), dtype=torch.uint8, device="cuda")
        s["k_out"] = torch.empty(c["slots"], Hk, D, dtype=BF16, device="cuda")
        s["v_out"] = torch.empty(c["slots"], Hk, D, dtype=BF16, device="cuda")
    elif op == "attn4":
        total = [a + b for a, b in zip(new, ctx)]
        used = [_cdiv(a, P) for a in total]
        pages = sum(used) + 5
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32)
        s["kv_len"] = torch.tensor(total, **i32)
        s["max_new"], s["max_kv"], s["scale"] = max(new), max(total), 1.0 / math.sqrt(D)
        s["table"] = _table(used, max(used) + 3, torch.randperm(pages, device="cuda", generator=g).to(torch.int32))
        Dp = _padded(D)
        s["cache"] = torch.randint(0, 256, (pages, Hk, P // 16, 18 * Dp), device="cuda", generator=g, dtype=torch.uint8)
        for at in (8 * Dp, 17 * Dp):   # scales of 0.19 to 0.94, those of values of size 1
            s["cache"][..., at:at + Dp] = torch.randint(100, 116, (pages, Hk, P // 16, Dp), device="cuda", generator=g,
                                                        dtype=torch.uint8)
        s["o"] = torch.empty(T, H, D, dtype=BF16, device="cuda")
        s["lse"] = torch.empty(T, H, dtype=torch.float32, device="cuda")
    elif op == "branch":
        _, ctx = _lengths(c)
        n, m = c["parents"], c["copies"]
        whole, part = [x // P for x in ctx], [int(x % P > 0) for x in ctx]
        # every parent's pages, then a page of their own for the rows' unfinished ones, then free ones
        fresh = sum(part) * m
        pages = sum(whole) + sum(part) + fresh + 7
        order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        used = [a + b for a, b in zip(whole, part)]
        width = max(used) + 2
        at = sum(used)
        mine = order[at:at + fresh].sort().values
        s["free"] = torch.cat([mine, order[at + fresh:]]).contiguous()   # the rows' own pages go back to their places
        s["head"] = torch.full((1,), fresh, **i32)
        table = _table(used, width, order)
        rows, k = [table], 0
        for i in range(n):
            for _ in range(m):
                row = table[i].clone()
                if part[i]:
                    row[whole[i]] = mine[k]
                    k += 1
                rows.append(row[None])
        s["table"] = torch.cat(rows).contiguous()
        s["ctx"] = torch.tensor(ctx + [x for x in ctx for _ in range(m)], **i32)
        s["parent"] = torch.arange(n, **i32).repeat_interleave(m).contiguous()
        s["child"] = torch.arange(n, n + n * m, **i32)
        s["ref"] = torch.zeros(pages, **i32)
        shared = torch.cat([table[i, :whole[i]] for i in range(n)]).long()
        s["ref"][shared] = m
        s["src"], s["dst"] = torch.empty(n * m, **i32), torch.empty(n * m, **i32)
        s["pages"] = pages
    else:
        _, ctx = _lengths(c)
        used = [_cdiv(x, P) for x in ctx]
        held = sum(used)
        pages = held + max(2, int(c["spare"] * held))
        order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        s["table"] = _table(used, max(used) + 2, order)
        s["ctx"] = torch.tensor(ctx, **i32)
        s["ref"] = torch.zeros(pages, **i32)
        s["free"] = order[held:].contiguous()
        s["head"] = torch.zeros(1, **i32)
        s["limit"], s["pages"] = _limit(c, held, pages), pages
        room = min(held, pages - held)
        s["out"] = dict(table=torch.empty_like(s["table"]), ref=torch.empty_like(s["ref"]), free=torch.empty_like(s["free"]),
                        head=torch.empty_like(s["head"]), src=torch.empty(room, **i32), dst=torch.empty(room, **i32))
    if op in ("branch", "compact"):
        s["k_cache"] = torch.randn(s["pages"], Hk, P, D, device="cuda", generator=g, dtype=BF16)
        s["v_cache"] = torch.randn(s["pages"], Hk, P, D, device="cuda", generator=g, dtype=BF16)
    if own:   # the workspace that a serving program keeps
        from segmented_gemm_gb300 import attn as A
        from segmented_gemm_gb300 import kv as KV
        if op == "attn4":
            s["ws"] = KV.Kv4Workspace(T, c["reqs"], H, Hk, D)
        elif op in ("rope", "quant"):
            s["ws"] = A.AttnWorkspace(T, 1)
        else:
            s["ws"] = KV.PagesWorkspace(s["pages"])
        if op in ("quant", "attn4"):
            s["cache4"] = KV.Kv4Cache(s["cache"], P, D)
    return s


def _table(used, width, order):
    """Block tables of rows that hold used[r] pages each, drawn from `order` in turn."""
    first = np.concatenate([[0], np.cumsum(used)])[:-1, None]
    col = np.arange(width)[None, :]
    idx = torch.from_numpy(np.where(col < np.array(used)[:, None], first + col, -1)).cuda()
    return torch.where(idx >= 0, order[idx.clamp(min=0)], torch.full_like(idx, -1, dtype=torch.int32)).to(torch.int32)


# --- one pass ----------------------------------------------------------------

def run(s):
    op = s["op"]
    if own:
        from segmented_gemm_gb300 import kv as KV
        if op == "rope":
            cache = s["case"]["cache"]
            KV.lora_qk_rope(s["q"], s["k"], s["pos"], s["freq"], s["ws"], q_weight=s["qw"], k_weight=s["kw"],
                            interleaved=s["case"]["pairs"], q_out=s["q_out"], k_out=None if cache else s["k_out"],
                            **(dict(v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"], slot_map=s["slot"]) if cache
                               else {}))
        elif op == "quant":
            KV.lora_kv4_store(s["k"], s["v"], s["cache4"], s["slot"], s["ws"])
            KV.lora_kv4_load(s["cache4"], s["all"], s["ws"], k=s["k_out"], v=s["v_out"])
        elif op == "attn4":
            KV.lora_kv4_attn(s["q"], s["cache4"], s["table"], s["cu"], s["kv_len"], s["scale"], s["ws"], o=s["o"],
                             lse=s["lse"])
        elif op == "branch":
            KV.lora_kv_release(s["child"], s["ctx"], s["table"], s["ref"], s["free"], s["head"], s["page"], s["ws"])
            KV.lora_kv_fork(s["parent"], s["child"], s["ctx"], s["table"], s["ref"], s["free"], s["head"], s["page"],
                            s["ws"], copy_src=s["src"], copy_dst=s["dst"])
            KV.lora_kv_copy(s["src"], s["dst"], s["k_cache"], s["v_cache"], s["ws"])
        else:
            o = s["out"]
            KV.lora_kv_compact(s["ctx"], s["table"], s["ref"], s["free"], s["head"], s["page"], s["limit"], s["ws"],
                               copy_src=o["src"], copy_dst=o["dst"], table_out=o["table"], ref_out=o["ref"],
                               free_out=o["free"], head_out=o["head"])
            KV.lora_kv_copy(o["src"], o["dst"], s["k_cache"], s["v_cache"], s["ws"])
    else:
        dict(rope=_plain_rope, quant=_plain_quant, attn4=_plain_attn4, branch=_plain_branch, compact=_plain_compact)[op](s)
    if op == "rope":
        return dict(q=s["q_out"], **(dict(k_cache=s["k_cache"], v_cache=s["v_cache"]) if s["case"]["cache"]
                                     else dict(k=s["k_out"])))
    if op == "quant":
        return dict(k=s["k_out"], v=s["v_out"])     # the values that the cache stands for, all of them
    if op == "attn4":
        return dict(o=s["o"], lse=s["lse"])
    cache = dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    if op == "branch":
        return dict(table=s["table"], ctx=s["ctx"], ref=s["ref"], free=s["free"], head=s["head"], src=s["src"],
                    dst=s["dst"], **cache)
    return dict(**s["out"], **cache)


def _plain_rope(s):
    c, rot = s["case"], s["case"]["rot"]
    angle = s["pos"].double()[:, None] * s["freq"].double()[None, :]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        y = x.clone()
        if c["pairs"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return y.to(BF16)

    s["q_out"].copy_(turned(s["q"], s["qw"]))
    k = turned(s["k"], s["kw"])
    if c["cache"]:
        slot, P = s["slot"].long(), s["page"]
        s["k_cache"][slot // P, :, slot % P] = k
        s["v_cache"][slot // P, :, slot % P] = s["v"]
    else:
        s["k_out"].copy_(k)


# A 4-bit tile is 16 keys of one head: [16][Dp / 2] bytes of key codes (two to a byte, the first in the low half),
# [16][Dp / 16] key scales, the value codes in the order (key / 8, d / (Dp / 8), key / 2 mod 4, 8 of d, key mod 2, d),
# and the value scales in the order (d / 16, key / 2 mod 4, key / 8, key mod 2).  A scale byte is a number with five
# bits of exponent and three of fraction, a 16-bit float's bits 14 to 7.

def _codes(x):
    """Codes (0 to 15) and scale bytes of x [..., Dp], for every 16 elements."""
    x = x.unflatten(-1, (-1, 16))
    a = x.abs().amax(-1) / 6
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -14)))
    step = torch.exp2(e - 3)                                                  # 2^-17 below 2^-14
    scale = (torch.round(a / step) * step).clamp(max=10240.0)                 # to the nearest, ties to even
    bits = (scale.to(torch.float16).view(torch.int16).to(torch.int32) >> 7).to(torch.uint8)
    y = torch.where(scale[..., None] > 0, x.abs() / scale[..., None], torch.zeros_like(x))
    code = ((y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5))
    code = code + 8 * ((x < 0) & (scale[..., None] > 0)).int()
    return code.flatten(-2).to(torch.uint8), bits


def _values(codes, scales):
    """fp32 of codes [..., Dp] and scale bytes [..., Dp / 16]."""
    v = torch.tensor(VALUES + tuple(-x for x in VALUES), device=codes.device)[codes.long()]
    f = (scales.to(torch.int32) << 7).to(torch.int16).view(torch.float16).float()
    return (v.unflatten(-1, (-1, 16)) * f[..., None]).flatten(-2)


def _unpack(tiles, Dp):
    """fp32 keys and values [..., 16, Dp] of tiles [..., 18 Dp]."""
    kc, ks, vc, vs = tiles.split([8 * Dp, Dp, 8 * Dp, Dp], -1)
    kc = torch.stack([kc & 15, kc >> 4], -1).flatten(-2).unflatten(-1, (16, Dp))
    k = _values(kc, ks.unflatten(-1, (16, Dp // 16)))
    vc = torch.stack([vc & 15, vc >> 4], -1).flatten(-2).unflatten(-1, (2, 8, 4, Dp // 64, 2, 8))
    n = vc.dim() - 6
    lead = tuple(range(n))
    vc = vc.permute(*lead, n, n + 2, n + 4, n + 1, n + 3, n + 5).flatten(n + 3).flatten(n, n + 2)
    vs = vs.unflatten(-1, (Dp // 16, 4, 2, 2)).permute(*lead, n + 2, n + 1, n + 3, n).flatten(n, n + 2)
    return k, _values(vc, vs)


def _plain_quant(s):
    P, D, Dp, cache = s["page"], s["D"], _padded(s["D"]), s["cache"]
    slot = s["slot"].long()[:, None, None]
    page, tile, key = slot // P, slot % P // 16, slot % 16
    head = torch.arange(s["Hk"], device=slot.device)[None, :, None]
    dev = slot.device
    for x, at in ((s["k"], 0), (s["v"], 9 * Dp)):
        codes, scales = _codes(torch.nn.functional.pad(x.float(), (0, Dp - D)))
        byte = codes[..., 0::2] | (codes[..., 1::2] << 4)
        b, e = torch.arange(Dp // 2, device=dev), torch.arange(Dp // 16, device=dev)
        if at == 0:
            place, scale_place = key * (Dp // 2) + b, 8 * Dp + key * (Dp // 16) + e
        else:
            lane, j = b // (Dp // 16), b % (Dp // 16)
            place = at + ((((key // 8) * 8 + lane) * 4 + key % 8 // 2) * (Dp // 64) + j // 4) * 8 + key % 2 * 4 + j % 4
            scale_place = 17 * Dp + (e * 4 + key % 8 // 2) * 4 + key // 8 * 2 + key % 2
        cache[page, head, tile, place] = byte
        cache[page, head, tile, scale_place] = scales
    k, v = _unpack(cache, Dp)                                                 # [pages, Hk, P / 16, 16, Dp]
    s["k_out"].copy_(k[..., :D].flatten(2, 3).transpose(1, 2).flatten(0, 1))
    s["v_out"].copy_(v[..., :D].flatten(2, 3).transpose(1, 2).flatten(0, 1))


def _plain_attn4(s):
    # requests padded to the longest, the packed rows and the cache gathered into them
    dev, R, P, D = s["cu"].device, s["case"]["reqs"], s["page"], s["D"]
    cu, kv_len = s["cu"].long(), s["kv_len"].long()
    at = torch.arange(s["max_new"], device=dev)
    n = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + at[None, :]).clamp(max=s["T"] - 1)                     # [R, Lq]
    t = s["table"][:, :_cdiv(s["max_kv"], P)].long().clamp(min=0)
    k, v = _unpack(s["cache"][t], _padded(D))                                     # [R, pages, Hk, P / 16, 16, Dp]
    k = k[..., :D].transpose(1, 2).flatten(2, 4)                                  # [R, Hk, Lk, D]
    v = v[..., :D].transpose(1, 2).flatten(2, 4)
    Hk = k.shape[1]
    G, Lq, Lk = s["H"] // Hk, s["max_new"], k.shape[2]
    q = s["q"][row].float().view(R, Lq, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(R, Hk, G * Lq, D)
    p = torch.matmul(q, k.transpose(2, 3)).view(R, Hk, G, Lq, Lk)
    p.mul_(s["scale"])
    limit = (kv_len - n)[:, None] + at[None, :] + 1                               # keys each row sees
    seen = torch.arange(Lk, device=dev)[None, None, :] < limit[:, :, None]        # [R, Lq, Lk]
    p.masked_fill_(~seen[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True).clamp(min=-3e38)                                 # a row that sees nothing: zeros
    p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, Hk, G * Lq, Lk), v).view(R, Hk, G, Lq, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))
    # back to the packed rows
    req = torch.repeat_interleave(torch.arange(R, device=dev), n, output_size=s["T"])
    local = torch.arange(s["T"], device=dev) - cu[req]
    s["o"].copy_(o.permute(0, 3, 1, 2, 4).reshape(R, Lq, Hk * G, D)[req, local])
    s["lse"].copy_(lse.permute(0, 3, 1, 2, 4).reshape(R, Lq, Hk * G)[req, local])


def _plain_branch(s):
    P, table, dev = s["page"], s["table"], s["table"].device
    col = torch.arange(table.shape[1], device=dev)[None, :]
    num = s["ref"].numel()
    # the dropped rows' pages: one holder less each, and free where none is left
    child, parent = s["child"].long(), s["parent"].long()
    held = col < ((s["ctx"][child].long() + P - 1) // P)[:, None]
    count = torch.zeros(num + 1, dtype=torch.int32, device=dev)
    count.index_add_(0, torch.where(held, table[child].long(), num).flatten(), torch.ones_like(held, dtype=torch.int32).flatten())
    count = count[:num]
    gone = count > s["ref"]
    place = torch.cumsum(gone, 0) - 1
    freed = gone.sum()
    first = s["head"].long() - freed
    free = torch.cat([s["free"], s["free"][:1]])                                  # the last place takes what is not freed
    free[torch.where(gone, first + place, s["free"].numel())] = torch.arange(num, dtype=torch.int32, device=dev)
    s["free"].copy_(free[:-1])
    s["ref"].sub_(torch.where(gone, s["ref"], count))
    # the kept rows' whole pages are shared, their unfinished ones copied into fresh pages
    length = s["ctx"][parent].long()
    whole, part = length // P, length % P > 0
    rows = table[parent].long()
    shared = col < whole[:, None]
    fresh = free[torch.where(part, first + torch.cumsum(part, 0) - 1, 0)]
    count = torch.zeros(num + 1, dtype=torch.int32, device=dev)
    count.index_add_(0, torch.where(shared, rows, num).flatten(), torch.ones_like(shared, dtype=torch.int32).flatten())
    s["ref"].add_(count[:num])
    unfinished = (col == whole[:, None]) & part[:, None]
    table[child] = torch.where(shared, rows.int(), torch.where(unfinished, fresh[:, None], table[child]))
    s["ctx"][child] = length.int()
    s["head"].copy_(first + part.sum())
    last = torch.gather(rows, 1, whole.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    s["src"].copy_(torch.where(part, last, -1))
    s["dst"].copy_(torch.where(part, fresh, -1))
    _plain_copy(s, s["src"], s["dst"])


def _plain_copy(s, src, dst):
    """A pair of -1 copies nothing: it writes what the page 0 of the other pairs gets, or what page 0 has."""
    on = src >= 0
    to = dst.long()
    at = torch.arange(s["pages"], device=src.device)
    comes = torch.cat([at, at[:1]])
    comes[torch.where(on, to, s["pages"])] = src.long()                           # for every page, the one whose rows it gets
    comes = comes[:-1]
    moved = torch.zeros(s["pages"] + 1, dtype=torch.bool, device=src.device)
    moved[torch.where(on, to, s["pages"])] = True
    order = torch.sort(moved[:-1].int(), descending=True, stable=True).indices[:src.numel()]   # the pages that change, and some that do not
    for c in (s["k_cache"], s["v_cache"]):
        c[order] = c[comes[order]]


def _plain_compact(s):
    o, P, L, table, dev = s["out"], s["page"], s["limit"], s["table"], s["table"].device
    num, room = s["pages"], o["src"].numel()
    held = torch.arange(table.shape[1], device=dev)[None, :] < ((s["ctx"].long() + P - 1) // P)[:, None]
    used = torch.zeros(num + 1, dtype=torch.bool, device=dev)
    used[torch.where(held, table.long(), num)] = True
    used = used[:num]
    free = torch.zeros(num + 1, dtype=torch.bool, device=dev)
    listed_ = torch.arange(s["free"].numel(), device=dev) >= s["head"]
    free[torch.where(listed_, s["free"].long(), num)] = True
    free = free[:num]
    at = torch.arange(num, device=dev)
    hole, mover = free & (at < L), used & (at >= L)
    hole_rank, mover_rank = torch.cumsum(hole, 0) - 1, torch.cumsum(mover, 0) - 1
    moved = torch.minimum(hole.sum(), mover.sum()).clamp(max=room)
    taken, left = hole & (hole_rank < moved), mover & (mover_rank < moved)
    dst = torch.full((room + 1,), -1, dtype=torch.int32, device=dev)
    src = dst.clone()
    dst[torch.where(taken, hole_rank, room)] = at.int()
    src[torch.where(left, mover_rank, room)] = at.int()
    o["dst"].copy_(dst[:room])
    o["src"].copy_(src[:room])
    new = torch.where(left, dst[torch.where(left, mover_rank, room)], at.int())
    o["table"].copy_(torch.where(held, new[torch.where(held, table.long(), 0)], table))
    on = o["src"] >= 0
    ref = torch.cat([s["ref"], s["ref"][:1]])
    ref[torch.where(on, o["dst"].long(), num)] = s["ref"][torch.where(on, o["src"].long(), 0)]
    ref[torch.where(on, o["src"].long(), num)] = 0
    o["ref"].copy_(ref[:num])
    still = (free & ~taken) | left
    count = still.sum()
    n = s["free"].numel()
    out = torch.cat([s["free"], s["free"][:1]])
    out[torch.where(still, n - count + torch.cumsum(still, 0) - 1, n)] = at.int()
    o["free"].copy_(out[:n])
    o["head"].copy_(n - count)
    _plain_copy(s, o["src"], o["dst"])


# --- what a pass cannot do without -------------------------------------------

def work(c):
    op, H, Hk, D, P = c["op"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    page = 2 * Hk * P * D * 2                                  # bytes of a page's keys and values in bf16
    if op == "rope":
        T = c["tokens"]
        b = T * (H + Hk) * D * 4 + T * 4 + (T * (Hk * D * 4 + 4) if c["cache"] else 0)
        return dict(bytes=b, flops=0)
    if op == "quant":
        row = 2 * Hk * (D // 2 + D // 16)                      # a token's codes and scales
        return dict(bytes=c["tokens"] * (4 * Hk * D + 4 + row) + c["slots"] * (row + 4 * Hk * D + 4), flops=0)
    new, ctx = _lengths(c)
    if op == "attn4":
        T = sum(new)
        kv = [(a + b) if a else 0 for a, b in zip(new, ctx)]   # a request without new tokens is not read
        pairs = sum(n * x + n * (n + 1) // 2 for n, x in zip(new, ctx))
        return dict(bytes=2 * T * H * D * 2 + T * H * 4 + sum(kv) * 2 * Hk * (D // 2 + D // 16) +
                    4 * sum(_cdiv(x, P) for x in kv), flops=4 * D * H * pairs)
    if op == "branch":
        copies = c["copies"] * sum(x % P > 0 for x in ctx)
        entries = c["copies"] * sum(_cdiv(x, P) for x in ctx)
        # a row's entries read to be released, the parent's read, its own and the counts written (twice); the pages
        return dict(bytes=4 * entries * 7 + 2 * copies * page, flops=0)
    held = sum(_cdiv(x, P) for x in ctx)
    pages = held + max(2, int(c["spare"] * held))
    moved = max(0, held * (pages - _limit(c, held, pages)) // pages)              # about so many, the pages being random
    return dict(bytes=4 * (2 * held + 2 * pages + 2 * (pages - held)) + 2 * moved * page, flops=0)


# --- the definition in 64 bits -----------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(c, s)
    if c["op"] == "quant":
        return _exact_quant(c, s)
    if c["op"] == "attn4":
        return _exact_attn4(c, s)
    kc, vc = s["k_cache"], s["v_cache"]
    if c["op"] == "branch":
        out = _exact_branch(c, s)
    else:
        out = _exact_compact(c, s)
    pairs = [(a, b) for a, b in zip(out["src"].tolist(), out["dst"].tolist()) if a >= 0]
    if pairs:
        src, dst = (torch.tensor(x, device="cuda") for x in zip(*pairs))
        kc[dst], vc[dst] = kc[src], vc[src]
    return dict(out, k_cache=kc.double(), v_cache=vc.double())


def _exact_rope(c, s):
    rot, D = c["rot"], c["dim"]
    first = torch.arange(0, rot, 2) if c["pairs"] else torch.arange(rot // 2)
    other = first + (1 if c["pairs"] else rot // 2)
    # the rotation as a complex factor for each pair of elements
    turn = torch.polar(torch.ones(s["T"], rot // 2, dtype=torch.float64, device="cuda"),
                       s["pos"].double()[:, None] * s["freq"].double())[:, None]
    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + 1e-6) * w.double()
        z = torch.complex(x[..., first], x[..., other]) * turn
        y = x.clone()
        y[..., first], y[..., other] = z.real, z.imag
        return y
    q, k = turned(s["q"], s["qw"]), turned(s["k"], s["kw"])
    if not c["cache"]:
        return dict(q=q, k=k)
    pages, P = s["k_cache"].shape[0], c["page"]
    out = []
    for x in (k, s["v"].double()):
        flat = torch.zeros(pages * P, c["kv_heads"], D, dtype=torch.float64, device="cuda")
        flat[s["slot"].long()] = x
        out.append(flat.view(pages, P, c["kv_heads"], D).transpose(1, 2))
    return dict(q=q, k_cache=out[0], v_cache=out[1])


def _exact_quant(c, s):
    grid = torch.tensor(VALUES, dtype=torch.float64, device="cuda")
    # every scale there is, in ascending order: 0, multiples of 2^-17 up to 2^-14, then eight to a power of two
    scales = torch.tensor([m * 2.0 ** -17 for m in range(8)] +
                          [(1 + m / 8) * 2.0 ** (e - 15) for e in range(1, 31) for m in range(8)], dtype=torch.float64)
    scales = scales[scales <= 10240].cuda()

    def nearest(x, to):
        """The entry of `to` nearest to x; ties go to the entry of even place."""
        hi = torch.searchsorted(to, x.contiguous()).clamp(1, to.numel() - 1)
        lo = hi - 1
        up, down = to[hi] - x, x - to[lo]
        return to[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]

    out = []
    for x in (s["k"].double(), s["v"].double()):
        x = torch.nn.functional.pad(x, (0, -c["dim"] % 16)).unflatten(-1, (-1, 16))
        f = nearest(x.abs().amax(-1, keepdim=True) / 6, scales)
        y = torch.where(f > 0, torch.sign(x) * nearest((x.abs() / f.clamp(min=1e-30)).clamp(max=6), grid) * f, torch.zeros_like(x))
        flat = torch.zeros(c["slots"], c["kv_heads"], c["dim"], dtype=torch.float64, device="cuda")
        flat[s["slot"].long()] = y.flatten(-2)[..., :c["dim"]]
        out.append(flat)
    return dict(k=out[0], v=out[1])


def _exact_attn4(c, s):
    new, ctx = _lengths(c)
    H, Hk, D, P, Dp = c["heads"], c["kv_heads"], c["dim"], c["page"], _padded(c["dim"])
    # where a key's or value's element lies in its tile, and the scale that goes with it
    key, d = torch.arange(16, device="cuda")[:, None], torch.arange(D, device="cuda")[None, :]
    k_at, k_scale = key * (Dp // 2) + d // 2, 8 * Dp + key * (Dp // 16) + d // 16
    w = Dp // 8
    v_at = (9 * Dp + (key // 8) * 4 * Dp + (d // w) * (Dp // 2) + (key % 8 // 2) * w + (d % w // 8) * 8 + (key % 2) * 4 +
            d % 8 // 2)
    v_scale = 17 * Dp + d // 16 * 16 + (key % 8 // 2) * 4 + (key // 8) * 2 + key % 2
    grid = torch.tensor(VALUES, dtype=torch.float64, device="cuda")

    def read(tiles, at, scale):                                # tiles [n, bytes] -> [16 n, D]
        nib = tiles[:, at].long() >> (4 * (d % 2)) & 15
        b = tiles[:, scale].double()
        e, m = torch.floor(b / 8), b % 8
        f = torch.where(e > 0, torch.exp2(e - 15) * (1 + m / 8), m * 2.0 ** -17)
        return (torch.where(nib >= 8, -grid[nib % 8], grid[nib % 8]) * f).flatten(0, 1)

    o = torch.zeros(s["T"], H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], H), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for r, (n, x) in enumerate(zip(new, ctx)):
        if n == 0:
            continue
        pages = s["cache"][s["table"][r, :_cdiv(n + x, P)].long()]
        for h in range(Hk):
            k, v = read(pages[:, h].flatten(0, 1), k_at, k_scale), read(pages[:, h].flatten(0, 1), v_at, v_scale)
            cols = slice(h * (H // Hk), (h + 1) * (H // Hk))
            for b in range(0, n, 512):                         # blocks of queries against the keys that they see
                e = min(n, b + 512)
                keys = x + e
                hidden = torch.arange(keys, device="cuda")[None, :] > x + torch.arange(b, e, device="cuda")[:, None]
                q = s["q"][t0 + b:t0 + e, cols].double()
                sc = torch.einsum("qgd,kd->qgk", q, k[:keys]) * s["scale"]
                sc = sc.masked_fill(hidden[:, None], -math.inf)
                lse[t0 + b:t0 + e, cols] = torch.logsumexp(sc, -1)
                o[t0 + b:t0 + e, cols] = torch.einsum("qgk,kd->qgd", torch.softmax(sc, -1), v[:keys])
        t0 += n
    return dict(o=o, lse=lse)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _exact_branch(c, s):
    P, table, ctx = c["page"], s["table"].tolist(), s["ctx"].tolist()
    ref, free, head = s["ref"].tolist(), s["free"].tolist(), int(s["head"])
    parent, child = s["parent"].tolist(), s["child"].tolist()
    freed = []
    for r in child:
        for p in table[r][:_cdiv(ctx[r], P)]:
            if ref[p] == 0:
                freed.append(p)
            else:
                ref[p] -= 1
        ctx[r] = 0
    head -= len(freed)
    free[head:head + len(freed)] = sorted(freed)
    src, dst = [], []
    for a, r in zip(parent, child):
        whole = ctx[a] // P
        for j in range(whole):
            table[r][j] = table[a][j]
            ref[table[a][j]] += 1
        if ctx[a] % P:
            src.append(table[a][whole])
            dst.append(free[head])
            table[r][whole] = free[head]
            head += 1
        else:
            src.append(-1)
            dst.append(-1)
        ctx[r] = ctx[a]
    return dict(table=_i32(table), ctx=_i32(ctx), ref=_i32(ref), free=_i32(free), head=_i32([head]), src=_i32(src),
                dst=_i32(dst))


def _exact_compact(c, s):
    P, L, table, ctx = c["page"], s["limit"], s["table"].tolist(), s["ctx"].tolist()
    ref, free, head, room = s["ref"].tolist(), s["free"].tolist(), int(s["head"]), s["out"]["src"].numel()
    holes = sorted(p for p in free[head:] if p < L)
    movers = sorted({p for r, x in enumerate(ctx) for p in table[r][:_cdiv(x, P)] if p >= L})
    pairs = list(zip(movers, holes))[:room]
    to = dict(pairs)
    for r, x in enumerate(ctx):
        for j in range(_cdiv(x, P)):
            table[r][j] = to.get(table[r][j], table[r][j])
    for a, b in pairs:
        ref[b], ref[a] = ref[a], 0
    left = sorted(set(free[head:]) - set(to.values()) | set(to))
    head = len(free) - len(left)
    free[head:] = left
    pad = [-1] * (room - len(pairs))
    return dict(table=_i32(table), ref=_i32(ref), free=_i32(free), head=_i32([head]), src=_i32([a for a, _ in pairs] + pad),
                dst=_i32([b for _, b in pairs] + pad))
