"""The calls on pages (include/lora_kv.h) with caches of several sizes on one
workspace, and at the largest sizes of their lists, against plain loops."""
import os
import random
import sys

import pytest
import torch

from segmented_gemm_gb300 import kv as KV
from segmented_gemm_gb300 import lora as L

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import kv_reference as ref  # noqa: E402
from test_gpu_kv import assert_state, device_state  # noqa: E402

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def random_state(pages, rows, width, page, rng):
    """Rows of random lengths, some pages held twice, some neither held nor free."""
    order = rng.sample(range(pages), pages)
    table, ctx, at = [], [], 0
    for _ in range(rows):
        n = rng.randrange(width + 1)
        n = min(n, max(0, pages - at))
        table.append(order[at:at + n] + [-1] * (width - n))
        ctx.append(n * page - (rng.randrange(page) if n else 0))
        at += n
    ref_counts = [0] * pages
    for a, b in ((0, 1), (2, 3)):                  # the second row continues the first
        whole = min(ctx[a] // page, -(-ctx[b] // page))
        for j in range(whole):
            ref_counts[table[a][j]] += 1
            table[b][j] = table[a][j]
    held = {p for row, c in zip(table, ctx) for p in row[:-(-c // page)]}
    free = [p for p in order if p not in held and rng.random() < 0.9]
    return ref.Pages(table, ctx, ref_counts, [-1] * 50 + free, 50, page)


@pytest.mark.parametrize("sizes", [(40000, 60000, 40000, 60000, 33000), (100, 50000, 100, 50000), (70000, 70000, 1030)])
def test_one_workspace_serves_caches_of_several_sizes(sizes):
    """What a smaller cache leaves in the workspace means nothing to a larger one."""
    ws = KV.PagesWorkspace(max(sizes))
    rng = random.Random(sizes[0])
    for pages in sizes:
        rows, width, page = 64, 2 * pages // 3 // 64 + 1, 16
        s = random_state(pages, rows, width, page, rng)
        d = device_state(s)
        limit = rng.randrange(pages // 4, pages)
        src, dst = KV.lora_kv_compact(limit=limit, ws=ws, max_copies=pages, **d)
        assert L.lora_get_status(ws) == 0, pages
        assert list(zip(src.tolist(), dst.tolist())) == s.compact(limit, pages), pages
        assert_state(d, s, f"{pages} pages: compact")
        rows = rng.sample(range(64), 40)
        KV.lora_kv_release(i32(rows), ws=ws, **d)
        s.release(rows)
        assert_state(d, s, f"{pages} pages: release")
        L.lora_get_status(ws)                       # (a list without room for what comes back)


@pytest.mark.parametrize("rows,width", [(4, 40), (100, 60)])
@pytest.mark.parametrize("extra", [0, 4 * 32768, (1 << 31) - 1 - 3000])
def test_lists_longer_than_the_cache(rows, width, extra):
    """A free list whose taken part is long, up to the longest there may be (8.6 GB), and as many places for pairs as
    fit: places past 2^31 - 2^13 in it once wrapped to negative ones."""
    pages, page = 3000, 16
    s = random_state(pages, rows, width, page, random.Random(rows))
    tail = s.free
    wide = torch.empty(extra + len(tail), dtype=torch.int32, device="cuda")
    wide[extra:] = i32(tail)
    d = device_state(s)
    d["free_pages"], d["free_head"] = wide, i32([extra + s.head])
    ws = KV.PagesWorkspace(pages)
    src, dst = KV.lora_kv_compact(limit=pages // 2, ws=ws, max_copies=pages, **d)
    assert L.lora_get_status(ws) == 0
    assert list(zip(src.tolist(), dst.tolist())) == s.compact(pages // 2, pages)
    for name, want in (("ctx_len", s.ctx), ("block_table", s.table), ("ref", s.ref), ("free_head", [extra + s.head])):
        assert d[name].tolist() == want, name
    assert wide[extra + s.head:].tolist() == s.free[s.head:]


def test_places_for_more_pairs_than_32_bits_step_over():
    """max_copies of 2^31 - 1 (two arrays of 8.6 GB): the places behind the last pair are all -1."""
    pages, page, most = 3000, 16, (1 << 31) - 1
    s = random_state(pages, 4, 40, page, random.Random(2))
    d, ws = device_state(s), KV.PagesWorkspace(pages)
    src, dst = KV.lora_kv_compact(limit=pages // 2, ws=ws, max_copies=most, **d)
    assert L.lora_get_status(ws) == 0
    pairs = s.compact(pages // 2, pages)
    assert list(zip(src[:pages].tolist(), dst[:pages].tolist())) == pairs
    n = sum(a >= 0 for a, _ in pairs)
    for x in (src, dst):
        for part in x[n:].split(1 << 28):
            assert int(part.min()) == -1 and int(part.max()) == -1
