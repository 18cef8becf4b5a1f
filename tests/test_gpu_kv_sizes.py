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
