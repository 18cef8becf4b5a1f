"""CPU checks of include/lora_kv.h's boundary (symbols, sizes, refusals) and of
the plain implementations that the GPU tests compare with.  No compute call
of the library runs here."""
import ctypes
import itertools
import os
import re
import sys

import pytest
import torch

from segmented_gemm_gb300 import attn as A
from segmented_gemm_gb300 import kv as KV
from segmented_gemm_gb300 import lora as L

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import kv_reference as ref  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "lora_kv.h")).read()
WS, BIG = 0x100, 1 << 40   # an aligned address that is never touched, and room enough


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from segmented_gemm_gb300 import build
        build.build()
    A._lib()
    return KV._lib()


def test_every_declared_symbol_is_exported_by_both_builds(lib):
    src = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    names = set(re.findall(r"\b(lora_[a-z0-9_]+)\s*\(", src))
    assert names == set(KV.EXPORTS)
    dbg = ctypes.CDLL(L.DEBUG_LIB_PATH)
    for n in names:
        assert hasattr(lib, n) and hasattr(dbg, n), n


def test_status_bit_is_its_own():
    bit = 1 << int(re.search(r"LORA_DEV_BAD_ROW = 1 << (\d+)", HEADER).group(1))
    assert bit == KV.LORA_DEV_BAD_ROW
    assert not bit & (L.LORA_DEV_BAD_ID | L.LORA_DEV_TIMEOUT | L.LORA_DEV_BAD_POOL | L.LORA_DEV_CHECK |
                      A.LORA_DEV_BAD_LENGTH | A.LORA_DEV_NO_PAGE | A.LORA_DEV_BAD_PAGE)


def test_sizes(lib):
    assert KV.lora_kv4_block_size(16, 128) == 2304 and KV.lora_kv4_block_size(64, 64) == 4 * 1152
    assert KV.lora_kv4_block_size(16, 80) == 2304 and KV.lora_kv4_block_size(16, 8) == 1152
    for args in ((8, 64), (24, 64), (8192, 64), (16, 136), (16, 12), (16, 0)):
        assert KV.lora_kv4_block_size(*args) == 0, args
    size = lib.lora_kv4_workspace_size
    assert 0 < size(32, 32, 32, 8, 128, 0) < size(4096, 8, 32, 8, 128, 4096) < size(4096, 8, 32, 8, 128, 65536)
    for args in ((-1, 1, 8, 2, 64, 0), (1, 5000, 8, 2, 64, 0), (1, 1, 8, 3, 64, 0), (1, 1, 8, 2, 136, 0),
                 (1, 1, 8, 2, 64, -1), (1, 1, 8, 2, 64, 1 << 25)):
        assert size(*args) == 0, args
    # room for the largest step is room for every smaller one
    for T, R in itertools.product((1, 7, 100, 512, 4096), (1, 3, 64, 512)):
        assert size(T, R, 32, 8, 128, 8192) <= size(4096, 512, 32, 8, 128, 8192), (T, R)
    pages = lib.lora_kv_pages_workspace_size
    assert 0 < pages(1) <= pages(100000) and pages(0) == 0 and pages(-1) == 0 and pages(1 << 28) == 0
    with pytest.raises(ValueError):
        KV.PagesWorkspace(0, device="cpu")
    with pytest.raises(ValueError):
        KV.Kv4Workspace(8, 1, 32, 5, 128, device="cpu")


_alive = []


def ptr(x):
    """The address of a structure, which stays."""
    _alive.append(x)
    return ctypes.addressof(x)


def rope(**kw):
    a = KV.lora_qk_rope_t()
    vals = dict(q=0x1000, k=0x2000, v=0x3000, q_out=0x4000, k_out=0x5000, q_weight=0x6000, k_weight=0x7000,
                position=0x8000, inv_freq=0x9000, slot_map=0xA000, q_token_stride=256, q_head_stride=64,
                k_token_stride=128, k_head_stride=64, v_token_stride=128, v_head_stride=64, qo_token_stride=256,
                qo_head_stride=64, ko_token_stride=128, ko_head_stride=64, num_tokens=8, heads=4, kv_heads=2, head_dim=64,
                rot_dim=64, interleaved=0, eps=1e-6)
    vals.update(kw)
    for k, v in vals.items():
        setattr(a, k, v)
    return a


def cache(**kw):
    c = A.lora_kv_cache_t(0x1000, 0x2000, 2 * 16 * 64, 16 * 64, 64, 10, 16, 2, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("change,code", [
    (dict(q=None), L.LORA_ERR_NULL), (dict(k=None), L.LORA_ERR_NULL), (dict(q_out=None), L.LORA_ERR_NULL),
    (dict(v=None), L.LORA_ERR_NULL), (dict(slot_map=None), L.LORA_ERR_NULL), (dict(position=None), L.LORA_ERR_NULL),
    (dict(inv_freq=None), L.LORA_ERR_NULL), (dict(q=0x1008), L.LORA_ERR_ALIGN), (dict(k_weight=0x7008), L.LORA_ERR_ALIGN),
    (dict(position=0x8002), L.LORA_ERR_ALIGN), (dict(inv_freq=0x9001), L.LORA_ERR_ALIGN),
    (dict(head_dim=136), L.LORA_ERR_SHAPE), (dict(head_dim=60), L.LORA_ERR_SHAPE), (dict(rot_dim=72), L.LORA_ERR_SHAPE),
    (dict(rot_dim=12), L.LORA_ERR_SHAPE), (dict(rot_dim=-8), L.LORA_ERR_SHAPE), (dict(heads=-1), L.LORA_ERR_SHAPE),
    (dict(kv_heads=3), L.LORA_ERR_SHAPE), (dict(num_tokens=-1), L.LORA_ERR_SHAPE), (dict(eps=-1.0), L.LORA_ERR_SHAPE),
    (dict(eps=float("nan")), L.LORA_ERR_SHAPE), (dict(q_token_stride=252), L.LORA_ERR_SHAPE),
    (dict(ko_head_stride=0), L.LORA_ERR_SHAPE), (dict(v_token_stride=-8), L.LORA_ERR_SHAPE),
    (dict(q_out=0x1000, qo_token_stride=512), L.LORA_ERR_SHAPE), (dict(k_out=0x2000, ko_head_stride=72), L.LORA_ERR_SHAPE),
])
def test_bad_rotations_are_refused(lib, change, code):
    assert lib.lora_qk_rope(ptr(rope(**change)), ptr(cache()), WS, BIG, None) == code


def test_rotation_workspace_cache_and_empty_calls(lib):
    F, a = lib.lora_qk_rope, ptr(rope())
    assert F(None, None, WS, BIG, None) == L.LORA_ERR_NULL
    assert F(a, None, None, BIG, None) == L.LORA_ERR_WORKSPACE
    assert F(a, None, WS, 64, None) == L.LORA_ERR_WORKSPACE
    assert F(a, None, 0x110, BIG, None) == L.LORA_ERR_ALIGN
    assert F(a, ptr(cache(page_size=12)), WS, BIG, None) == L.LORA_ERR_SHAPE
    assert F(a, ptr(cache(k=None)), WS, BIG, None) == L.LORA_ERR_NULL
    assert F(ptr(rope(k_out=None)), None, WS, BIG, None) == L.LORA_ERR_NULL   # nowhere to go
    assert F(ptr(rope(num_tokens=0, q=None, k=None)), None, None, 0, None) == L.LORA_OK
    assert F(ptr(rope(heads=0, kv_heads=0, q=None, k=None)), None, None, 0, None) == L.LORA_OK


def cache4(**kw):
    c = KV.lora_kv4_cache_t(0x1000, 2 * 2304, 2304, 10, 16, 2, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def attn(**kw):
    a = A.lora_attn_t(0x1000, 0x2000, 0x3000, 0x4000, 512, 128, 512, 128, 8, 2, 4, 2, 128, 0.125)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,code", [
    (dict(data=None), L.LORA_ERR_NULL), (dict(data=0x1008), L.LORA_ERR_ALIGN), (dict(head_dim=132), L.LORA_ERR_SHAPE),
    (dict(head_dim=136), L.LORA_ERR_SHAPE), (dict(page_size=8), L.LORA_ERR_SHAPE), (dict(page_size=48), L.LORA_ERR_SHAPE),
    (dict(page_size=8192), L.LORA_ERR_SHAPE), (dict(num_pages=0), L.LORA_ERR_SHAPE),
    (dict(num_pages=1 << 27), L.LORA_ERR_SHAPE), (dict(page_stride=100), L.LORA_ERR_SHAPE),
    (dict(page_stride=0), L.LORA_ERR_SHAPE), (dict(head_stride=-16), L.LORA_ERR_SHAPE),
    (dict(head_stride=1 << 36), L.LORA_ERR_SHAPE), (dict(kv_heads=0), L.LORA_ERR_SHAPE),
])
def test_bad_4_bit_caches_are_refused(lib, change, code):
    c, a = ptr(cache4(**change)), ptr(attn())
    assert lib.lora_kv4_store(0x1000, 0x1000, 4, 256, 128, 256, 128, c, 0x1000, WS, BIG, None) == code
    assert lib.lora_kv4_load(c, 0x1000, 4, 0x1000, 0x1000, 256, 128, 256, 128, WS, BIG, None) == code
    assert lib.lora_kv4_copy(0x1000, 0x1000, 4, c, WS, BIG, None) == code
    assert lib.lora_kv4_attn(a, c, 0x1000, 4, 4, 0x1000, 0, WS, BIG, None) == code


def test_4_bit_calls_refuse_bad_arguments(lib):
    c_, a = ptr(cache4()), ptr(attn())
    S, G, F, C = lib.lora_kv4_store, lib.lora_kv4_load, lib.lora_kv4_attn, lib.lora_kv4_copy
    assert S(None, 0x1000, 4, 256, 128, 256, 128, c_, 0x1000, WS, BIG, None) == L.LORA_ERR_NULL
    assert S(0x1000, 0x1000, 4, 256, 128, 256, 128, c_, None, WS, BIG, None) == L.LORA_ERR_NULL
    assert S(0x1000, 0x1008, 4, 256, 128, 256, 128, c_, 0x1000, WS, BIG, None) == L.LORA_ERR_ALIGN
    assert S(0x1000, 0x1000, 4, 252, 128, 256, 128, c_, 0x1000, WS, BIG, None) == L.LORA_ERR_SHAPE
    assert S(0x1000, 0x1000, -1, 256, 128, 256, 128, c_, 0x1000, WS, BIG, None) == L.LORA_ERR_SHAPE
    assert S(0x1000, 0x1000, 4, 256, 128, 256, 128, c_, 0x1000, None, BIG, None) == L.LORA_ERR_WORKSPACE
    assert S(None, None, 0, 256, 128, 256, 128, c_, None, None, 0, None) == L.LORA_OK
    assert G(c_, None, 4, 0x1000, 0x1000, 256, 128, 256, 128, WS, BIG, None) == L.LORA_ERR_NULL
    assert G(c_, 0x1000, 4, 0x1008, 0x1000, 256, 128, 256, 128, WS, BIG, None) == L.LORA_ERR_ALIGN
    assert G(c_, 0x1000, 4, 0x1000, 0x1000, 256, 0, 256, 128, WS, BIG, None) == L.LORA_ERR_SHAPE
    assert G(c_, None, 4, None, None, 0, 0, 0, 0, None, 0, None) == L.LORA_OK
    assert F(a, c_, 0x1000, 4, 4, 0x1000, -1, WS, BIG, None) == L.LORA_ERR_SHAPE
    assert F(a, c_, 0x1000, 4, 3, 0x1000, 0, WS, BIG, None) == L.LORA_ERR_SHAPE      # rows overlap
    assert F(a, c_, 0x1000, -1, 4, 0x1000, 0, WS, BIG, None) == L.LORA_ERR_SHAPE
    assert F(a, c_, None, 4, 4, 0x1000, 0, WS, BIG, None) == L.LORA_ERR_NULL
    assert F(a, c_, 0x1000, 4, 4, None, 0, WS, BIG, None) == L.LORA_ERR_NULL
    assert F(a, c_, 0x1000, 4, 4, 0x1002, 0, WS, BIG, None) == L.LORA_ERR_ALIGN
    assert F(a, c_, 0x1000, 4, 4, 0x1000, 0, WS, 4096, None) == L.LORA_ERR_WORKSPACE
    assert F(a, c_, 0x1000, 4, 4, 0x1000, 0, 0x110, BIG, None) == L.LORA_ERR_ALIGN
    assert F(ptr(attn(head_dim=64, q_head_stride=64)), c_, 0x1000, 4, 4, 0x1000, 0, WS, BIG,
             None) == L.LORA_ERR_SHAPE
    for bad in (dict(q=None), dict(cu=None)):
        assert F(ptr(attn(**bad)), c_, 0x1000, 4, 4, 0x1000, 0, WS, BIG, None) == L.LORA_ERR_NULL
    assert F(ptr(attn(num_tokens=(1 << 31) - 200, heads=8)), c_, 0x1000, 4, 4, 0x1000, 0, WS, BIG,
             None) == L.LORA_ERR_SHAPE                                               # rows past 32 bits
    for empty in (attn(num_tokens=0), attn(num_requests=0)):
        assert F(ptr(empty), c_, None, 0, 0, None, 0, None, 0, None) == L.LORA_OK
    assert C(None, 0x1000, 4, c_, WS, BIG, None) == L.LORA_ERR_NULL
    assert C(0x1000, 0x1001, 4, c_, WS, BIG, None) == L.LORA_ERR_ALIGN
    assert C(0x1000, 0x1000, -4, c_, WS, BIG, None) == L.LORA_ERR_SHAPE
    assert C(None, None, 0, c_, None, 0, None) == L.LORA_OK
    b = ptr(cache())
    assert lib.lora_kv_copy(0x1000, 0x1000, 4, b, None, BIG, None) == L.LORA_ERR_WORKSPACE
    assert lib.lora_kv_copy(0x1000, None, 4, b, WS, BIG, None) == L.LORA_ERR_NULL
    assert lib.lora_kv_copy(0x1000, 0x1000, 4, ptr(cache(head_dim=12)), WS, BIG, None) == L.LORA_ERR_SHAPE


@pytest.mark.parametrize("change,code", [
    (dict(block_table=None), L.LORA_ERR_NULL), (dict(ctx_len=None), L.LORA_ERR_NULL), (dict(ref=None), L.LORA_ERR_NULL),
    (dict(free_pages=None), L.LORA_ERR_NULL), (dict(free_head=None), L.LORA_ERR_NULL), (dict(ref=0x1002), L.LORA_ERR_ALIGN),
    (dict(num_rows=-1), L.LORA_ERR_SHAPE), (dict(num_rows=5000), L.LORA_ERR_SHAPE), (dict(table_width=-1), L.LORA_ERR_SHAPE),
    (dict(table_stride=3), L.LORA_ERR_SHAPE), (dict(table_width=1 << 28), L.LORA_ERR_SHAPE),
    (dict(num_free=-1), L.LORA_ERR_SHAPE), (dict(page_size=4), L.LORA_ERR_SHAPE), (dict(page_size=24), L.LORA_ERR_SHAPE),
    (dict(num_pages=0), L.LORA_ERR_SHAPE), (dict(num_pages=1 << 28), L.LORA_ERR_SHAPE),
])
def test_bad_page_states_are_refused(lib, change, code):
    p = KV.lora_kv_pages_t(0x1000, 4, 4, 3, 0x2000, 0x3000, 0x4000, 0x5000, 6, 16, 20)
    for k, v in change.items():
        setattr(p, k, v)
    a = ptr(p)
    assert lib.lora_kv_release(a, 0x6000, 2, WS, BIG, None) == code
    assert lib.lora_kv_fork(a, 0x6000, 0x7000, 2, 0x8000, 0x9000, WS, BIG, None) == code
    assert lib.lora_kv_compact(a, 10, 0x8000, 0x9000, 4, None, None, None, None, WS, BIG, None) == code


def test_page_calls_refuse_bad_arguments(lib):
    a = ptr(KV.lora_kv_pages_t(0x1000, 4, 4, 3, 0x2000, 0x3000, 0x4000, 0x5000, 6, 16, 20))
    R, K, C = lib.lora_kv_release, lib.lora_kv_fork, lib.lora_kv_compact
    assert R(None, 0x6000, 2, WS, BIG, None) == L.LORA_ERR_NULL
    assert R(a, None, 2, WS, BIG, None) == L.LORA_ERR_NULL
    assert R(a, 0x6001, 2, WS, BIG, None) == L.LORA_ERR_ALIGN
    assert R(a, 0x6000, 5000, WS, BIG, None) == L.LORA_ERR_SHAPE
    assert R(a, 0x6000, 2, WS, 256, None) == L.LORA_ERR_WORKSPACE
    assert R(a, None, 0, WS, BIG, None) == L.LORA_OK
    assert K(a, 0x6000, None, 2, 0x8000, 0x9000, WS, BIG, None) == L.LORA_ERR_NULL
    assert K(a, 0x6000, 0x7000, 2, 0x8000, None, WS, BIG, None) == L.LORA_ERR_NULL
    assert K(a, 0x6000, 0x7000, -2, 0x8000, 0x9000, WS, BIG, None) == L.LORA_ERR_SHAPE
    assert K(a, 0x6000, 0x7002, 2, 0x8000, 0x9000, WS, BIG, None) == L.LORA_ERR_ALIGN
    assert C(a, -1, 0x8000, 0x9000, 4, None, None, None, None, WS, BIG, None) == L.LORA_ERR_SHAPE
    assert C(a, 10, 0x8000, 0x9000, -1, None, None, None, None, WS, BIG, None) == L.LORA_ERR_SHAPE
    assert C(a, 10, None, 0x9000, 4, None, None, None, None, WS, BIG, None) == L.LORA_ERR_NULL
    assert C(a, 10, 0x8000, 0x9000, 4, 0x1001, None, None, None, WS, BIG, None) == L.LORA_ERR_ALIGN


def test_binding_refuses_what_the_kernels_cannot_address(lib):
    f = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        KV.lora_qk_rope(f, f, torch.zeros(4, dtype=torch.int32), None, None)     # host memory
    with pytest.raises(ValueError):
        KV.Kv4Cache(torch.zeros(3, 2, 2304, dtype=torch.uint8), 16, 128)         # host memory
    with pytest.raises(ValueError):
        KV._weight(torch.zeros(64), 64, "q_weight")
    with pytest.raises(ValueError):
        KV._pairs(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


# --- the plain implementations -------------------------------------------------

def test_reference_scales_are_the_middle_bits_of_fp16():
    bits = torch.arange(248, dtype=torch.int32) << 7
    assert torch.equal(ref.SCALES, bits.to(torch.int16).view(torch.float16).double())
    assert ref.SCALES[226] == 10240


def test_reference_quantiser_picks_the_nearest_by_trying_all():
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(40, 16, generator=g) * torch.exp2(torch.randint(-12, 12, (40, 1), generator=g).float())).to(torch.bfloat16)
    code, byte = ref.quantise(x)
    assert code.shape == (40, 64) and (code[:, 16:] == 0).all()
    for i in range(40):
        want = float(x[i].double().abs().max()) / 6
        best = min(range(227), key=lambda b: (abs(float(ref.SCALES[b]) - want), b % 2))
        assert int(byte[i, 0]) == best
        for d in range(16):
            v = float(x[i, d]) / float(ref.SCALES[best])
            c = min(range(8), key=lambda c: (abs(float(ref.GRID[c]) - abs(v)), c % 2))
            assert int(code[i, d]) == c + 8 * (v < 0)


def test_reference_tile_layout_is_a_permutation_and_reads_back():
    for D in (64, 128):
        seen = torch.zeros(18 * D, dtype=torch.long)
        for key in range(16):
            kc, ks, vc, vs = ref.places(D, key)
            for at in (kc[0::2], ks, vc[0::2], vs):
                seen[at] += 1
            assert torch.equal(kc[0::2], kc[1::2]) and torch.equal(vc[0::2], vc[1::2])
        assert (seen == 1).all()
    g = torch.Generator().manual_seed(1)
    for D in (8, 72, 128):
        tile = torch.zeros(18 * ref.padded(D), dtype=torch.uint8)
        rows = [(torch.randn(D, generator=g).to(torch.bfloat16), torch.randn(D, generator=g).to(torch.bfloat16)) for _ in range(16)]
        for key, (k, v) in enumerate(rows):
            ref.put(tile, key, k, v)
        for key, (k, v) in enumerate(rows):
            for got, row in zip(ref.get(tile, key, D), (k, v)):
                assert torch.equal(got, ref.dequantise(*ref.quantise(row))[:D])


def test_reference_pages_keep_their_books():
    import random
    rng = random.Random(2)
    rows, width, page, n = 6, 5, 8, 24
    s = ref.Pages([[-1] * width for _ in range(rows)], [0] * rows, [0] * n, list(range(n)), 0, page)
    for _ in range(300):
        what = rng.choice(["grow", "release", "fork", "compact"])
        if what == "grow":                            # as lora_kv_plan does
            r = rng.randrange(rows)
            have, new = s.held(r), rng.randrange(1, 12)
            need = -(-(s.ctx[r] + new) // page) - have
            if s.ctx[r] + new <= width * page and s.head + need <= n:
                s.table[r][have:have + need] = s.free[s.head:s.head + need]
                s.head += need
                s.ctx[r] += new
        elif what == "release":
            s.release([rng.randrange(rows)])
        elif what == "fork":
            a, b = rng.sample(range(rows), 2)
            s.release([b])
            s.fork([a], [b])
        else:
            s.compact(rng.randrange(n + 1), rng.randrange(6))
        holders = [sum(p in s.table[r][:s.held(r)] for r in range(rows)) for p in range(n)]
        assert s.ref == [max(0, h - 1) for h in holders]
        assert sorted(s.free[s.head:]) == [p for p in range(n) if holders[p] == 0]
