"""CPU checks of include/lora_attn.h's boundary: symbols, sizes and refusals.
No compute call runs here."""
import ctypes
import os
import re

import pytest
import torch

from segmented_gemm_gb300 import attn as A
from segmented_gemm_gb300 import lora as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "lora_attn.h")).read()


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from segmented_gemm_gb300 import build
        build.build()
    return A._lib()


def test_every_declared_symbol_is_exported_by_both_builds(lib):
    src = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    names = set(re.findall(r"\b(lora_[a-z_]+)\s*\(", src))
    assert names == set(A.EXPORTS)
    dbg = ctypes.CDLL(L.DEBUG_LIB_PATH)
    for n in names:
        assert hasattr(lib, n) and hasattr(dbg, n), n


def test_constants_match_the_header():
    bits = {m.group(1): 1 << int(m.group(2)) for m in re.finditer(r"\b(LORA_DEV_[A-Z_]+)\s*=\s*1\s*<<\s*(\d+)", HEADER)}
    assert set(bits) == {"LORA_DEV_BAD_LENGTH", "LORA_DEV_NO_PAGE", "LORA_DEV_BAD_PAGE"}
    for name, v in bits.items():
        assert getattr(A, name) == v
    assert not any(v & (L.LORA_DEV_BAD_ID | L.LORA_DEV_TIMEOUT | L.LORA_DEV_BAD_POOL | L.LORA_DEV_CHECK)
                   for v in bits.values())
    for name in ("LORA_MAX_REQUESTS", "LORA_MAX_HEAD_DIM", "LORA_MAX_GROUP"):
        assert int(re.search(rf"#define {name} (\d+)", HEADER).group(1)) == getattr(A, name)


def test_workspace_sizes(lib):
    size = A.lora_attn_workspace_size
    assert 0 < size(32, 32) < size(32, 32, 32, 8, 128) < size(16384, 32, 32, 8, 128)
    for args in ((-1, 1), (1, -1), (1, 5000), (1 << 31, 1), (8, 1, 32, 0, 128), (8, 1, 32, 5, 128), (8, 1, 32, 8, 136),
                 (8, 1, 32, 8, 12), (8, 1, 129, 1, 64)):
        assert size(*args) == 0, args
    with pytest.raises(ValueError):
        A.AttnWorkspace(8, 1, 32, 5, 128, device="cpu")


def cache(**kw):
    c = A.lora_kv_cache_t(0x1000, 0x2000, 2 * 16 * 64, 16 * 64, 64, 10, 16, 2, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def attn(**kw):
    a = A.lora_attn_t(0x1000, 0x2000, 0x3000, 0x4000, 256, 64, 256, 64, 8, 2, 4, 2, 64, 0.125)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_CACHES = [(dict(k=None), L.LORA_ERR_NULL), (dict(v=0x2008), L.LORA_ERR_ALIGN), (dict(head_dim=12), L.LORA_ERR_SHAPE),
              (dict(head_dim=136), L.LORA_ERR_SHAPE), (dict(page_size=12), L.LORA_ERR_SHAPE),
              (dict(page_size=4), L.LORA_ERR_SHAPE), (dict(page_size=8192), L.LORA_ERR_SHAPE),
              (dict(num_pages=0), L.LORA_ERR_SHAPE), (dict(num_pages=1 << 27), L.LORA_ERR_SHAPE),
              (dict(slot_stride=60), L.LORA_ERR_SHAPE), (dict(page_stride=0), L.LORA_ERR_SHAPE),
              (dict(head_stride=-64), L.LORA_ERR_SHAPE), (dict(kv_heads=0), L.LORA_ERR_SHAPE)]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_bad_caches_are_refused(lib, change, code):
    c = cache(**change)
    assert lib.lora_kv_store(0x1000, 0x1000, 4, 128, 64, 128, 64, ctypes.addressof(c), 0x1000, 0x100, 1 << 30,
                             None) == code
    a = attn()
    rc = lib.lora_attn_paged(ctypes.addressof(a), ctypes.addressof(c), 0x1000, 4, 4, 0x1000, None, 0x100, 1 << 30, None)
    assert rc in (code, L.LORA_ERR_SHAPE) and rc != L.LORA_OK


@pytest.mark.parametrize("change,code", [
    (dict(q=None), L.LORA_ERR_NULL), (dict(o=None), L.LORA_ERR_NULL), (dict(cu=None), L.LORA_ERR_NULL),
    (dict(q=0x1008), L.LORA_ERR_ALIGN), (dict(lse=0x3002), L.LORA_ERR_ALIGN), (dict(heads=5), L.LORA_ERR_SHAPE),
    (dict(heads=0), L.LORA_ERR_SHAPE), (dict(head_dim=192), L.LORA_ERR_SHAPE), (dict(num_tokens=-1), L.LORA_ERR_SHAPE),
    (dict(num_requests=5000), L.LORA_ERR_SHAPE), (dict(scale=0.0), L.LORA_ERR_SHAPE),
    (dict(scale=float("nan")), L.LORA_ERR_SHAPE), (dict(scale=float("inf")), L.LORA_ERR_SHAPE),
    (dict(q_token_stride=252), L.LORA_ERR_SHAPE), (dict(o_head_stride=0), L.LORA_ERR_SHAPE),
])
def test_bad_attention_arguments_are_refused(lib, change, code):
    a, c = attn(**change), cache()
    assert lib.lora_attn_paged(ctypes.addressof(a), ctypes.addressof(c), 0x1000, 4, 4, 0x1000, None, 0x100, 1 << 30,
                               None) == code
    assert lib.lora_attn_prompt(ctypes.addressof(a), 0x1000, 128, 64, 0x1000, 128, 64, None, 0x100, 1 << 30,
                                None) == code


def test_workspace_tables_and_empty_steps(lib):
    a, c = attn(), cache()
    A_, C_ = ctypes.addressof(a), ctypes.addressof(c)
    F = lib.lora_attn_paged
    assert F(A_, C_, 0x1000, 4, 4, 0x1000, None, None, 1 << 30, None) == L.LORA_ERR_WORKSPACE
    assert F(A_, C_, 0x1000, 4, 4, 0x1000, None, 0x100, 64, None) == L.LORA_ERR_WORKSPACE
    assert F(A_, C_, 0x1000, 4, 4, 0x1000, None, 0x110, 1 << 30, None) == L.LORA_ERR_ALIGN
    assert F(A_, C_, None, 4, 4, 0x1000, None, 0x100, 1 << 30, None) == L.LORA_ERR_NULL
    assert F(A_, C_, 0x1000, 4, 4, None, None, 0x100, 1 << 30, None) == L.LORA_ERR_NULL
    assert F(A_, C_, 0x1000, -1, 4, 0x1000, None, 0x100, 1 << 30, None) == L.LORA_ERR_SHAPE
    assert F(A_, C_, 0x1000, 4, 3, 0x1000, None, 0x100, 1 << 30, None) == L.LORA_ERR_SHAPE   # rows overlap
    c2 = cache(head_dim=128, slot_stride=128)
    assert F(A_, ctypes.addressof(c2), 0x1000, 4, 4, 0x1000, None, 0x100, 1 << 30, None) == L.LORA_ERR_SHAPE
    for empty in (attn(num_tokens=0), attn(num_requests=0)):
        assert F(ctypes.addressof(empty), C_, None, 0, 0, None, None, None, 0, None) == L.LORA_OK
        assert lib.lora_attn_prompt(ctypes.addressof(empty), None, 128, 64, None, 128, 64, None, None, 0,
                                    None) == L.LORA_OK
    assert lib.lora_kv_store(None, None, 0, 128, 64, 128, 64, C_, None, None, 0, None) == L.LORA_OK
    assert lib.lora_kv_store(None, 0x1000, 4, 128, 64, 128, 64, C_, 0x1000, 0x100, 1 << 20, None) == L.LORA_ERR_NULL
    out = A.lora_attn_sched_t()
    S = lib.lora_attn_schedule
    assert S(0x1000, None, 2, 8, 8, 4, 2, 64, None, 0x100, 1 << 30, None) == L.LORA_ERR_NULL
    assert S(None, None, 2, 8, 8, 4, 2, 64, ctypes.addressof(out), 0x100, 1 << 30, None) == L.LORA_ERR_NULL
    assert S(0x1000, None, 2, 8, -1, 4, 2, 64, ctypes.addressof(out), 0x100, 1 << 30, None) == L.LORA_ERR_SHAPE
    assert S(0x1000, None, 2, 8, 8, 4, 3, 64, ctypes.addressof(out), 0x100, 1 << 30, None) == L.LORA_ERR_SHAPE


@pytest.mark.parametrize("change,code", [
    (dict(num_requests=-1), L.LORA_ERR_SHAPE), (dict(max_tokens=-1), L.LORA_ERR_SHAPE),
    (dict(page_size=24), L.LORA_ERR_SHAPE), (dict(num_pages=0), L.LORA_ERR_SHAPE),
    (dict(table_width=1 << 28), L.LORA_ERR_SHAPE), (dict(table_stride=3), L.LORA_ERR_SHAPE),
    (dict(free_head=None), L.LORA_ERR_NULL), (dict(new_len=None), L.LORA_ERR_NULL),
    (dict(block_table=None), L.LORA_ERR_NULL), (dict(slot_map=None), L.LORA_ERR_NULL),
    (dict(free_pages=None), L.LORA_ERR_NULL), (dict(lora_id_map=None), L.LORA_ERR_NULL),
    (dict(free_head_out=0x9000), L.LORA_ERR_SHAPE), (dict(kv_len=0x2000), L.LORA_ERR_SHAPE),
    (dict(num_free=-1), L.LORA_ERR_SHAPE),
])
def test_bad_plans_are_refused(lib, change, code):
    p = A.lora_kv_plan_t(0x1000, 0x2000, 0x3000, 2, 0x4000, 4, 4, 0x8000, 5, 0x9000, 16, 10, 8, 0xA000, 0xB000, 0xC000,
                         0xD000, 0xE000, 0xF000)
    for k, v in change.items():
        setattr(p, k, v)
    assert lib.lora_kv_plan(ctypes.addressof(p), 0x100, 1 << 20, None) == code
    assert lib.lora_kv_plan(None, 0x100, 1 << 20, None) == L.LORA_ERR_NULL


def test_binding_refuses_what_the_kernels_cannot_address():
    f = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        A._rows(f, "q")                                        # not bf16, not on the device
    with pytest.raises(ValueError):
        A._ints(torch.zeros(4, dtype=torch.int32), 4, "cu")    # host memory
    with pytest.raises(ValueError):
        A._cache(f, f)
