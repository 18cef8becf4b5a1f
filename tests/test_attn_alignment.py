"""CPU checks: an int32 array that does not start on 4 bytes is refused by every
entry point of include/lora_attn.h that reads or writes it, before anything is
launched."""
import ctypes

import pytest

from segmented_gemm_gb300 import attn as A
from segmented_gemm_gb300 import lora as L
from test_attn_boundary import attn, cache, lib  # noqa: F401  (lib: a fixture)

PLAN = dict(new_len=0x1000, ctx_len=0x2000, req_adapter=0x3000, block_table=0x4000, free_pages=0x8000, free_head=0x9000,
            cu_new=0xA000, kv_len=0xB000, slot_map=0xC000, position=0xD000, lora_id_map=0xE000, free_head_out=0xF000)


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("name", sorted(PLAN))
def test_plan(lib, name, off):  # noqa: F811
    p = A.lora_kv_plan_t(num_requests=2, table_width=4, table_stride=4, num_free=5, page_size=16, num_pages=10,
                         max_tokens=8, **PLAN)
    setattr(p, name, PLAN[name] + off)
    assert lib.lora_kv_plan(ctypes.addressof(p), 0x100, 1 << 20, None) == L.LORA_ERR_ALIGN


@pytest.mark.parametrize("off", [1, 2, 3])
def test_store_schedule_and_attention(lib, off):  # noqa: F811
    a, c, out = attn(), cache(), A.lora_attn_sched_t()
    A_, C_, S_ = ctypes.addressof(a), ctypes.addressof(c), ctypes.addressof(out)
    assert lib.lora_kv_store(0x1000, 0x1000, 4, 128, 64, 128, 64, C_, 0x1000 + off, 0x100, 1 << 30, None) == L.LORA_ERR_ALIGN
    for table, kv in ((0x1000 + off, 0x1000), (0x1000, 0x1000 + off)):
        assert lib.lora_attn_paged(A_, C_, table, 4, 4, kv, None, 0x100, 1 << 30, None) == L.LORA_ERR_ALIGN
    for cu, kv in ((0x1000 + off, 0x1000), (0x1000, 0x1000 + off), (0x1000 + off, None)):
        assert lib.lora_attn_schedule(cu, kv, 2, 8, 8, 4, 2, 64, S_, 0x100, 1 << 30, None) == L.LORA_ERR_ALIGN
    a.cu = 0x4000 + off
    assert lib.lora_attn_paged(A_, C_, 0x1000, 4, 4, 0x1000, None, 0x100, 1 << 30, None) == L.LORA_ERR_ALIGN
    assert lib.lora_attn_prompt(A_, 0x1000, 128, 64, 0x1000, 128, 64, None, 0x100, 1 << 30, None) == L.LORA_ERR_ALIGN
