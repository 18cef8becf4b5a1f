"""CPU checks of the cache operators' workspaces (include/lora_kv.h): sizes and defaults."""
import itertools
import os

import pytest

from segmented_gemm_gb300 import kv as KV
from segmented_gemm_gb300 import lora as L


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from segmented_gemm_gb300 import build
        build.build()
    return KV._lib()


@pytest.mark.parametrize("T,R,H,Hk,D,room", [
    (512, 256, 32, 8, 128, True),      # a server's most: single tokens of 256 requests, or one chunk of 512
    (512, 1, 32, 8, 128, True), (200, 4096, 32, 8, 128, True),
    (199, 1, 32, 8, 128, False),       # fewer than 6400 rows of all heads
    (32, 32, 32, 8, 128, False),
    (150, 1, 64, 64, 64, False),       # no request of such a step has more than 160 rows
    (150, 1, 64, 64, 128, True),       # (96 with heads of 128)
])
def test_default_room_for_unpacked_keys(lib, T, R, H, Hk, D, room):
    ws = KV.Kv4Workspace(T, R, H, Hk, D, device="cpu")
    none = lib.lora_kv4_workspace_size(T, R, H, Hk, D, 0)
    assert (ws.unpack_tokens > 0) == room
    if room:
        assert ws.unpack_tokens == (256 << 20) // (4 * Hk * D) and ws.nbytes >= none + (256 << 20)
    else:
        assert ws.nbytes == none


def test_room_for_the_largest_step_is_room_for_every_smaller_one(lib):
    size = lib.lora_kv4_workspace_size
    for H, Hk, D in ((32, 8, 128), (64, 64, 64), (8, 1, 128), (128, 1, 64)):
        most = size(2048, 300, H, Hk, D, 8192)
        for T, R in itertools.product((1, 3, 49, 50, 51, 99, 100, 101, 150, 161, 800, 2048), (1, 2, 64, 300)):
            assert size(T, R, H, Hk, D, 8192) <= most, (H, Hk, D, T, R)
    pages = lib.lora_kv_pages_workspace_size
    sizes = [pages(n) for n in (1, 1023, 1024, 1025, 40000, 60000, 1 << 20)]
    assert sizes == sorted(sizes)
