"""What a call of the binding allocates itself belongs to the stream that it runs
on, so that neither the allocator nor a caller reuses it too early."""
import os
import sys

import pytest
import torch

from segmented_gemm_gb300 import lora as L
from segmented_gemm_gb300 import workloads

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def test_outputs_of_the_projections_belong_to_their_stream():
    from test_gpu_attn_edges import stream_of
    wl = workloads.make_custom(100, 256, 256, [16, 32, 64], seed=7)
    pool = L.build_pool(wl.A, wl.B, wl.K, wl.N, "cuda")
    x, W, bias, ids = wl.x.cuda(), wl.W.cuda(), wl.bias.cuda(), wl.ids.cuda()
    ws = L.Workspace(wl.M, wl.N, len(wl.A))
    lws = L.LayersWorkspace(wl.M, wl.N, len(wl.A), 2)
    want = L.lora_linear(x, W, bias, ids, pool, wl.scale, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = L.lora_linear(x, W, bias, ids, pool, wl.scale, ws, stream=side)
    two = L.lora_linear_layers([(x, W, bias, pool, wl.scale)] * 2, ids, lws, stream=side)
    S = L.lora_shrink(x, ids, pool, ws, stream=side)
    fixed = L.lora_linear_noalloc(x, W, bias, ids, pool, wl.scale, stream=side)
    for t in (y, *two, S, fixed):
        assert stream_of(t) == side.cuda_stream
    side.synchronize()
    assert torch.equal(y, want)


def test_the_pairs_of_a_mixture_of_experts_outlive_its_call():
    """lora_moe's buffer of pairs is dropped when the call returns, while its kernels may still run."""
    from test_gpu_attn_edges import stream_of
    M, K, N, E, topk = 64, 256, 256, 4, 2
    g = torch.Generator().manual_seed(1)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
    W = (torch.randn(E, N, K, generator=g) / 16).to(torch.bfloat16).cuda()
    expert = torch.randint(0, E, (M, topk), generator=g, dtype=torch.int32).cuda()
    weight = torch.rand(M, topk, generator=g).cuda()
    ws = L.MoeWorkspace(M, topk, E)
    want = L.lora_moe(x, W, expert, weight, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()
    y = L.lora_moe(x, W, expert, weight, ws, stream=side)
    assert stream_of(y) == side.cuda_stream
    # the pairs came first out of the same fresh segment
    segs = [s for s in torch.cuda.memory_snapshot() if s["stream"] == side.cuda_stream]
    assert [s["address"] for s in segs if s["address"] < y.data_ptr() < s["address"] + s["total_size"]], segs
    side.synchronize()
    assert torch.equal(y, want)
