"""Serving steps of a small attention-only stack with LoRA projections, run
through the library from one end to the other:

    lora_kv_plan -> lora_attn_schedule                          once a step
    lora_linear (merged QKV) -> lora_kv_store -> attention
        -> lora_linear (output projection), added to x          in every layer

    python examples/serve_attention.py [--requests 6] [--layers 2] [--steps 12] [--rope] [--bits 4]

With --rope, queries and keys get a norm for each head and are rotated by
their positions (lora_qk_rope, which also writes the cache); with --bits 4 the
cache is held in 4 bits (lora_kv4_store, lora_kv4_attn).

Each request has a LoRA adapter of its own rank, or none.  The first step
takes most requests' prompts whole (lora_attn_prompt); the last request's
prompt comes in chunks of 48 tokens in the steps after it, next to the single
tokens of the others (lora_attn_paged).  The inputs are random: a step's
outputs are not fed back.  At the end the outputs are compared with every
request recomputed from its first token in fp64 (over unquantised keys and
values: with --bits 4 the difference is the quantisation's).
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from segmented_gemm_gb300 import attn as A  # noqa: E402
from segmented_gemm_gb300 import kv as KV  # noqa: E402
from segmented_gemm_gb300 import lora as L  # noqa: E402

BF = torch.bfloat16


class Model:
    """Weights, adapters, and the device state of the serving loop."""

    def __init__(self, requests, layers, hidden, heads, kv_heads, head_dim, page, max_len, max_tokens, seed=0,
                 rope=False, bits=16):
        g = torch.Generator().manual_seed(seed)
        self.H, self.Hk, self.D, self.page, self.hidden = heads, kv_heads, head_dim, page, hidden
        self.n_qkv, self.n_o = (heads + 2 * kv_heads) * head_dim, heads * head_dim
        self.R, self.lora_scale = requests, 0.5
        # one adapter fewer than requests: the last request has none
        ranks = [16 * (1 + i % 4) for i in range(max(1, requests - 1))]

        def linear(n, k):
            def mat(rows, cols):
                return (torch.randn(rows, cols, generator=g) / math.sqrt(cols)).to(BF)
            W, As, Bs = mat(n, k), [mat(r, k) for r in ranks], [mat(n, r) for r in ranks]
            return {"W": W.cuda(), "A": As, "B": Bs, "pool": L.build_pool(As, Bs, k, n, "cuda")}

        self.layers = [(linear(self.n_qkv, hidden), linear(hidden, self.n_o)) for _ in range(layers)]
        self.adapter = torch.tensor([r if r < len(ranks) and r < requests - 1 else -1 for r in range(requests)],
                                    dtype=torch.int32, device="cuda")
        width = -(-max_len // page)
        self.num_pages, self.max_kv = requests * width, width * page
        self.bits, self.rope = bits, rope
        if bits == 4:
            self.cache = [(KV.Kv4Cache.zeros(self.num_pages, kv_heads, page, head_dim), None) for _ in range(layers)]
            self.ws4 = KV.Kv4Workspace(max_tokens, requests, heads, kv_heads, head_dim)
        else:
            self.cache = [[torch.zeros(self.num_pages, kv_heads, page, head_dim, dtype=BF, device="cuda") for _ in "kv"]
                          for _ in range(layers)]
        if rope:
            self.inv_freq = (10000.0 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)).float().cuda()
            self.norms = [[(1 + 0.1 * torch.randn(head_dim, generator=g)).to(BF).cuda() for _ in "qk"] for _ in range(layers)]
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(self.num_pages, generator=g).to(torch.int32).cuda()
        self.ctx = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.plans = [A.KvPlan(max_tokens, requests) for _ in range(2)]   # a step reads the free count of the one before
        self.plans[1].free_head.zero_()
        self.steps = 0
        self.ws = A.AttnWorkspace(max_tokens, requests, heads, kv_heads, head_dim)
        self.lws = L.Workspace(max_tokens, max(self.n_qkv, hidden), len(ranks))

    def step(self, x, new, prompts):
        """x [T, hidden] of the new tokens, new[r] of them of request r; prompts:
        no request has a token in the cache yet."""
        T, H, Hk, D = x.shape[0], self.H, self.Hk, self.D
        scale = 1.0 / math.sqrt(D)
        plan, last = self.plans[self.steps % 2], self.plans[(self.steps + 1) % 2]
        new_dev = torch.tensor(new, dtype=torch.int32).cuda()
        A.lora_kv_plan(new_dev, self.ctx, self.table, self.free, last.free_head, self.page, self.num_pages, self.ws,
                       req_adapter=self.adapter, out=plan)
        ids, slots = plan.lora_id_map[:T], plan.slot_map[:T]
        sched = A.lora_attn_schedule(plan.cu_new, None if prompts else plan.kv_len, T, T if prompts else self.max_kv,
                                     H, Hk, D, self.ws)
        for i, ((qkv, out), (kc, vc)) in enumerate(zip(self.layers, self.cache)):
            y = L.lora_linear(x, qkv["W"], None, ids, qkv["pool"], self.lora_scale, self.lws, static_weights=True)
            heads = y.unflatten(1, (H + 2 * Hk, D))
            q, k, v = heads[:, :H], heads[:, H:H + Hk], heads[:, H + Hk:]
            if self.rope:   # prompts attend over the rows themselves, so these are written too
                cache = {} if self.bits == 4 else dict(v=v, k_cache=kc, v_cache=vc, slot_map=slots)
                q, k = KV.lora_qk_rope(q, k, plan.position[:T], self.inv_freq, self.ws, *self.norms[i],
                                       k_out=torch.empty_like(k) if prompts else None, **cache)
            elif self.bits == 16:
                A.lora_kv_store(k, v, kc, vc, slots, self.ws)
            if self.bits == 4:
                KV.lora_kv4_store(k, v, kc, slots, self.ws)
            if prompts:
                o = A.lora_attn_prompt(q, k, v, plan.cu_new, scale, self.ws, sched=sched)
            elif self.bits == 4:
                o = KV.lora_kv4_attn(q, kc, self.table, plan.cu_new, plan.kv_len, scale, self.ws4)
            else:
                o = A.lora_attn_paged(q, kc, vc, self.table, plan.cu_new, plan.kv_len, scale, self.ws, sched=sched)
            x = x + L.lora_linear(o.flatten(1), out["W"], None, ids, out["pool"], self.lora_scale, self.lws,
                                  static_weights=True)
        # kv_len is 0 for a request that the plan could not give a page: none of its tokens were stored, its
        # cached ones are still there, and the caller offers the same tokens again
        self.ctx.copy_(torch.where(plan.kv_len > 0, plan.kv_len, self.ctx))
        self.steps += 1
        return x

    def recompute(self, r, x):
        """Request r's outputs from all its inputs x [n, hidden], in fp64 on the host."""
        n, H, Hk, D = x.shape[0], self.H, self.Hk, self.D
        a = int(self.adapter[r])

        def linear(w, v):
            y = v @ w["W"].cpu().double().T
            return y if a < 0 else y + self.lora_scale * (v @ w["A"][a].double().T) @ w["B"][a].double().T

        x = x.double()
        hidden_keys = torch.triu(torch.ones(n, n, dtype=torch.bool), 1)

        def turned(y, w):   # norm and rotation of rows [heads, n, D]
            y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.cpu().double()
            z = torch.complex(y[..., :D // 2], y[..., D // 2:]) * torch.polar(
                torch.ones(n, D // 2, dtype=torch.float64), torch.arange(n).double()[:, None] * self.inv_freq.cpu().double())
            return torch.cat([z.real, z.imag], -1)

        for i, (qkv, out) in enumerate(self.layers):
            h = linear(qkv, x).unflatten(1, (H + 2 * Hk, D)).transpose(0, 1)
            if self.rope:
                h = torch.cat([turned(h[:H], self.norms[i][0]), turned(h[H:H + Hk], self.norms[i][1]), h[H + Hk:]])
            q, k, v = h[:H], h[H:H + Hk].repeat_interleave(H // Hk, 0), h[H + Hk:].repeat_interleave(H // Hk, 0)
            s = (q @ k.transpose(1, 2) / math.sqrt(D)).masked_fill(hidden_keys, -math.inf)
            x = x + linear(out, (torch.softmax(s, -1) @ v).transpose(0, 1).flatten(1))
        return x


def serve(requests=6, layers=2, steps=12, hidden=512, heads=8, kv_heads=2, head_dim=64, page=16, chunk=48, seed=0,
          rope=False, bits=16):
    """Runs the loop; returns the device status and each request's relative error (Euclidean norm)."""
    g = torch.Generator().manual_seed(seed + 1)
    prompt = [1 + (37 * r + 20) % 150 for r in range(requests)]
    prompt[-1] = 2 * chunk + 5
    max_len = max(prompt) + steps + 1
    m = Model(requests, layers, hidden, heads, kv_heads, head_dim, page, max_len, sum(prompt), seed, rope, bits)
    left = list(prompt)
    xs, ys = [[] for _ in range(requests)], [[] for _ in range(requests)]
    for i in range(steps):
        if i == 0:      # whole prompts, but the last request's
            new = left[:-1] + [0]
        else:           # a token of each, and what is left of the last one's prompt by chunks
            new = [1] * (requests - 1) + [min(chunk, left[-1]) if left[-1] else 1]
        left = [max(0, a - b) for a, b in zip(left, new)]
        x = torch.randn(sum(new), hidden, generator=g).to(BF)
        y = m.step(x.cuda(), new, prompts=i == 0).cpu()
        at = 0
        for r, n in enumerate(new):
            xs[r].append(x[at:at + n])
            ys[r].append(y[at:at + n])
            at += n
    status = L.lora_get_status(m.ws) | L.lora_get_status(m.lws)
    if bits == 4:
        status |= L.lora_get_status(m.ws4)
    errors = []
    for r in range(requests):
        got, ref = torch.cat(ys[r]).double(), m.recompute(r, torch.cat(xs[r]))
        errors.append(float((got - ref).norm() / ref.norm()))
    return status, errors


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("requests", 6), ("layers", 2), ("steps", 12), ("hidden", 512), ("heads", 8), ("kv-heads", 2),
                          ("head-dim", 64), ("page", 16)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--rope", action="store_true", help="norms of queries and keys, and their rotation by position")
    ap.add_argument("--bits", type=int, default=16, choices=(4, 16), help="of a value in the cache")
    status, errors = serve(**vars(ap.parse_args()))
    print(f"device status {status}; relative error of each request against fp64: "
          + ", ".join(f"{e:.4f}" for e in errors))
    sys.exit(1 if status else 0)
