"""Python binding of include/lora_attn.h: the paged key/value cache and the
attention between a layer's LoRA projections.  Argument marshalling only; all
arithmetic runs in the library's CUDA kernels.

    plan = lora_kv_plan(new_len, ctx_len, block_table, free_pages, free_head, page_size, num_pages, ws)
    sched = lora_attn_schedule(plan.cu_new, plan.kv_len, T, max_kv, heads, kv_heads, head_dim, ws)
    # in every layer
    lora_kv_store(k, v, k_cache, v_cache, plan.slot_map, ws)
    o = lora_attn_paged(q, k_cache, v_cache, block_table, plan.cu_new, plan.kv_len, scale, ws, sched=sched)

q, k and v may be views of a merged projection's rows.  A cache is a pair of
bf16 tensors [num_pages, kv_heads, page_size, head_dim] of equal strides (a
permuted view of any order whose last dimension is contiguous fits).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .lora import LORA_OK, LoraError, load_library

LORA_DEV_BAD_LENGTH, LORA_DEV_NO_PAGE, LORA_DEV_BAD_PAGE = 1 << 8, 1 << 9, 1 << 10
LORA_MAX_REQUESTS, LORA_MAX_HEAD_DIM, LORA_MAX_GROUP = 4096, 128, 128

EXPORTS = ("lora_kv_plan", "lora_kv_store", "lora_attn_workspace_size", "lora_attn_schedule", "lora_attn_paged",
           "lora_attn_prompt")

_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class lora_kv_cache_t(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("page_stride", _I64), ("head_stride", _I64), ("slot_stride", _I64),
                ("num_pages", _I32), ("page_size", _I32), ("kv_heads", _I32), ("head_dim", _I32)]


class lora_kv_plan_t(ctypes.Structure):
    _fields_ = [("new_len", _P), ("ctx_len", _P), ("req_adapter", _P), ("num_requests", _I32), ("block_table", _P),
                ("table_width", _I32), ("table_stride", _I64), ("free_pages", _P), ("num_free", _I32),
                ("free_head", _P), ("page_size", _I32), ("num_pages", _I32), ("max_tokens", _I64), ("cu_new", _P),
                ("kv_len", _P), ("slot_map", _P), ("position", _P), ("lora_id_map", _P), ("free_head_out", _P)]


class lora_attn_t(ctypes.Structure):
    _fields_ = [("q", _P), ("o", _P), ("lse", _P), ("cu", _P), ("q_token_stride", _I64), ("q_head_stride", _I64),
                ("o_token_stride", _I64), ("o_head_stride", _I64), ("num_tokens", _I64), ("num_requests", _I32),
                ("heads", _I32), ("kv_heads", _I32), ("head_dim", _I32), ("scale", ctypes.c_float)]


class lora_attn_sched_t(ctypes.Structure):
    _fields_ = [("plan", _P), ("num_tokens", _I64), ("max_kv", _I64), ("num_requests", _I32), ("heads", _I32),
                ("kv_heads", _I32), ("head_dim", _I32), ("prompt", _I32)]


_bound = {}


def _lib():
    lib = load_library()
    f = _bound.get(lib._name)
    if f is None:
        VP, CP = ctypes.c_void_p, ctypes.c_void_p   # structures go by address
        sig = {
            "lora_kv_plan": (ctypes.c_int, [VP, _P, _SZ, _P]),
            "lora_kv_store": (ctypes.c_int, [_P, _P, _I64, _I64, _I64, _I64, _I64, CP, _P, _P, _SZ, _P]),
            "lora_attn_workspace_size": (_SZ, [_I64, _I32, _I32, _I32, _I32]),
            "lora_attn_schedule": (ctypes.c_int, [_P, _P, _I32, _I64, _I64, _I32, _I32, _I32, VP, _P, _SZ, _P]),
            "lora_attn_paged": (ctypes.c_int, [VP, CP, _P, _I32, _I64, _P, VP, _P, _SZ, _P]),
            "lora_attn_prompt": (ctypes.c_int, [VP, _P, _I64, _I64, _P, _I64, _I64, VP, _P, _SZ, _P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        f = _bound[lib._name] = lib
    return f


def _check(code: int, where: str):
    if code != LORA_OK:
        raise LoraError(code, where)


def _raw_stream(t: torch.Tensor, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _need(t: torch.Tensor, dtype, ndim: int, name: str):
    if t.dtype != dtype or t.dim() != ndim or not t.is_cuda:
        raise ValueError(f"{name}: a {ndim}-dimensional {dtype} tensor on the device")


def _ints(t: Optional[torch.Tensor], n: int, name: str) -> Optional[int]:
    """The address of a contiguous device int32 vector of at least n entries."""
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_cuda or t.dim() != 1 or t.shape[0] < n or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 vector of {n} entries on the device")
    return t.data_ptr()


def lora_attn_workspace_size(T: int, R: int, heads: int = 0, kv_heads: int = 0, head_dim: int = 0) -> int:
    return int(_lib().lora_attn_workspace_size(T, R, heads, kv_heads, head_dim))


class AttnWorkspace:
    """A zero-initialised device workspace for steps of T packed tokens and R
    requests; without head counts, for lora_kv_plan and lora_kv_store only.
    lora_get_status reads and clears its status bits."""

    def __init__(self, T: int, R: int, heads: int = 0, kv_heads: int = 0, head_dim: int = 0, device="cuda"):
        self.nbytes = lora_attn_workspace_size(T, R, heads, kv_heads, head_dim)
        if self.nbytes == 0:
            raise ValueError("AttnWorkspace: token, request or head counts out of range")
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device)

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())


class KvPlan:
    """The outputs of lora_kv_plan for up to max_tokens packed tokens of R requests."""

    def __init__(self, max_tokens: int, R: int, device="cuda"):
        def new(n):
            return torch.empty(n, dtype=torch.int32, device=device)
        self.max_tokens, self.num_requests = max_tokens, R
        self.cu_new, self.kv_len, self.free_head = new(R + 1), new(R), new(1)
        self.slot_map, self.position, self.lora_id_map = new(max_tokens), new(max_tokens), new(max_tokens)


def lora_kv_plan(new_len: torch.Tensor, ctx_len: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                 free_head: torch.Tensor, page_size: int, num_pages: int, ws: AttnWorkspace,
                 req_adapter: Optional[torch.Tensor] = None, max_tokens: Optional[int] = None,
                 out: Optional[KvPlan] = None, stream=None) -> KvPlan:
    """Block tables (filled in place) and slot map of a step, from the
    requests' new and cached lengths.  ``out`` (or ``max_tokens``) says how
    many packed tokens there is room for."""
    R = new_len.shape[0]
    if out is None:
        if max_tokens is None:
            raise ValueError("lora_kv_plan: out or max_tokens")
        out = KvPlan(max_tokens, R, new_len.device)
    _need(block_table, torch.int32, 2, "block_table")
    if block_table.shape[0] != R or (block_table.shape[1] > 1 and block_table.stride(1) != 1) or out.num_requests != R:
        raise ValueError("lora_kv_plan: one table row and one output a request, rows contiguous")
    T = out.max_tokens
    a = lora_kv_plan_t(
        _ints(new_len, R, "new_len"), _ints(ctx_len, R, "ctx_len"), _ints(req_adapter, R, "req_adapter"), R,
        block_table.data_ptr(), block_table.shape[1], block_table.stride(0),
        _ints(free_pages, 0, "free_pages"), free_pages.shape[0], _ints(free_head, 1, "free_head"), page_size, num_pages,
        T, out.cu_new.data_ptr(), out.kv_len.data_ptr(), out.slot_map.data_ptr(), out.position.data_ptr(),
        out.lora_id_map.data_ptr() if req_adapter is not None else None, out.free_head.data_ptr())
    _check(_lib().lora_kv_plan(ctypes.addressof(a), ws.buf.data_ptr(), ws.nbytes, _raw_stream(new_len, stream)),
           "lora_kv_plan")
    return out


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor) -> lora_kv_cache_t:
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(v_cache, torch.bfloat16, 4, "v_cache")
    s = k_cache.stride()
    if v_cache.shape != k_cache.shape or v_cache.stride() != s or s[3] != 1:
        raise ValueError("k_cache, v_cache: [pages, kv_heads, page_size, head_dim] of equal strides, last contiguous")
    n, h, p, d = k_cache.shape
    return lora_kv_cache_t(k_cache.data_ptr(), v_cache.data_ptr(), s[0], s[1], s[2], n, p, h, d)


def _rows(t: torch.Tensor, name: str):
    """[tokens, heads, head_dim] bf16: token and head strides."""
    _need(t, torch.bfloat16, 3, name)
    s = t.stride()
    if s[2] != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    return s[0], s[1]


def lora_kv_store(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  slot_map: torch.Tensor, ws: AttnWorkspace, stream=None):
    """Write k, v [T, kv_heads, head_dim] into the cache's slots slot_map [T]
    (-1: skipped)."""
    c = _cache(k_cache, v_cache)
    ks, vs = _rows(k, "k"), _rows(v, "v")
    if v.shape != k.shape or k.shape[1] != c.kv_heads or k.shape[2] != c.head_dim:
        raise ValueError("lora_kv_store: k and v are [T, kv_heads, head_dim] of the cache")
    _check(_lib().lora_kv_store(k.data_ptr(), v.data_ptr(), k.shape[0], ks[0], ks[1], vs[0], vs[1], ctypes.addressof(c),
                                _ints(slot_map, k.shape[0], "slot_map"), ws.buf.data_ptr(), ws.nbytes,
                                _raw_stream(k, stream)), "lora_kv_store")


def lora_attn_schedule(cu: torch.Tensor, kv_len: Optional[torch.Tensor], T: int, max_kv: int, heads: int, kv_heads: int,
                       head_dim: int, ws: AttnWorkspace, stream=None) -> lora_attn_sched_t:
    """The step's work list for cu [R + 1] and kv_len [R] (None: whole
    prompts, max_kv = T), built in ws; it serves every layer of the step."""
    R = cu.shape[0] - 1
    out = lora_attn_sched_t()
    _check(_lib().lora_attn_schedule(_ints(cu, 1, "cu"), _ints(kv_len, R, "kv_len"), R, T, max_kv, heads, kv_heads,
                                     head_dim, ctypes.addressof(out), ws.buf.data_ptr(), ws.nbytes,
                                     _raw_stream(cu, stream)), "lora_attn_schedule")
    return out


def _attn(q, kv_heads, cu, scale, o, lse):
    qs = _rows(q, "q")
    T, H, D = q.shape
    if o is None:
        o = torch.empty(T, H, D, dtype=torch.bfloat16, device=q.device)
    os_ = _rows(o, "o")
    if o.shape != q.shape:
        raise ValueError("o: the shape of q")
    lp = None
    if lse is not None:
        if lse.dtype != torch.float32 or lse.shape != (T, H) or not lse.is_contiguous() or not lse.is_cuda:
            raise ValueError("lse: contiguous float32 [tokens, heads] on the device")
        lp = lse.data_ptr()
    return lora_attn_t(q.data_ptr(), o.data_ptr(), lp, _ints(cu, 1, "cu"), qs[0], qs[1], os_[0], os_[1], T,
                       cu.shape[0] - 1, H, kv_heads, D, scale), o


def lora_attn_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    cu: torch.Tensor, kv_len: torch.Tensor, scale: float, ws: AttnWorkspace,
                    sched: Optional[lora_attn_sched_t] = None, o: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of the step's new tokens q [T, heads, head_dim] over the
    paged cache: rows [cu[r], cu[r+1]) against request r's kv_len[r] keys,
    causal.  ``lse``: fp32 [T, heads], written when given."""
    c = _cache(k_cache, v_cache)
    a, o = _attn(q, c.kv_heads, cu, scale, o, lse)
    _need(block_table, torch.int32, 2, "block_table")
    if (block_table.shape[0] < a.num_requests or (block_table.shape[1] > 1 and block_table.stride(1) != 1) or
            a.head_dim != c.head_dim):
        raise ValueError("lora_attn_paged: one contiguous table row a request, and the cache's head dimension")
    _check(_lib().lora_attn_paged(ctypes.addressof(a), ctypes.addressof(c), block_table.data_ptr(),
                                  block_table.shape[1], block_table.stride(0), _ints(kv_len, a.num_requests, "kv_len"),
                                  None if sched is None else ctypes.addressof(sched), ws.buf.data_ptr(), ws.nbytes,
                                  _raw_stream(q, stream)), "lora_attn_paged")
    return o


def lora_attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, scale: float,
                     ws: AttnWorkspace, sched: Optional[lora_attn_sched_t] = None, o: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention over packed prompts: q [T, heads, head_dim], k and v
    [T, kv_heads, head_dim], request r's rows [cu[r], cu[r+1])."""
    ks, vs = _rows(k, "k"), _rows(v, "v")
    if k.shape != v.shape or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise ValueError("lora_attn_prompt: k and v are [T, kv_heads, head_dim]")
    a, o = _attn(q, k.shape[1], cu, scale, o, lse)
    _check(_lib().lora_attn_prompt(ctypes.addressof(a), k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
                                   None if sched is None else ctypes.addressof(sched), ws.buf.data_ptr(), ws.nbytes,
                                   _raw_stream(q, stream)), "lora_attn_prompt")
    return o
