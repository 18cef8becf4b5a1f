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
import struct
from typing import Optional

import torch

from . import lora as _lora
from .lora import LORA_OK, LoraError, _on, load_library

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


# The same structures as packed bytes: a decode step makes a handful of these
# calls a layer, and a ctypes structure costs twice as much to fill.
_CACHE = struct.Struct("@QQqqqiiii")
_PLAN = struct.Struct("@QQQi4xQi4xqQi4xQiiqQQQQQQ")
_ATTN = struct.Struct("@QQQQqqqqqiiiif4x")
assert (_CACHE.size, _PLAN.size, _ATTN.size) == tuple(
    ctypes.sizeof(t) for t in (lora_kv_cache_t, lora_kv_plan_t, lora_attn_t))

_BF16, _I32T, _F32 = torch.bfloat16, torch.int32, torch.float32
_raw_stream = torch._C._cuda_getCurrentRawStream
_bound = {}


def _lib():
    lib = _bound.get(_lora._active)
    if lib is None:
        lib = load_library()
        VP = ctypes.c_void_p   # structures go by address
        sig = {
            "lora_kv_plan": (ctypes.c_int, [VP, _P, _SZ, _P]),
            "lora_kv_store": (ctypes.c_int, [_P, _P, _I64, _I64, _I64, _I64, _I64, VP, _P, _P, _SZ, _P]),
            "lora_attn_workspace_size": (_SZ, [_I64, _I32, _I32, _I32, _I32]),
            "lora_attn_schedule": (ctypes.c_int, [_P, _P, _I32, _I64, _I64, _I32, _I32, _I32, VP, _P, _SZ, _P]),
            "lora_attn_paged": (ctypes.c_int, [VP, VP, _P, _I32, _I64, _P, VP, _P, _SZ, _P]),
            "lora_attn_prompt": (ctypes.c_int, [VP, _P, _I64, _I64, _P, _I64, _I64, VP, _P, _SZ, _P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _bound[_lora._active] = lib
    return lib


def _check(code: int, where: str):
    if code != LORA_OK:
        raise LoraError(code, where)


def _ints(t: Optional[torch.Tensor], n: int, name: str) -> int:
    """The address of a contiguous device int32 vector of at least n entries (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not _I32T or not t.is_cuda or t.ndim != 1 or t.shape[0] < n or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 vector of {n} entries on the device")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str):
    """Shape and (token, head) strides of [tokens, heads, head_dim] bf16 on the device."""
    shape, s = t.shape, t.stride()
    if len(s) != 3 or s[2] != 1 or t.dtype is not _BF16 or not t.is_cuda:
        raise ValueError(f"{name}: [tokens, heads, head_dim] bfloat16 on the device, the last dimension contiguous")
    return shape, s


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor):
    """The packed lora_kv_cache_t, and its shape."""
    shape, s = k_cache.shape, k_cache.stride()
    if (len(s) != 4 or s[3] != 1 or v_cache.shape != shape or v_cache.stride() != s or k_cache.dtype is not _BF16 or
            v_cache.dtype is not _BF16 or not k_cache.is_cuda or not v_cache.is_cuda):
        raise ValueError("k_cache, v_cache: bfloat16 [pages, kv_heads, page_size, head_dim] on the device, of equal "
                         "strides, the last dimension contiguous")
    n, h, p, d = shape
    return _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), s[0], s[1], s[2], n, p, h, d), shape


def _table(t: torch.Tensor, R: int):
    shape, s = t.shape, t.stride()
    if len(s) != 2 or shape[0] < R or (shape[1] > 1 and s[1] != 1) or t.dtype is not _I32T or not t.is_cuda:
        raise ValueError("block_table: int32 on the device, a contiguous row a request")
    return shape[1], s[0]


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
        self.addr = self.buf.data_ptr()

    @property
    def ptr(self):
        return ctypes.c_void_p(self.addr)


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
        with _on(stream):
            out = KvPlan(max_tokens, R, new_len.device)
    width, row = _table(block_table, R)
    if out.num_requests != R:
        raise ValueError("lora_kv_plan: out was made for another number of requests")
    a = _PLAN.pack(_ints(new_len, R, "new_len"), _ints(ctx_len, R, "ctx_len"), _ints(req_adapter, R, "req_adapter"), R,
                   block_table.data_ptr(), width, row, _ints(free_pages, 0, "free_pages"), free_pages.shape[0],
                   _ints(free_head, 1, "free_head"), page_size, num_pages, out.max_tokens, out.cu_new.data_ptr(),
                   out.kv_len.data_ptr(), out.slot_map.data_ptr(), out.position.data_ptr(),
                   0 if req_adapter is None else out.lora_id_map.data_ptr(), out.free_head.data_ptr())
    _check(_lib().lora_kv_plan(a, ws.addr, ws.nbytes,
                               _raw_stream(new_len.get_device()) if stream is None else stream.cuda_stream),
           "lora_kv_plan")
    return out


def lora_kv_store(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  slot_map: torch.Tensor, ws: AttnWorkspace, stream=None):
    """Write k, v [T, kv_heads, head_dim] into the cache's slots slot_map [T]
    (-1: skipped)."""
    c, (_, heads, _, dim) = _cache(k_cache, v_cache)
    shape, ks = _rows(k, "k")
    v_shape, vs = _rows(v, "v")
    if v_shape != shape or shape[1] != heads or shape[2] != dim:
        raise ValueError("lora_kv_store: k and v are [T, kv_heads, head_dim] of the cache")
    T = shape[0]
    _check(_lib().lora_kv_store(k.data_ptr(), v.data_ptr(), T, ks[0], ks[1], vs[0], vs[1], c,
                                _ints(slot_map, T, "slot_map"), ws.addr, ws.nbytes,
                                _raw_stream(k.get_device()) if stream is None else stream.cuda_stream), "lora_kv_store")


def lora_attn_schedule(cu: torch.Tensor, kv_len: Optional[torch.Tensor], T: int, max_kv: int, heads: int, kv_heads: int,
                       head_dim: int, ws: AttnWorkspace, stream=None) -> lora_attn_sched_t:
    """The step's work list for cu [R + 1] and kv_len [R] (None: whole
    prompts, max_kv = T), built in ws; it serves every layer of the step."""
    R = cu.shape[0] - 1
    out = lora_attn_sched_t()
    _check(_lib().lora_attn_schedule(_ints(cu, 1, "cu"), _ints(kv_len, R, "kv_len") or None, R, T, max_kv, heads,
                                     kv_heads, head_dim, ctypes.addressof(out), ws.addr, ws.nbytes,
                                     _raw_stream(cu.get_device()) if stream is None else stream.cuda_stream),
           "lora_attn_schedule")
    out.addr = ctypes.addressof(out)
    return out


def _attn(q, kv_heads, cu, R, scale, o, lse, stream):
    """The packed lora_attn_t, and o."""
    shape, qs = _rows(q, "q")
    if o is None:
        with _on(stream):
            o = torch.empty(shape, dtype=_BF16, device=q.device)
    o_shape, os_ = _rows(o, "o")
    if o_shape != shape:
        raise ValueError("o: the shape of q")
    T, H, D = shape
    lp = 0
    if lse is not None:
        if lse.dtype is not _F32 or lse.shape != (T, H) or not lse.is_contiguous() or not lse.is_cuda:
            raise ValueError("lse: contiguous float32 [tokens, heads] on the device")
        lp = lse.data_ptr()
    return _ATTN.pack(q.data_ptr(), o.data_ptr(), lp, _ints(cu, 1, "cu"), qs[0], qs[1], os_[0], os_[1], T, R, H, kv_heads,
                      D, scale), o


def lora_attn_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    cu: torch.Tensor, kv_len: torch.Tensor, scale: float, ws: AttnWorkspace,
                    sched: Optional[lora_attn_sched_t] = None, o: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of the step's new tokens q [T, heads, head_dim] over the
    paged cache: rows [cu[r], cu[r+1]) against request r's kv_len[r] keys,
    causal.  ``lse``: fp32 [T, heads], written when given."""
    c, (_, kv_heads, _, dim) = _cache(k_cache, v_cache)
    R = cu.shape[0] - 1
    a, o = _attn(q, kv_heads, cu, R, scale, o, lse, stream)
    width, row = _table(block_table, R)
    if q.shape[2] != dim:
        raise ValueError("lora_attn_paged: q and the cache have the same head dimension")
    _check(_lib().lora_attn_paged(a, c, block_table.data_ptr(), width, row, _ints(kv_len, R, "kv_len"),
                                  None if sched is None else sched.addr, ws.addr, ws.nbytes,
                                  _raw_stream(q.get_device()) if stream is None else stream.cuda_stream),
           "lora_attn_paged")
    return o


def lora_attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, scale: float,
                     ws: AttnWorkspace, sched: Optional[lora_attn_sched_t] = None, o: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention over packed prompts: q [T, heads, head_dim], k and v
    [T, kv_heads, head_dim], request r's rows [cu[r], cu[r+1])."""
    shape, ks = _rows(k, "k")
    v_shape, vs = _rows(v, "v")
    if v_shape != shape or q.ndim != 3 or shape[0] != q.shape[0] or shape[2] != q.shape[2]:
        raise ValueError("lora_attn_prompt: k and v are [T, kv_heads, head_dim] with q's tokens and head dimension")
    a, o = _attn(q, shape[1], cu, cu.shape[0] - 1, scale, o, lse, stream)
    _check(_lib().lora_attn_prompt(a, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
                                   None if sched is None else sched.addr, ws.addr, ws.nbytes,
                                   _raw_stream(q.get_device()) if stream is None else stream.cuda_stream),
           "lora_attn_prompt")
    return o
