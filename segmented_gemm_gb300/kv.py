"""Python binding of include/lora_kv.h: norms and rotation of queries and keys,
the cache held in 4 bits, and the sharing, freeing and moving of pages.
Argument marshalling only; all arithmetic runs in the library's CUDA kernels.

    # in every layer, between the QKV projection and the attention (attn.py)
    q, _ = lora_qk_rope(q, k, plan.position, inv_freq, ws, q_weight, k_weight,
                        v=v, k_cache=k_cache, v_cache=v_cache, slot_map=plan.slot_map)
    # or over a cache of 4.5 bits a value
    q, k = lora_qk_rope(q, k, plan.position, inv_freq, ws, q_weight, k_weight)
    lora_kv4_store(k, v, cache4, plan.slot_map, ws)
    o = lora_kv4_attn(q, cache4, block_table, plan.cu_new, plan.kv_len, scale, ws4)
    # between steps
    lora_kv_release(rows, ctx_len, block_table, ref, free_pages, free_head, page_size, wsp)
    src, dst = lora_kv_fork(parent, child, ctx_len, block_table, ref, free_pages, free_head, page_size, wsp)
    lora_kv_copy(src, dst, k_cache, v_cache, wsp)   # in every layer
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Tuple

import torch

from . import lora as _lora
from .attn import (_BF16, _F32, _I32T, _attn, _cache, _check, _ints, _raw_stream, _rows, _table)
from .lora import _on, load_library

LORA_DEV_BAD_ROW = 1 << 11

EXPORTS = ("lora_qk_rope", "lora_kv4_block_size", "lora_kv4_store", "lora_kv4_load", "lora_kv4_workspace_size",
           "lora_kv4_attn", "lora_kv_pages_workspace_size", "lora_kv_release", "lora_kv_fork", "lora_kv_compact",
           "lora_kv_copy", "lora_kv4_copy")

_P, _I32, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class lora_qk_rope_t(ctypes.Structure):
    _fields_ = ([(n, _P) for n in ("q", "k", "v", "q_out", "k_out", "q_weight", "k_weight", "position", "inv_freq",
                                   "slot_map")] +
                [(n, _I64) for n in ("q_token_stride", "q_head_stride", "k_token_stride", "k_head_stride",
                                     "v_token_stride", "v_head_stride", "qo_token_stride", "qo_head_stride",
                                     "ko_token_stride", "ko_head_stride", "num_tokens")] +
                [(n, _I32) for n in ("heads", "kv_heads", "head_dim", "rot_dim", "interleaved")] + [("eps", _F)])


class lora_kv4_cache_t(ctypes.Structure):
    _fields_ = [("data", _P), ("page_stride", _I64), ("head_stride", _I64), ("num_pages", _I32), ("page_size", _I32),
                ("kv_heads", _I32), ("head_dim", _I32)]


class lora_kv_pages_t(ctypes.Structure):
    _fields_ = [("block_table", _P), ("table_stride", _I64), ("table_width", _I32), ("num_rows", _I32), ("ctx_len", _P),
                ("ref", _P), ("free_pages", _P), ("free_head", _P), ("num_free", _I32), ("page_size", _I32),
                ("num_pages", _I32)]


# The same structures as packed bytes (see attn.py).
_ROPE = struct.Struct("@10Q11q5if")
_CACHE4 = struct.Struct("@Qqqiiii")
_PAGES = struct.Struct("@QqiiQQQQiii4x")
assert (_ROPE.size, _CACHE4.size, _PAGES.size) == tuple(
    ctypes.sizeof(t) for t in (lora_qk_rope_t, lora_kv4_cache_t, lora_kv_pages_t))

_bound = {}


def _lib():
    lib = _bound.get(_lora._active)
    if lib is None:
        lib = load_library()
        VP = ctypes.c_void_p   # structures go by address
        sig = {
            "lora_qk_rope": (ctypes.c_int, [VP, VP, _P, _SZ, _P]),
            "lora_kv4_block_size": (_SZ, [_I32, _I32]),
            "lora_kv4_store": (ctypes.c_int, [_P, _P, _I64, _I64, _I64, _I64, _I64, VP, _P, _P, _SZ, _P]),
            "lora_kv4_load": (ctypes.c_int, [VP, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _P, _SZ, _P]),
            "lora_kv4_workspace_size": (_SZ, [_I64, _I32, _I32, _I32, _I32, _I64]),
            "lora_kv4_attn": (ctypes.c_int, [VP, VP, _P, _I32, _I64, _P, _I64, _P, _SZ, _P]),
            "lora_kv_pages_workspace_size": (_SZ, [_I32]),
            "lora_kv_release": (ctypes.c_int, [VP, _P, _I32, _P, _SZ, _P]),
            "lora_kv_fork": (ctypes.c_int, [VP, _P, _P, _I32, _P, _P, _P, _SZ, _P]),
            "lora_kv_compact": (ctypes.c_int, [VP, _I32, _P, _P, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
            "lora_kv_copy": (ctypes.c_int, [_P, _P, _I32, VP, _P, _SZ, _P]),
            "lora_kv4_copy": (ctypes.c_int, [_P, _P, _I32, VP, _P, _SZ, _P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _bound[_lora._active] = lib
    return lib


def _stream(t: torch.Tensor, stream) -> int:
    return _raw_stream(t.get_device()) if stream is None else stream.cuda_stream


def _weight(w: Optional[torch.Tensor], dim: int, name: str) -> int:
    if w is None:
        return 0
    if w.dtype is not _BF16 or not w.is_cuda or w.shape != (dim,) or not w.is_contiguous():
        raise ValueError(f"{name}: contiguous bfloat16 [head_dim] on the device")
    return w.data_ptr()


def lora_qk_rope(q: torch.Tensor, k: torch.Tensor, position: torch.Tensor, inv_freq: Optional[torch.Tensor], ws,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False, v: Optional[torch.Tensor] = None, k_cache: Optional[torch.Tensor] = None,
                 v_cache: Optional[torch.Tensor] = None, slot_map: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None
                 ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Norms (where weights are given) and rotation of q [T, heads, head_dim]
    and k [T, kv_heads, head_dim] at position [T]; inv_freq: fp32 [rot_dim / 2]
    (None: no rotation).  With a cache (k_cache, v_cache, v and slot_map), keys
    and values go there too, and k_out is written when given.  q_out, k_out may
    be q and k.  Returns q_out and k_out; rows of negative position are not written."""
    shape, qs = _rows(q, "q")
    k_shape, ks = _rows(k, "k")
    T, H, D = shape
    Hk = k_shape[1]
    if k_shape[0] != T or k_shape[2] != D:
        raise ValueError("lora_qk_rope: q and k have the same tokens and head dimension")
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype is not _F32 or not inv_freq.is_cuda or inv_freq.ndim != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq: a contiguous float32 vector on the device")
        rot = 2 * inv_freq.shape[0]
    with_cache = k_cache is not None
    if with_cache != (v_cache is not None) or (with_cache and (v is None or slot_map is None)):
        raise ValueError("lora_qk_rope: k_cache, v_cache, v and slot_map go together")
    c, vs = None, (0, 0)
    if with_cache:
        c, (_, heads, _, dim) = _cache(k_cache, v_cache)
        v_shape, vs = _rows(v, "v")
        if v_shape != k_shape or heads != Hk or dim != D:
            raise ValueError("lora_qk_rope: k and v are [T, kv_heads, head_dim] of the cache")
    if q_out is None or (k_out is None and not with_cache):
        with _on(stream):
            q_out = torch.empty(shape, dtype=_BF16, device=q.device) if q_out is None else q_out
            k_out = torch.empty(k_shape, dtype=_BF16, device=q.device) if k_out is None and not with_cache else k_out
    qo_shape, qo = _rows(q_out, "q_out")
    if qo_shape != shape:
        raise ValueError("q_out: the shape of q")
    ko = (0, 0)
    if k_out is not None:
        ko_shape, ko = _rows(k_out, "k_out")
        if ko_shape != k_shape:
            raise ValueError("k_out: the shape of k")
    a = _ROPE.pack(q.data_ptr(), k.data_ptr(), v.data_ptr() if with_cache else 0, q_out.data_ptr(),
                   0 if k_out is None else k_out.data_ptr(), _weight(q_weight, D, "q_weight"),
                   _weight(k_weight, D, "k_weight"), _ints(position, T, "position"),
                   0 if inv_freq is None else inv_freq.data_ptr(), _ints(slot_map, T, "slot_map") if with_cache else 0,
                   qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], qo[0], qo[1], ko[0], ko[1], T, H, Hk, D, rot,
                   1 if interleaved else 0, eps)
    _check(_lib().lora_qk_rope(a, c, ws.addr, ws.nbytes, _stream(q, stream)), "lora_qk_rope")
    return q_out, k_out


def lora_kv4_block_size(page_size: int, head_dim: int) -> int:
    return int(_lib().lora_kv4_block_size(page_size, head_dim))


class Kv4Cache:
    """A 4-bit cache over uint8 ``data`` [num_pages, kv_heads, ...] whose trailing
    dimensions are contiguous and hold a page's head (lora_kv4_block_size bytes).
    The layout is in include/lora_kv.h."""

    def __init__(self, data: torch.Tensor, page_size: int, head_dim: int):
        size = lora_kv4_block_size(page_size, head_dim)
        if size == 0:
            raise ValueError("Kv4Cache: page_size a power of two from 16 to 4096, head_dim a multiple of 8 up to 128")
        if data.dtype is not torch.uint8 or not data.is_cuda or data.ndim < 3 or data.shape[0] < 1 or data.shape[1] < 1:
            raise ValueError("Kv4Cache: uint8 [num_pages, kv_heads, ...] on the device")
        n = 1
        for extent, step in zip(reversed(data.shape[2:]), reversed(data.stride()[2:])):
            if extent != 1 and step != n:
                raise ValueError("Kv4Cache: a page's head is contiguous")
            n *= extent
        if n != size:
            raise ValueError(f"Kv4Cache: a page's head has {size} bytes")
        self.data, self.page_size, self.head_dim = data, page_size, head_dim
        self.num_pages, self.kv_heads = data.shape[:2]
        self.packed = _CACHE4.pack(data.data_ptr(), data.stride(0), data.stride(1), self.num_pages, page_size,
                                   self.kv_heads, head_dim)

    @classmethod
    def zeros(cls, num_pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> "Kv4Cache":
        size = lora_kv4_block_size(page_size, head_dim)
        return cls(torch.zeros(num_pages, kv_heads, size, dtype=torch.uint8, device=device), page_size, head_dim)


def lora_kv4_store(k: torch.Tensor, v: torch.Tensor, cache: Kv4Cache, slot_map: torch.Tensor, ws, stream=None):
    """Write k, v [T, kv_heads, head_dim] into the 4-bit cache's slots slot_map [T] (-1: skipped)."""
    shape, ks = _rows(k, "k")
    v_shape, vs = _rows(v, "v")
    if v_shape != shape or shape[1] != cache.kv_heads or shape[2] != cache.head_dim:
        raise ValueError("lora_kv4_store: k and v are [T, kv_heads, head_dim] of the cache")
    T = shape[0]
    _check(_lib().lora_kv4_store(k.data_ptr(), v.data_ptr(), T, ks[0], ks[1], vs[0], vs[1], cache.packed,
                                 _ints(slot_map, T, "slot_map"), ws.addr, ws.nbytes, _stream(k, stream)),
           "lora_kv4_store")


def lora_kv4_load(cache: Kv4Cache, slots: torch.Tensor, ws, k: Optional[torch.Tensor] = None,
                  v: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The keys and values that slots [n] hold, bf16 [n, kv_heads, head_dim] each (-1: zeros)."""
    n = slots.shape[0]
    shape = (n, cache.kv_heads, cache.head_dim)
    if k is None or v is None:
        with _on(stream):
            k = torch.empty(shape, dtype=_BF16, device=slots.device) if k is None else k
            v = torch.empty(shape, dtype=_BF16, device=slots.device) if v is None else v
    k_shape, ks = _rows(k, "k")
    v_shape, vs = _rows(v, "v")
    if k_shape != shape or v_shape != shape:
        raise ValueError("lora_kv4_load: k and v are [n, kv_heads, head_dim] of the cache")
    _check(_lib().lora_kv4_load(cache.packed, _ints(slots, n, "slots"), n, k.data_ptr(), v.data_ptr(), ks[0], ks[1],
                                vs[0], vs[1], ws.addr, ws.nbytes, _stream(slots, stream)), "lora_kv4_load")
    return k, v


class _Workspace:
    def __init__(self, nbytes: int, what: str, device):
        if nbytes == 0:
            raise ValueError(what)
        self.nbytes = nbytes
        self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.addr = self.buf.data_ptr()

    @property
    def ptr(self):
        return ctypes.c_void_p(self.addr)


class Kv4Workspace(_Workspace):
    """A zero-initialised device workspace for lora_kv4_attn over steps of up to T
    packed tokens and R requests; serves the small calls (lora_qk_rope, lora_kv4_store,
    lora_kv4_load) too.  unpack_tokens: how many cached tokens of chunks of
    prompts it has room for in 16 bits; by default what 256 MiB hold if a step of T tokens of any number of
    requests may have chunks that take them, else none.  0 for steps of single tokens saves that."""

    def __init__(self, T: int, R: int, heads: int, kv_heads: int, head_dim: int, unpack_tokens: Optional[int] = None,
                 device="cuda"):
        size = _lib().lora_kv4_workspace_size
        if unpack_tokens is None:
            unpack_tokens = (256 << 20) // max(1, 4 * kv_heads * head_dim)
            if size(T, R, heads, kv_heads, head_dim, unpack_tokens) == size(T, R, heads, kv_heads, head_dim, 0):
                unpack_tokens = 0
        self.unpack_tokens = unpack_tokens
        super().__init__(int(size(T, R, heads, kv_heads, head_dim, unpack_tokens)),
                         "Kv4Workspace: token, request or head counts out of range", device)


class PagesWorkspace(_Workspace):
    """A zero-initialised device workspace for the calls on the pages of a cache of num_pages, or of fewer."""

    def __init__(self, num_pages: int, device="cuda"):
        self.num_pages = num_pages
        super().__init__(int(_lib().lora_kv_pages_workspace_size(num_pages)), "PagesWorkspace: num_pages out of range",
                         device)


def lora_kv4_attn(q: torch.Tensor, cache: Kv4Cache, block_table: torch.Tensor, cu: torch.Tensor, kv_len: torch.Tensor,
                  scale: float, ws: Kv4Workspace, o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """lora_attn_paged over a 4-bit cache: the step's new tokens q [T, heads,
    head_dim], rows [cu[r], cu[r+1]) against request r's kv_len[r] keys,
    causal.  ``lse``: fp32 [T, heads], written when given."""
    R = cu.shape[0] - 1
    a, o = _attn(q, cache.kv_heads, cu, R, scale, o, lse, stream)
    width, row = _table(block_table, R)
    if q.shape[2] != cache.head_dim:
        raise ValueError("lora_kv4_attn: q and the cache have the same head dimension")
    _check(_lib().lora_kv4_attn(a, cache.packed, block_table.data_ptr(), width, row, _ints(kv_len, R, "kv_len"),
                                ws.unpack_tokens, ws.addr, ws.nbytes, _stream(q, stream)), "lora_kv4_attn")
    return o


def _pages(ctx_len, block_table, ref, free_pages, free_head, page_size) -> bytes:
    """The packed lora_kv_pages_t."""
    rows = ctx_len.shape[0]
    width, row = _table(block_table, rows)
    return _PAGES.pack(block_table.data_ptr(), row, width, rows, _ints(ctx_len, rows, "ctx_len"), _ints(ref, 1, "ref"),
                       _ints(free_pages, 0, "free_pages"), _ints(free_head, 1, "free_head"), free_pages.shape[0],
                       page_size, ref.shape[0])


def lora_kv_release(rows: torch.Tensor, ctx_len: torch.Tensor, block_table: torch.Tensor, ref: torch.Tensor,
                    free_pages: torch.Tensor, free_head: torch.Tensor, page_size: int, ws: PagesWorkspace, stream=None):
    """Rows ``rows`` of the block table give up their pages; those that nobody
    else holds join the free list in front of free_head.  ref: int32
    [num_pages], holders beyond the first; everything is updated in place."""
    n = rows.shape[0]
    a = _pages(ctx_len, block_table, ref, free_pages, free_head, page_size)
    _check(_lib().lora_kv_release(a, _ints(rows, n, "rows"), n, ws.addr, ws.nbytes, _stream(rows, stream)),
           "lora_kv_release")


def lora_kv_fork(parent: torch.Tensor, child: torch.Tensor, ctx_len: torch.Tensor, block_table: torch.Tensor,
                 ref: torch.Tensor, free_pages: torch.Tensor, free_head: torch.Tensor, page_size: int,
                 ws: PagesWorkspace, copy_src: Optional[torch.Tensor] = None, copy_dst: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Row child[i] continues row parent[i]: full pages are shared, an
    unfinished one is to be copied to a fresh page.  Returns the pairs of pages
    to copy (-1 for none) for lora_kv_copy."""
    n = parent.shape[0]
    if copy_src is None or copy_dst is None:
        with _on(stream):
            copy_src = torch.empty(n, dtype=_I32T, device=parent.device) if copy_src is None else copy_src
            copy_dst = torch.empty(n, dtype=_I32T, device=parent.device) if copy_dst is None else copy_dst
    a = _pages(ctx_len, block_table, ref, free_pages, free_head, page_size)
    _check(_lib().lora_kv_fork(a, _ints(parent, n, "parent"), _ints(child, n, "child"), n, _ints(copy_src, n, "copy_src"),
                               _ints(copy_dst, n, "copy_dst"), ws.addr, ws.nbytes, _stream(parent, stream)),
           "lora_kv_fork")
    return copy_src, copy_dst


def lora_kv_compact(ctx_len: torch.Tensor, block_table: torch.Tensor, ref: torch.Tensor, free_pages: torch.Tensor,
                    free_head: torch.Tensor, page_size: int, limit: int, ws: PagesWorkspace,
                    max_copies: Optional[int] = None, copy_src: Optional[torch.Tensor] = None,
                    copy_dst: Optional[torch.Tensor] = None, table_out: Optional[torch.Tensor] = None,
                    ref_out: Optional[torch.Tensor] = None, free_out: Optional[torch.Tensor] = None,
                    head_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Moves held pages >= limit to free ones < limit, as many as there are
    (and copy_src, or max_copies, has room for; by default as many as the list has
    entries).  Returns the pairs of pages to copy (-1 behind the last) for
    lora_kv_copy.  The new state goes to the *_out arrays, or in place."""
    if copy_src is None or copy_dst is None:
        n = (max_copies if max_copies is not None else copy_src.shape[0] if copy_src is not None
             else copy_dst.shape[0] if copy_dst is not None else free_pages.shape[0])
        with _on(stream):
            copy_src = torch.empty(n, dtype=_I32T, device=ref.device) if copy_src is None else copy_src
            copy_dst = torch.empty(n, dtype=_I32T, device=ref.device) if copy_dst is None else copy_dst
    n = copy_src.shape[0] if max_copies is None else max_copies
    a = _pages(ctx_len, block_table, ref, free_pages, free_head, page_size)
    if table_out is not None and (table_out.shape != block_table.shape or table_out.stride() != block_table.stride()):
        raise ValueError("table_out: the shape and strides of block_table")
    rows = ctx_len.shape[0]
    if table_out is not None:
        _table(table_out, rows)
    _check(_lib().lora_kv_compact(a, limit, _ints(copy_src, n, "copy_src"), _ints(copy_dst, n, "copy_dst"), n,
                                  None if table_out is None else table_out.data_ptr(),
                                  _ints(ref_out, ref.shape[0], "ref_out") or None,
                                  _ints(free_out, free_pages.shape[0], "free_out") or None,
                                  _ints(head_out, 1, "head_out") or None, ws.addr, ws.nbytes, _stream(ref, stream)),
           "lora_kv_compact")
    return copy_src, copy_dst


def _pairs(src, dst):
    n = src.shape[0]
    return _ints(src, n, "src"), _ints(dst, n, "dst"), n


def lora_kv_copy(src: torch.Tensor, dst: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, ws, stream=None):
    """Copies pages src[i] of a bf16 cache to pages dst[i] (-1 in both: none)."""
    c, _ = _cache(k_cache, v_cache)
    s, d, n = _pairs(src, dst)
    _check(_lib().lora_kv_copy(s, d, n, c, ws.addr, ws.nbytes, _stream(src, stream)), "lora_kv_copy")


def lora_kv4_copy(src: torch.Tensor, dst: torch.Tensor, cache: Kv4Cache, ws, stream=None):
    """Copies pages src[i] of a 4-bit cache to pages dst[i] (-1 in both: none)."""
    s, d, n = _pairs(src, dst)
    _check(_lib().lora_kv4_copy(s, d, n, cache.packed, ws.addr, ws.nbytes, _stream(src, stream)), "lora_kv4_copy")
