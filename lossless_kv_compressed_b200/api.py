"""Python names for the C ABI, taking torch CUDA tensors.

Argument marshalling only: every step runs in libvericache.so.  torch provides
device memory, streams and events.  Shapes and layouts are those of
include/vericache.h.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import CompCache, PagedCacheStruct, check, lib


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, dtype, name: str, cuda: bool = True):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")


@dataclass
class IndexedCache:
    """Token-evicted compressed cache: bf16 base rows picked by ``idx`` with degrees.

    k, v: [B, Hkv, T_cap, D] bf16; idx, deg: [B, Hkv, S_cap] int32 or None;
    k_tail, v_tail: [B, Hkv, R_cap, D] bf16 or None with n_tail live rows."""

    k: torch.Tensor
    v: torch.Tensor
    S: int
    Hq: int
    idx: Optional[torch.Tensor] = None
    deg: Optional[torch.Tensor] = None
    k_tail: Optional[torch.Tensor] = None
    v_tail: Optional[torch.Tensor] = None
    n_tail: int = 0
    err_flag: Optional[torch.Tensor] = None

    def struct(self) -> CompCache:
        B, Hkv, T_cap, D = self.k.shape
        _need(self.k, torch.bfloat16, "k")
        _need(self.v, torch.bfloat16, "v")
        c = CompCache()
        c.kind = _lib.VC_CACHE_INDEXED
        c.B, c.Hq, c.Hkv, c.D = B, self.Hq, Hkv, D
        c.S, c.T_cap = self.S, T_cap
        c.S_cap = 0
        for t, n in ((self.idx, "idx"), (self.deg, "deg")):
            if t is not None:
                _need(t, torch.int32, n)
                c.S_cap = t.shape[-1]
        c.k, c.v = _ptr(self.k), _ptr(self.v)
        c.idx, c.deg = _ptr(self.idx), _ptr(self.deg)
        _fill_tail(c, self)
        return c


@dataclass
class Int4Cache:
    """4-bit group-quantised cache (layout in include/vericache.h).

    kq: uint32 words as int32 [B, Hkv, T_cap/32, 32, 4, D/32]; k_scale/k_zero fp16
    [B, Hkv, T_cap/32, D]; vq: int32 [B, Hkv, T_cap/32, D, 4]; v_scale/v_zero fp16
    [B, Hkv, T_cap/32, D/32, 32]; S quantised tokens live."""

    kq: torch.Tensor
    k_scale: torch.Tensor
    k_zero: torch.Tensor
    vq: torch.Tensor
    v_scale: torch.Tensor
    v_zero: torch.Tensor
    S: int
    Hq: int
    k_tail: Optional[torch.Tensor] = None
    v_tail: Optional[torch.Tensor] = None
    n_tail: int = 0
    err_flag: Optional[torch.Tensor] = None

    def struct(self) -> CompCache:
        B, Hkv, nb, D = self.k_scale.shape
        _need(self.kq, torch.int32, "kq")
        _need(self.vq, torch.int32, "vq")
        for t, n in ((self.k_scale, "k_scale"), (self.k_zero, "k_zero"),
                     (self.v_scale, "v_scale"), (self.v_zero, "v_zero")):
            _need(t, torch.float16, n)
        c = CompCache()
        c.kind = _lib.VC_CACHE_INT4
        c.B, c.Hq, c.Hkv, c.D = B, self.Hq, Hkv, D
        c.S, c.T_cap, c.S_cap = self.S, nb * 32, 0
        c.kq, c.vq = _ptr(self.kq), _ptr(self.vq)
        c.k_scale, c.k_zero = _ptr(self.k_scale), _ptr(self.k_zero)
        c.v_scale, c.v_zero = _ptr(self.v_scale), _ptr(self.v_zero)
        _fill_tail(c, self)
        return c


def _fill_tail(c: CompCache, cache) -> None:
    if cache.k_tail is not None:
        _need(cache.k_tail, torch.bfloat16, "k_tail")
        _need(cache.v_tail, torch.bfloat16, "v_tail")
        c.k_tail, c.v_tail = _ptr(cache.k_tail), _ptr(cache.v_tail)
        c.R_cap = cache.k_tail.shape[2]
    c.n_tail = cache.n_tail
    if cache.err_flag is not None:
        _need(cache.err_flag, torch.int32, "err_flag")
        c.err_flag = _ptr(cache.err_flag)


# ------------------------------------------------------------------ draft
def draft_workspace_size(cache) -> int:
    s = cache.struct()
    n = lib().vc_draft_workspace_size(ctypes.byref(s))
    if n == 0:
        check(_lib.VC_ERR_INVALID, "vc_draft_workspace_size")
    return int(n)


def _out_flag(out: torch.Tensor) -> int:
    if out.dtype == torch.float32:
        return _lib.VC_OUT_F32
    if out.dtype != torch.bfloat16:
        raise TypeError("out must be bfloat16 or float32")
    return 0


def draft_attn(q: torch.Tensor, cache, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
               scale: float = 0.0, stream=None) -> torch.Tensor:
    """o[b, h] = softmax_t(q.k_t * scale + ln n_t) . v over KV_comp plus the tail.
    ``out`` may be bfloat16 (default) or float32."""
    _need(q, torch.bfloat16, "q")
    s = cache.struct()
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = torch.empty(draft_workspace_size(cache), dtype=torch.uint8, device=q.device)
    check(lib().vc_draft_attn(q.data_ptr(), ctypes.byref(s), float(scale), _out_flag(out),
                              out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(),
                              _stream(stream)), "vc_draft_attn")
    return out


def draft_attn_noalloc(q: torch.Tensor, cache, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, scale: float = 0.0,
                       stream=None) -> torch.Tensor:
    """draft_attn for callers that cannot provide a workspace: the library keeps the
    split-K partials in a fixed 8 MiB per-device array (see vc_draft_attn_noalloc).
    Calls that overlap on the GPU share that array and must be serialised."""
    _need(q, torch.bfloat16, "q")
    s = cache.struct()
    if out is None:
        out = torch.empty_like(q)
    check(lib().vc_draft_attn_noalloc(q.data_ptr(), ctypes.byref(s), float(scale),
                                      _out_flag(out), out.data_ptr(), _ptr(lse),
                                      _stream(stream)), "vc_draft_attn_noalloc")
    return out


# ------------------------------------------------------------------ verify
def verify_workspace_size(B, n_q, Hq, Hkv, D, kv_start, kv_len) -> int:
    return int(lib().vc_verify_workspace_size(B, n_q, Hq, Hkv, D, kv_start, kv_len))


def verify_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, P: int, kv_start: int = 0,
                kv_len: Optional[int] = None, state=None, flags: int = 0,
                out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                scale: float = 0.0, stream=None) -> torch.Tensor:
    """Verify attention of q [B, n_q, Hq, D] over keys [kv_start, kv_start+kv_len) held
    in k, v [B, Hkv, L_cap, D]; ``state`` = (m, l, acc) for the chunked form.
    ``out`` may be bfloat16 (default) or float32."""
    _need(q, torch.bfloat16, "q")
    _need(k, torch.bfloat16, "k")
    _need(v, torch.bfloat16, "v")
    B, n_q, Hq, D = q.shape
    Hkv, L_cap = k.shape[1], k.shape[2]
    if kv_len is None:
        kv_len = P + n_q - kv_start
    m = l = acc = None
    if state is not None:
        m, l, acc = state
        for t, n in ((m, "m"), (l, "l"), (acc, "acc")):
            _need(t, torch.float32, n)
    if out is None and (state is None or flags & _lib.VC_VERIFY_LAST):
        out = torch.empty_like(q)
    if ws is None:
        ws = torch.empty(max(1, verify_workspace_size(B, n_q, Hq, Hkv, D, kv_start, kv_len)),
                         dtype=torch.uint8, device=q.device)
    if out is not None:
        flags |= _out_flag(out)
    check(lib().vc_verify_attn(q.data_ptr(), B, n_q, Hq, Hkv, D, k.data_ptr(), v.data_ptr(),
                               L_cap, kv_start, kv_len, P, _ptr(m), _ptr(l), _ptr(acc),
                               int(flags), float(scale), _ptr(out), ws.data_ptr(), ws.numel(),
                               _stream(stream)), "vc_verify_attn")
    return out


# ------------------------------------------------------------------ accept
def accept(logits: torch.Tensor, drafts: Optional[torch.Tensor] = None, target=None,
           accept_len=None, commit=None, n_commit=None, err_flag=None, stream=None) -> dict:
    """Greedy acceptance over logits [B, n_q, V] fp32 with drafts [B, n_q-1] int32."""
    _need(logits, torch.float32, "logits")
    B, n_q, V = logits.shape
    dev = logits.device
    i32 = dict(dtype=torch.int32, device=dev)
    if target is None:
        target = torch.empty((B, n_q), **i32)
    if err_flag is None:
        err_flag = torch.empty((B,), **i32)
    want_accept = drafts is not None
    if drafts is not None:
        _need(drafts, torch.int32, "drafts")
        if drafts.numel() == 0:
            drafts = None   # n_q == 1: nothing to compare
    if want_accept:
        accept_len = torch.empty((B,), **i32) if accept_len is None else accept_len
        commit = torch.empty((B, n_q), **i32) if commit is None else commit
        n_commit = torch.empty((B,), **i32) if n_commit is None else n_commit
    check(lib().vc_accept(logits.data_ptr(), _ptr(drafts), B, n_q, V, target.data_ptr(),
                          _ptr(accept_len), _ptr(commit), _ptr(n_commit), _ptr(err_flag),
                          _stream(stream)), "vc_accept")
    return {"target": target, "accept_len": accept_len, "commit": commit,
            "n_commit": n_commit, "err": err_flag}


# ------------------------------------------------------------------ staging
def make_events(n: int, stream=None) -> list:
    """n CUDA events (materialised by one record so their handles exist)."""
    s = stream if stream is not None else torch.cuda.current_stream()
    evs = [torch.cuda.Event() for _ in range(n)]
    for e in evs:
        e.record(s)
    return evs


def stage_full_kv(dst: torch.Tensor, src_pinned: torch.Tensor, chunk_bytes: int,
                  copy_stream, events=None, nbytes: Optional[int] = None) -> None:
    """Copy pinned host ``src_pinned`` into device ``dst`` chunk by chunk on
    ``copy_stream``, recording events[i] after chunk i."""
    if not src_pinned.is_pinned():
        raise ValueError("src_pinned must be page-locked")
    n = nbytes if nbytes is not None else src_pinned.numel() * src_pinned.element_size()
    arr = None
    if events:
        arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    check(lib().vc_stage_full_kv(dst.data_ptr(), src_pinned.data_ptr(), n, chunk_bytes,
                                 _stream(copy_stream), arr, len(events) if events else 0),
          "vc_stage_full_kv")


def event_wait(event, timeout_s: float) -> None:
    check(lib().vc_event_wait(event.cuda_event, float(timeout_s)), "vc_event_wait")


def device_error(clear: bool = True) -> int:
    """The library's device error word (bit 0: a bounded wait in verify expired)."""
    v = ctypes.c_int32(0)
    check(lib().vc_device_error(ctypes.byref(v), int(clear)), "vc_device_error")
    return int(v.value)


def int4_quantize(k: torch.Tensor, v: torch.Tensor, cache: "Int4Cache", n_blocks: int,
                  src_t0: int = 0, blk0: int = 0, stream=None) -> None:
    """Quantise rows [src_t0, src_t0 + 32 n_blocks) of k, v [B, Hkv, src_cap, D] (bf16)
    into blocks [blk0, blk0 + n_blocks) of every pair of ``cache``'s int4 arrays."""
    _need(k, torch.bfloat16, "k")
    _need(v, torch.bfloat16, "v")
    B, Hkv, src_cap, D = k.shape
    blk_cap = cache.k_scale.shape[2]
    check(lib().vc_int4_quantize(k.data_ptr(), v.data_ptr(), B * Hkv, D, src_cap, src_t0,
                                 n_blocks, cache.kq.data_ptr(), cache.k_scale.data_ptr(),
                                 cache.k_zero.data_ptr(), cache.vq.data_ptr(),
                                 cache.v_scale.data_ptr(), cache.v_zero.data_ptr(), blk_cap,
                                 blk0, _stream(stream)), "vc_int4_quantize")


def empty_int4_cache(B: int, Hq: int, Hkv: int, D: int, T_cap: int, device="cuda") -> "Int4Cache":
    """Uninitialised int4 arrays for T_cap tokens per pair (S = 0 live tokens)."""
    nb = T_cap // 32
    i32, f16 = dict(dtype=torch.int32, device=device), dict(dtype=torch.float16, device=device)
    return Int4Cache(kq=torch.empty((B, Hkv, nb, 32, 4, D // 32), **i32),
                     k_scale=torch.empty((B, Hkv, nb, D), **f16),
                     k_zero=torch.empty((B, Hkv, nb, D), **f16),
                     vq=torch.empty((B, Hkv, nb, D, 4), **i32),
                     v_scale=torch.empty((B, Hkv, nb, D // 32, 32), **f16),
                     v_zero=torch.empty((B, Hkv, nb, D // 32, 32), **f16), S=0, Hq=Hq)


def evict_scores(q: torch.Tensor, k: torch.Tensor, n: int, score: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None, scale: float = 0.0, stream=None) -> torch.Tensor:
    """Attention mass per key from the last W prompt queries q [B, W, Hq, D] over keys
    [0, n) of k [B, Hkv, L_cap, D]; returns score fp32 [B, Hkv, >= n]."""
    _need(q, torch.bfloat16, "q")
    _need(k, torch.bfloat16, "k")
    B, W, Hq, D = q.shape
    Hkv, L_cap = k.shape[1], k.shape[2]
    if score is None:
        score = torch.empty((B, Hkv, n), dtype=torch.float32, device=q.device)
    _need(score, torch.float32, "score")
    if ws is None:
        ws = torch.empty(int(lib().vc_evict_workspace_size(B, W, Hq)), dtype=torch.uint8,
                         device=q.device)
    check(lib().vc_evict_scores(q.data_ptr(), B, W, Hq, Hkv, D, k.data_ptr(), L_cap, n,
                                float(scale), score.data_ptr(), score.shape[-1], ws.data_ptr(),
                                ws.numel(), _stream(stream)), "vc_evict_scores")
    return score


def evict_select(score: torch.Tensor, n: int, budget: int, n_sinks: int, n_recent: int,
                 idx: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Kept positions (ascending) per row of score [..., score_cap]: sinks, the top
    middle scores (ties to the lower position) up to the budget, the recent window."""
    _need(score, torch.float32, "score")
    rows = score.numel() // score.shape[-1]
    if idx is None:
        idx = torch.empty(score.shape[:-1] + (min(budget, n),), dtype=torch.int32,
                          device=score.device)
    _need(idx, torch.int32, "idx")
    check(lib().vc_evict_select(score.data_ptr(), rows, score.shape[-1], n, budget, n_sinks,
                                n_recent, idx.data_ptr(), idx.shape[-1], _stream(stream)),
          "vc_evict_select")
    return idx


def set_wait_limit(seconds: float) -> float:
    """Time limit of the verify kernel's pipeline waits for the launches that follow
    (0 restores the 2 s default); returns the previous limit in seconds."""
    prev = ctypes.c_double(0.0)
    check(lib().vc_set_wait_limit(float(seconds), ctypes.byref(prev)), "vc_set_wait_limit")
    return float(prev.value)


def csm_out_len(T: int, n_sinks: int, n_recent: int, chunk: int, r: float) -> int:
    """Rows left by one Chunked Soft Matching round over T rows (-1 if invalid)."""
    return int(lib().vc_csm_out_len(T, n_sinks, n_recent, chunk, r))


def csm_compress(k: torch.Tensor, v: torch.Tensor, n_sinks: int, n_recent: int, chunk: int,
                 r: float, deg: Optional[torch.Tensor] = None, T: Optional[int] = None,
                 k_out=None, v_out=None, deg_out=None, dest=None, stream=None):
    """One Chunked Soft Matching round (CentroidKV) over rows [0, T) of every pair.

    k, v: [B, Hkv, T_cap, D] bf16; deg: [B, Hkv, T_cap] int32 or None (all 1).
    Returns (k_out, v_out, deg_out, n_out): a compact cache of n_out rows per pair."""
    _need(k, torch.bfloat16, "k")
    _need(v, torch.bfloat16, "v")
    B, Hkv, T_cap, D = k.shape
    T = T_cap if T is None else T
    n_out = csm_out_len(T, n_sinks, n_recent, chunk, r)
    if n_out < 0:
        raise ValueError("csm_compress: invalid sizes or ratio")
    if k_out is None:
        k_out = torch.empty((B, Hkv, max(n_out, 1), D), dtype=k.dtype, device=k.device)
    if v_out is None:
        v_out = torch.empty_like(k_out)
    if deg_out is None:
        deg_out = torch.empty(k_out.shape[:3], dtype=torch.int32, device=k.device)
    if deg is not None:
        _need(deg, torch.int32, "deg")
    if dest is not None:
        _need(dest, torch.int32, "dest")
    check(lib().vc_csm_compress(k.data_ptr(), v.data_ptr(), _ptr(deg), B * Hkv, D, T, T_cap,
                                n_sinks, n_recent, chunk, float(r), k_out.data_ptr(),
                                v_out.data_ptr(), deg_out.data_ptr(), k_out.shape[2], _ptr(dest),
                                _stream(stream)), "vc_csm_compress")
    return k_out, v_out, deg_out, n_out


# ------------------------------------------------------------------ paged cache
_PAGE_TYPES = {torch.bfloat16: _lib.VC_PAGE_BF16, torch.float8_e4m3fn: _lib.VC_PAGE_E4M3,
               torch.int8: _lib.VC_PAGE_INT8}


def _same_device(dev, **tensors):
    for n, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{n}: on {t.device}, expected {dev}")


_MOST = 2 ** 31 - 1


def _fits(name: str, *sizes):
    """Sizes go to the library as 32-bit numbers (ctypes would take them modulo 2^32)."""
    if max(sizes) > _MOST:
        raise ValueError(f"{name}: a size past 2^31 - 1")


def _on(stream, dev):
    """Context in which a call's own tensors are made: they belong to the stream that uses
    them, or freeing them here would hand their memory on while that stream still runs.  A
    stream given as a number is one of ``dev``, whichever device is current."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    return torch.cuda.stream(stream)


def _call(name: str, dev, stream, *args) -> None:
    """Call an entry point with ``dev`` current, on ``stream`` or dev's current one."""
    # (the raw handle: torch.cuda.current_stream(dev) builds an object first, 2 us)
    s = torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else _stream(stream)
    fn = getattr(lib(), name)
    if dev.index == torch.cuda.current_device():
        st = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, s)
    if st:
        check(st, name)


@dataclass(frozen=True, eq=False)
class PagedCache:
    """K and V rows of B sequences in pages of a shared pool (see vc_paged_cache).

    k_pages, v_pages: [n_pages, Hkv, page, D] bfloat16, float8_e4m3fn or int8 (any strides
    that are multiples of 16 bytes, the last dimension contiguous); page_table: int32
    [B, max_pages]; kv_len: int32 [B], the tokens of each sequence including the new ones of
    a call; k_scale, v_scale: fp32 [n_pages, Hkv, page] for 8-bit pages; err_flag: int32 [1]
    or None, into which the calls OR VC_PAGED_BAD_PAGE, VC_PAGED_BAD_LENGTH and
    VC_PAGED_NOT_FINITE.  The tensors are fixed; their contents may change between calls."""

    k_pages: torch.Tensor
    v_pages: torch.Tensor
    page_table: torch.Tensor
    kv_len: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None
    err_flag: Optional[torch.Tensor] = None

    def __post_init__(self):
        k, v = self.k_pages, self.v_pages
        if k.dtype not in _PAGE_TYPES or v.dtype != k.dtype:
            raise TypeError("k_pages, v_pages: expected bfloat16, float8_e4m3fn or int8, both alike")
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k_pages, v_pages: expected [n_pages, Hkv, page, D], both alike")
        for t, n in ((k, "k_pages"), (v, "v_pages")):
            if not t.is_cuda:
                raise ValueError(f"{n}: expected a CUDA tensor")
            if t.stride(3) != 1:
                raise ValueError(f"{n}: the last dimension must be contiguous")
        n_pages, Hkv, page, D = k.shape
        _fits("k_pages, page_table", *k.shape, *self.page_table.shape)
        _need(self.page_table, torch.int32, "page_table")
        _need(self.kv_len, torch.int32, "kv_len")
        if self.page_table.dim() != 2 or self.kv_len.shape != self.page_table.shape[:1]:
            raise ValueError("page_table: expected [B, max_pages] with kv_len [B]")
        quantised = k.dtype != torch.bfloat16
        for t, n in ((self.k_scale, "k_scale"), (self.v_scale, "v_scale")):
            if (t is not None) != quantised:
                raise ValueError(f"{n}: needed for 8-bit pages, and only for them")
            if quantised:
                _need(t, torch.float32, n)
                if t.shape != k.shape[:3]:
                    raise ValueError(f"{n}: expected [n_pages, Hkv, page]")
        if self.err_flag is not None:
            _need(self.err_flag, torch.int32, "err_flag")
            if self.err_flag.numel() < 1:
                raise ValueError("err_flag: expected one entry")
        _same_device(k.device, v_pages=v, page_table=self.page_table, kv_len=self.kv_len,
                     k_scale=self.k_scale, v_scale=self.v_scale, err_flag=self.err_flag)
        c = PagedCacheStruct()
        c.type = _PAGE_TYPES[k.dtype]
        c.B, c.max_pages = self.page_table.shape
        c.n_pages, c.Hkv, c.page, c.D = n_pages, Hkv, page, D
        c.k, c.v = _ptr(k), _ptr(v)
        c.k_page_stride, c.k_head_stride, c.k_row_stride = k.stride()[:3]
        c.v_page_stride, c.v_head_stride, c.v_row_stride = v.stride()[:3]
        c.k_scale, c.v_scale = _ptr(self.k_scale), _ptr(self.v_scale)
        c.page_table, c.kv_len = _ptr(self.page_table), _ptr(self.kv_len)
        c.err_flag = _ptr(self.err_flag)
        # what every call needs, read once
        for name, value in (("_struct", c), ("_ref", ctypes.byref(c)), ("_device", k.device),
                            ("B", c.B), ("Hkv", Hkv), ("D", D)):
            object.__setattr__(self, name, value)

    def struct(self) -> PagedCacheStruct:
        return self._struct


def empty_paged_cache(B: int, Hkv: int, D: int, n_pages: int, max_pages: int, page: int = 64,
                      dtype=torch.bfloat16, device="cuda") -> PagedCache:
    """A pool of n_pages uninitialised pages with an empty page table (-1) for B sequences of
    no tokens, and a zeroed err_flag."""
    pool = dict(size=(n_pages, Hkv, page, D), dtype=dtype, device=device)
    scale = ((lambda: torch.ones((n_pages, Hkv, page), dtype=torch.float32, device=device))
             if dtype != torch.bfloat16 else (lambda: None))
    i32 = dict(dtype=torch.int32, device=device)
    return PagedCache(k_pages=torch.empty(**pool), v_pages=torch.empty(**pool),
                      page_table=torch.full((B, max_pages), -1, **i32),
                      kv_len=torch.zeros((B,), **i32), k_scale=scale(), v_scale=scale(),
                      err_flag=torch.zeros((1,), **i32))


def _new_rows(t: torch.Tensor, name: str, D: int, dev):
    """Rows, heads, and the strides of both (0 where there is one entry) of [N, heads, D]."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != D:
        raise ValueError(f"{name}: expected [N, heads, D = {D}]")
    tok, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if t.device != dev:
        raise ValueError(f"{name}: on {t.device}, expected {dev}")
    if shape[0] > _MOST:
        _fits(name, shape[0])
    return shape[0], shape[1], tok if shape[0] > 1 else 0, head if shape[1] > 1 else 0


def _cu(cu_q: Optional[torch.Tensor], B: int, dev) -> Optional[int]:
    if cu_q is None:
        return None
    _need(cu_q, torch.int32, "cu_q")
    if cu_q.numel() != B + 1:
        raise ValueError("cu_q: expected B + 1 entries")
    if cu_q.device != dev:
        raise ValueError(f"cu_q: on {cu_q.device}, expected {dev}")
    return cu_q.data_ptr()


def paged_write(k: torch.Tensor, v: torch.Tensor, cache: PagedCache,
                cu_q: Optional[torch.Tensor] = None, stream=None) -> None:
    """Store new K and V rows k, v [N, Hkv, D] (bf16; strided views of a fused projection will
    do) in their pages, quantised when the pages are 8-bit.  Sequence b's rows are
    cu_q[b] .. cu_q[b + 1] - 1 (N / B each without cu_q) and go to its last positions."""
    dev, D = cache._device, cache.D
    N, heads, k_tok, k_head = _new_rows(k, "k", D, dev)
    N_v, heads_v, v_tok, v_head = _new_rows(v, "v", D, dev)
    if (N_v, heads_v) != (N, heads) or heads != cache.Hkv:
        raise ValueError("k, v: expected [N, Hkv, D], both alike")
    cu = _cu(cu_q, cache.B, dev)
    _call("vc_paged_write", dev, stream, cache._ref, k.data_ptr(), k_tok, k_head, v.data_ptr(),
          v_tok, v_head, N, cu)


def paged_read(cache: PagedCache, k_out: torch.Tensor, v_out: torch.Tensor, start=0,
               stream=None) -> None:
    """Read rows back into k_out, v_out bf16 [B, Hkv, T_cap, D]: row r becomes position
    start + r where the sequence has one, and is left as it was elsewhere.  start: a number,
    or int32 [B] on the device."""
    dev, D = cache._device, cache.D
    shape = k_out.shape
    if len(shape) != 4 or shape[0] != cache.B or shape[1] != cache.Hkv or shape[3] != D or \
            v_out.shape != shape:
        raise ValueError("k_out, v_out: expected [B, Hkv, T_cap, D], both alike")
    for t, n in ((k_out, "k_out"), (v_out, "v_out")):
        _need(t, torch.bfloat16, n)
        if t.device != dev:
            raise ValueError(f"{n}: on {t.device}, expected {dev}")
    starts = None
    if isinstance(start, torch.Tensor):
        _need(start, torch.int32, "start")
        if start.numel() != cache.B or start.device != dev:
            raise ValueError("start: expected B entries on the cache's device")
        starts, start = start.data_ptr(), 0
    _call("vc_paged_read", dev, stream, cache._ref, int(start), starts, k_out.data_ptr(),
          v_out.data_ptr(), shape[2])


def paged_attn_workspace_size(cache: PagedCache, N: int, Hq: int, max_q: int = 0) -> int:
    """Workspace bytes of paged_attn for N rows; depends on sizes only."""
    _fits("N, Hq, max_q", N, Hq, max_q)
    if cache._device.index == torch.cuda.current_device():
        n = lib().vc_paged_attn_workspace_size(cache._ref, N, Hq, max_q)
    else:
        with torch.cuda.device(cache._device):
            n = lib().vc_paged_attn_workspace_size(cache._ref, N, Hq, max_q)
    if n == 0:
        check(_lib.VC_ERR_INVALID, "vc_paged_attn_workspace_size")
    return int(n)


_attn_ws = {}


def paged_attn(q: torch.Tensor, cache: PagedCache, cu_q: Optional[torch.Tensor] = None,
               max_q: Optional[int] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
               scale: float = 0.0, stream=None) -> torch.Tensor:
    """Attention of new tokens q [N, Hq, D] (bf16, strided views will do) over a paged cache
    that holds their keys and values already, causal within each sequence.  Rows are laid out
    as in paged_write; max_q is an upper bound on a sequence's rows, if known.  ``out``
    [N, Hq, D] may be bfloat16 (default) or float32; lse fp32 [N, Hq] or None.  Rows of no
    sequence are left as they were (zero in an ``out`` made here)."""
    dev, D = cache._device, cache.D
    N, Hq, tok, head = _new_rows(q, "q", D, dev)
    cu = _cu(cu_q, cache.B, dev)
    if out is None:
        with _on(stream, dev):
            out = (torch.empty if cu_q is None else torch.zeros)((N, Hq, D), dtype=q.dtype, device=dev)
    elif out.shape != q.shape or not out.is_contiguous() or out.device != dev:
        raise ValueError("out: expected a contiguous [N, Hq, D] on the cache's device")
    if lse is not None:
        _need(lse, torch.float32, "lse")
        if lse.shape != (N, Hq) or lse.device != dev:
            raise ValueError("lse: expected [N, Hq] on the cache's device")
    bound = 0 if max_q is None else int(max_q)
    if bound < 0:
        raise ValueError("max_q: negative")
    if bound > N:                                  # (it goes to the library as 32 bits)
        bound = N
    if ws is None:
        # the size does not depend on the rows: asked for once per head dim and device
        size = _attn_ws.get((D, dev.index))
        if size is None:
            size = _attn_ws[D, dev.index] = paged_attn_workspace_size(cache, N, Hq, bound)
        if stream is None:
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
        else:
            with _on(stream, dev):
                ws = torch.empty(size, dtype=torch.uint8, device=dev)
    elif ws.device != dev or not ws.is_contiguous():
        raise ValueError("ws: expected a contiguous tensor on the cache's device")
    _call("vc_paged_attn", dev, stream, cache._ref, q.data_ptr(), tok, head, N, Hq, cu, bound,
          float(scale), _out_flag(out), out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.nbytes)
    return out


# ------------------------------------------------------------------ acceptance by sampling
def accept_sample_workspace_size(B: int, n_q: int, V: int) -> int:
    _fits("B, n_q, V", B, n_q, V)
    n = lib().vc_accept_sample_workspace_size(B, n_q, V)
    if n == 0:
        raise ValueError("accept_sample: invalid sizes")
    return int(n)


def accept_sample(logits: torch.Tensor, drafts: Optional[torch.Tensor], u: torch.Tensor,
                  draft_logits: Optional[torch.Tensor] = None,
                  temperature: Optional[torch.Tensor] = None,
                  n_drafts: Optional[torch.Tensor] = None, accept_len=None, commit=None,
                  n_commit=None, err_flag=None, ws: Optional[torch.Tensor] = None,
                  stream=None) -> dict:
    """Acceptance by sampling over logits [B, n_q, V] (fp32 or bf16) with drafts
    [B, n_q - 1] int32 and random numbers u [B, n_q] fp64 in [0, 1): the committed tokens are
    samples of softmax(logits / temperature).  draft_logits [B, n_q - 1, V] (the logits' type):
    what the drafts were drawn from; without it they count as drawn with probability one.
    temperature fp32 [B] (0: greedy), n_drafts int32 [B] (a sequence's live drafts).  logits and
    draft_logits start on 16-byte boundaries."""
    dtype, dev = logits.dtype, logits.device
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits: expected float32 or bfloat16, got {dtype}")
    _need(logits, dtype, "logits")
    if logits.dim() != 3:
        raise ValueError("logits: expected [B, n_q, V]")
    B, n_q, V = logits.shape
    if B > _MOST or n_q > _MOST or V > _MOST:
        _fits("logits", B, n_q, V)
    if n_q > 1 and drafts is None:
        raise ValueError("drafts: needed when n_q > 1")
    i32 = torch.int32
    for t, n, dt, shape in ((drafts, "drafts", i32, (B, n_q - 1)), (u, "u", torch.float64, (B, n_q)),
                            (draft_logits, "draft_logits", dtype, (B, n_q - 1, V)),
                            (temperature, "temperature", torch.float32, (B,)),
                            (n_drafts, "n_drafts", i32, (B,)), (accept_len, "accept_len", i32, (B,)),
                            (commit, "commit", i32, (B, n_q)), (n_commit, "n_commit", i32, (B,)),
                            (err_flag, "err_flag", i32, (B,))):
        if t is not None and not (t.dtype is dt and t.shape == shape and t.device == dev
                                  and t.is_contiguous()):
            _need(t, dt, n)
            raise ValueError(f"{n}: expected shape {shape} on {dev}, got {tuple(t.shape)} on {t.device}")
    if drafts is not None and drafts.numel() == 0:
        drafts = draft_logits = None
    i32 = dict(dtype=torch.int32, device=dev)
    with _on(stream, dev):
        if accept_len is None and commit is None and n_commit is None and err_flag is None:
            # one allocation; each is contiguous
            accept_len, n_commit, err_flag, commit = torch.empty((n_q + 3) * B, **i32).split(
                (B, B, B, n_q * B))
            commit = commit.view(B, n_q)
        if accept_len is None:
            accept_len = torch.empty((B,), **i32)
        if commit is None:
            commit = torch.empty((B, n_q), **i32)
        if n_commit is None:
            n_commit = torch.empty((B,), **i32)
        if err_flag is None:
            err_flag = torch.empty((B,), **i32)
        if ws is None:
            if dev.index == torch.cuda.current_device():
                n = accept_sample_workspace_size(B, n_q, V)
            else:
                with torch.cuda.device(dev):
                    n = accept_sample_workspace_size(B, n_q, V)
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError("ws: expected a contiguous tensor on the logits' device")
    _call("vc_accept_sample", dev, stream, logits.data_ptr(), _ptr(draft_logits), _ptr(drafts),
          u.data_ptr(), _ptr(temperature), _ptr(n_drafts), B, n_q, V,
          _lib.VC_LOGITS_BF16 if logits.dtype == torch.bfloat16 else 0, accept_len.data_ptr(),
          commit.data_ptr(), n_commit.data_ptr(), err_flag.data_ptr(), ws.data_ptr(), ws.nbytes)
    return {"accept_len": accept_len, "commit": commit, "n_commit": n_commit, "err": err_flag}
