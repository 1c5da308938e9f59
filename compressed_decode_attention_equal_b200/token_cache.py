"""The exact-token cache: keys and values of tokens that are not (yet) coarsened.

  TokenCache        paged storage, as the inputs' type ("raw") or 8-bit with a scale per vector ("e4m3")
  cache_append(...) write new tokens, quantising them on the way
  cache_read(...)   read a range back into the packed layout that coarsen() takes
  paged_attn(...)   attention of the new token's query rows over the cache, optionally joined with another
                    attention's output and partition (decode_attn's over the coarsened prefix)

Every call checks its tensors, passes raw device pointers to libskv (include/skv.h) and returns after
one launch on the current stream of the tensors' device (or on `stream`). There is no CPU or PyTorch fallback.
"""
from __future__ import annotations

import array
import ctypes
import functools

import torch

from . import _lib
from ._lib import CACHE_GROUP_TOKENS, CACHE_PAGE_TOKENS, SkvError

FORMATS = {"raw": _lib.SKV_CACHE_RAW, "e4m3": _lib.SKV_CACHE_E4M3}
_DTYPES = {torch.bfloat16: _lib.SKV_BF16, torch.float32: _lib.SKV_F32}


def token_pages_for(T: int) -> int:
    """Pages that T tokens of one sequence take."""
    return -(-int(T) // CACHE_PAGE_TOKENS)


def cache_page_bytes(dtype: torch.dtype, Hkv: int, d: int, format: str = "raw") -> int:
    return int(_lib.load().skv_cache_page_bytes(_dtype_code(dtype), _format_code(format), Hkv, d))


def _dtype_code(dtype: torch.dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}; use torch.bfloat16 or torch.float32")
    return _DTYPES[dtype]


def _format_code(format: str) -> int:
    if format not in FORMATS:
        raise ValueError(f"format must be one of {sorted(FORMATS)}")
    return FORMATS[format]


class TokenCache:
    """Paged storage of exact tokens: one uint8 tensor `pages` [num_pages, page_bytes]; a page holds 64
    tokens of one sequence for all Hkv heads as [Hkv][4 groups][group], a group 16 tokens as
    [keys 16 x d | values 16 x d] in `dtype` (format "raw"), or as e4m3 codes followed by the scale
    exponent bytes [16 | 16] (format "e4m3"; the value held is code * 2^(byte - 127)). `k`, `v` (and
    `k_exp`, `v_exp`) are strided views of those blocks, [num_pages, Hkv, 4, 16, d] (and
    [num_pages, Hkv, 4, 16]), in which the 16-byte chunk c of slot n lies at chunk
    c ^ (((n & 6) ^ ((n & 1) << 2)) & (chunks - 1)). `pages` may be given (a uint8 tensor of that
    shape); new ones start as zeros."""

    def __init__(self, num_pages: int, Hkv: int, d: int, dtype: torch.dtype, device="cuda", format: str = "raw",
                 pages: torch.Tensor | None = None):
        self.num_pages, self.Hkv, self.d, self.dtype, self.format = int(num_pages), int(Hkv), int(d), dtype, format
        self._dtype_code, self._format_code = _dtype_code(dtype), _format_code(format)
        if self.d not in (64, 128):
            raise ValueError("d must be 64 or 128")
        if self.Hkv < 1 or self.num_pages < 0:
            raise ValueError("Hkv must be at least 1 and num_pages not negative")
        e4m3 = format == "e4m3"
        elem = 1 if e4m3 else 2 if dtype == torch.bfloat16 else 4
        block, G = CACHE_GROUP_TOKENS * self.d * elem, CACHE_GROUP_TOKENS
        group = 2 * block + (2 * G if e4m3 else 0)
        self.page_bytes = self.Hkv * (CACHE_PAGE_TOKENS // G) * group
        if pages is None:
            pages = torch.zeros(self.num_pages, self.page_bytes, dtype=torch.uint8, device=device)
        if pages.dtype != torch.uint8 or tuple(pages.shape) != (self.num_pages, self.page_bytes) or not pages.is_contiguous():
            raise ValueError(f"pages must be contiguous uint8 [{self.num_pages}, {self.page_bytes}]")
        self._pages, self._at, self.device, self.on_gpu = pages, pages.data_ptr(), pages.device, pages.is_cuda
        self._struct = _lib.SkvTokenCache(self._at, self.num_pages)
        self._ref = ctypes.byref(self._struct)
        p = pages.view(self.num_pages, self.Hkv, CACHE_PAGE_TOKENS // G, group)
        held = torch.float8_e4m3fn if e4m3 else dtype
        shape = (*p.shape[:3], G, self.d)
        self.k = p[..., :block].view(held).view(shape)
        self.v = p[..., block:2 * block].view(held).view(shape)
        self.k_exp = p[..., 2 * block:2 * block + G] if e4m3 else None
        self.v_exp = p[..., 2 * block + G:] if e4m3 else None

    @property
    def pages(self) -> torch.Tensor:
        """The storage that the views and the calls go to: written in place, never another tensor."""
        return self._pages

    def struct(self):
        """What the C calls take, by reference, of the pages' address now (their storage may be new)."""
        at = self._pages.data_ptr()
        if at != self._at:
            if self._pages.numel() != self.nbytes() or self._pages.device != self.device:
                raise ValueError("the cache's pages have another size or device than it was made with")
            self._struct.pages = self._at = at
        return self._ref

    def nbytes(self) -> int:
        return self.num_pages * self.page_bytes


# ---------------------------------------------------------------------------
# Argument checks shared by the three calls. A decode step makes these calls for every layer, and a call
# of few tokens takes less time on the GPU than its checks do here: each is a handful of attribute reads on the
# way through, and says what is wrong only once something is.
# ---------------------------------------------------------------------------
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # a tenth of current_stream()'s time


def _stream_handle(device: torch.device) -> int:
    return _raw_stream(device.index) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream


def _ptr(t, name: str, device: torch.device, dtype: torch.dtype, shape) -> int:
    """Device pointer of a contiguous tensor of this device, type and shape."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype is not dtype or t.shape != shape:
            raise ValueError(f"{name} must be {dtype} {list(shape)}")
        if t.device != device:
            raise ValueError(f"{name} must be on {device}")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _vector_ptr(t, name: str, cache: TokenCache, dims: int) -> int:
    """Device pointer of keys, values or queries: any strides, d contiguous."""
    if t.dtype is not cache.dtype or t.device != cache.device or t.dim() != dims or t.stride(-1) != 1:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device != cache.device:
            raise ValueError(f"{name} must be on {cache.device}")
        if t.dim() != dims or t.dtype is not cache.dtype:
            raise ValueError(f"{name} must have {dims} dimensions and the cache's dtype")
        raise ValueError(f"{name} must be contiguous along d")
    return t.data_ptr()


def _table_ptr(table, B: int, cache: TokenCache):
    """Device pointer of the page table and its pages per sequence."""
    shape = table.shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError("page_table must be int32 [B, max_pages]")
    return _ptr(table, "page_table", cache.device, torch.int32, shape), shape[1]


def _workspace(ws, device: torch.device, size: int):
    """The given workspace, or a zeroed one of `size` bytes."""
    if ws is None:
        return torch.zeros(size, dtype=torch.uint8, device=device)
    if ws.dtype is not torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace must be contiguous uint8 on {device}")
    return ws


def _scoped(call, cache: TokenCache, stream, *args):
    """Run `call` where its launch and all it allocates belong: on the cache's device, and on `stream`."""
    device = cache.device
    if not cache.on_gpu:
        raise ValueError("the cache's pages must be a CUDA tensor")
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream must be on {device}")
        with torch.cuda.stream(stream):
            return call(*args)
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return call(*args)
    return call(*args)


# ---------------------------------------------------------------------------
# calls
# ---------------------------------------------------------------------------
def cache_append(k: torch.Tensor, v: torch.Tensor, cache: TokenCache, page_table: torch.Tensor, lens: torch.Tensor,
                 cu_new: torch.Tensor | None = None, new_lens: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Append tokens k, v [n, Hkv, d] (slices of a fused projection will do: only d must be contiguous) to B
    sequences that hold `lens` [B] int32 tokens: rows cu_new[b] .. cu_new[b + 1] - 1 to sequence b (cu_new
    [B + 1] int32 on the device; rows behind the last sequence are ignored), or n / B rows to each.
    page_table: int32 [B, max_pages], naming the pages of the new positions too. Returns the new lengths:
    new_lens if given (it may be lens: updated in place), else a new tensor. workspace: at least 256
    bytes of uint8, zeroed once (workspace_error() reads its error flags)."""
    return _scoped(_append, cache, stream, k, v, cache, page_table, lens, cu_new, new_lens, workspace)


def _append(k, v, cache, page_table, lens, cu_new, new_lens, workspace):
    device = cache.device
    k_p, v_p = _vector_ptr(k, "k", cache, 3), _vector_ptr(v, "v", cache, 3)
    shape = k.shape
    n, Hkv, d = shape
    if v.shape != shape or Hkv != cache.Hkv or d != cache.d:
        raise ValueError("k and v must be [n, Hkv, d] of the cache's Hkv and d")
    per_seq = lens.shape
    if len(per_seq) != 1 or per_seq[0] < 1:
        raise ValueError("lens must be int32 [B]")
    B = per_seq[0]
    lens_p = _ptr(lens, "lens", device, torch.int32, per_seq)
    table_p, max_pages = _table_ptr(page_table, B, cache)
    if cu_new is not None:
        cu_p = _ptr(cu_new, "cu_new", device, torch.int32, (B + 1,))
    elif n % B != 0:
        raise ValueError("without cu_new the rows of k must divide evenly among the sequences")
    else:
        cu_p = None
    if new_lens is None:
        new_lens = torch.empty_like(lens)
    new_p = lens_p if new_lens is lens else _ptr(new_lens, "new_lens", device, torch.int32, per_seq)
    ws = _workspace(workspace, device, 256)
    kt, kh, _ = k.stride()
    vt, vh, _ = v.stride()
    st = _lib.load().skv_cache_append(k_p, v_p, cache._dtype_code, kt, kh, vt, vh, B, Hkv, d, n, cu_p, cache._format_code,
                                      cache.struct(), table_p, max_pages, lens_p, new_p, ws.data_ptr(), ws.numel(),
                                      _stream_handle(device))
    if st:
        raise SkvError(st, "skv_cache_append")
    return new_lens


def cache_read(cache: TokenCache, page_table: torch.Tensor, first_list, T_list, k: torch.Tensor | None = None,
               v: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Read positions first_list[b] .. first_list[b] + T_list[b] - 1 of every sequence (host lists) into k, v
    [sum_b Hkv * T_b, d] of the cache's dtype, sequence b a contiguous [Hkv, T_b, d] block: what coarsen() takes.
    Returns (k, v)."""
    return _scoped(_read, cache, stream, cache, page_table, first_list, T_list, k, v, workspace)


def _read(cache, page_table, first_list, T_list, k, v, workspace):
    device, B = cache.device, len(T_list)
    if len(first_list) != B or B < 1:
        raise ValueError("first_list and T_list must name the same sequences, at least one")
    table_p, max_pages = _table_ptr(page_table, B, cache)
    T, first = _int32s(T_list, "T_list"), _int32s(first_list, "first_list")
    rows = (cache.Hkv * sum(T), cache.d)
    if k is None:
        k = torch.empty(rows, dtype=cache.dtype, device=device)
    if v is None:
        v = torch.empty(rows, dtype=cache.dtype, device=device)
    k_p, v_p = _ptr(k, "k", device, cache.dtype, rows), _ptr(v, "v", device, cache.dtype, rows)
    ws = _workspace(workspace, device, 256)
    st = _lib.load().skv_cache_read(cache.struct(), cache._dtype_code, cache._format_code, B, cache.Hkv, cache.d,
                                    first, T, table_p, max_pages, k_p, v_p, ws.data_ptr(), ws.numel(),
                                    _stream_handle(device))
    if st:
        raise SkvError(st, "skv_cache_read")
    return k, v


@functools.lru_cache(maxsize=None)
def _int_array(n: int):
    return ctypes.c_int32 * n


def _int32s(values, name: str):
    """A C array of host integers (ctypes alone would cut them to 32 bits)."""
    try:
        got = array.array("i", values)
    except OverflowError:
        got = (-1,)
    if min(got) < 0:
        raise ValueError(f"{name} must be integers from 0 to 2^31 - 1")
    return _int_array(len(got)).from_buffer(got)


def paged_attn_workspace_bytes(B: int, R: int, Hq: int, Hkv: int, d: int, max_pages: int) -> int:
    return int(_lib.load().skv_paged_attn_workspace_bytes(B, R, Hq, Hkv, d, max_pages))


def paged_attn(q: torch.Tensor, cache: TokenCache, page_table: torch.Tensor, lens: torch.Tensor,
               first: torch.Tensor | None = None, window: int = 0, scale: float | None = None, softcap: float = 0.0,
               slopes: torch.Tensor | None = None, prior=None, out: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Attention of q [B, R, Hq, d] (the new token's query rows, at position lens - 1; only d must be contiguous)
    over the cached keys at positions max(first, lens - window) .. lens - 1 (first: int32 [B]; window 0: none).
    scale: None for 1 / sqrt(d). softcap c > 0: logits become c tanh(s / c). slopes: fp32 [Hq], s -= slope *
    distance. prior: (out, lse) of another attention of the same queries over other keys, joined as it stands: the
    result is that of one attention over all keys if the prior's logits were scaled, capped and biased alike. So
    decode_attn's over the coarsened tokens before `first` joins calls without scale, softcap and slopes (it has none
    of them); a paged_attn over the first n tokens joins any, once slope * (lens - n) is taken off its lse where there
    are slopes (it counts distances from n - 1). out may be prior's out, or q itself where q is contiguous; lse not
    prior's lse. A row without keys gives out 0, lse -inf. workspace: paged_attn_workspace_bytes bytes of uint8, zeroed
    once; the cache's calls may share it, ordered on one stream, but coarsen, the streaming calls and decode_attn may
    not, whose scratch lies where its counters are. Returns (out [B, R, Hq, d], lse [B, R, Hq] fp32)."""
    return _scoped(_attn, cache, stream, q, cache, page_table, lens, first, window, scale, softcap, slopes, prior, out,
                   lse, workspace)


def _attn(q, cache, page_table, lens, first, window, scale, softcap, slopes, prior, out, lse, workspace):
    device = cache.device
    q_p = _vector_ptr(q, "q", cache, 4)
    shape = q.shape
    B, R, Hq, d = shape
    if d != cache.d:
        raise ValueError("q must have the cache's d")
    lens_p = _ptr(lens, "lens", device, torch.int32, (B,))
    table_p, max_pages = _table_ptr(page_table, B, cache)
    rows = shape[:3]
    opts = None
    if scale is not None or softcap or window or first is not None or slopes is not None or prior is not None:
        if not 0 <= window < 1 << 31:
            raise ValueError("window must be from 0 to 2^31 - 1")
        opts = _lib.SkvPagedAttnOptions(0.0 if scale is None else scale, softcap, window)
        if opts.scale == 0.0 and scale is not None or opts.softcap == 0.0 and softcap:   # there 0 stands for the defaults
            raise ValueError("scale and softcap must not be zero in 32 bits")
        if first is not None:
            opts.first = _ptr(first, "first", device, torch.int32, (B,))
        if slopes is not None:
            opts.slopes = _ptr(slopes, "slopes", device, torch.float32, (Hq,))
        if prior is not None:
            opts.prior_out = _ptr(prior[0], "prior out", device, q.dtype, shape)
            opts.prior_lse = _ptr(prior[1], "prior lse", device, torch.float32, rows)
        opts = ctypes.byref(opts)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=device)
    if lse is None:
        lse = torch.empty(rows, dtype=torch.float32, device=device)
    out_p = _ptr(out, "out", device, q.dtype, shape)
    lse_p = _ptr(lse, "lse", device, torch.float32, rows)
    if workspace is None:
        size = paged_attn_workspace_bytes(B, R, Hq, cache.Hkv, d, max_pages)
        workspace = torch.zeros(max(size, 256), dtype=torch.uint8, device=device)
    ws = _workspace(workspace, device, 256)
    qb, qr, qh, _ = q.stride()
    st = _lib.load().skv_paged_attn(q_p, cache._dtype_code, qb, qr, qh, B, R, Hq, cache.Hkv, d, cache._format_code,
                                    cache.struct(), table_p, max_pages, lens_p, out_p, lse_p, ws.data_ptr(), ws.numel(), opts,
                                    _stream_handle(device))
    if st:
        raise SkvError(st, "skv_paged_attn")
    return out, lse
