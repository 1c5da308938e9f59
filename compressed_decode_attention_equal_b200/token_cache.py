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

import contextlib
import ctypes

import torch

from . import _lib
from ._lib import CACHE_GROUP_TOKENS, CACHE_PAGE_TOKENS, SkvError

FORMATS = {"raw": _lib.SKV_CACHE_RAW, "e4m3": _lib.SKV_CACHE_E4M3}
_DTYPES = {torch.bfloat16: _lib.SKV_BF16, torch.float32: _lib.SKV_F32}
_NULL_SCOPE = contextlib.nullcontext()


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
        self.pages = pages
        p = pages.view(self.num_pages, self.Hkv, CACHE_PAGE_TOKENS // G, group)
        held = torch.float8_e4m3fn if e4m3 else dtype
        shape = (*p.shape[:3], G, self.d)
        self.k = p[..., :block].view(held).view(shape)
        self.v = p[..., block:2 * block].view(held).view(shape)
        self.k_exp = p[..., 2 * block:2 * block + G] if e4m3 else None
        self.v_exp = p[..., 2 * block + G:] if e4m3 else None
        self._struct = _lib.SkvTokenCache(pages.data_ptr(), self.num_pages)
        self._ref = ctypes.byref(self._struct)

    def nbytes(self) -> int:
        return self.pages.numel()


# ---------------------------------------------------------------------------
# argument checks shared by the three calls
# ---------------------------------------------------------------------------
def _check(t, name: str, device: torch.device, dtype: torch.dtype, shape: tuple) -> int:
    """Device pointer of a contiguous tensor of this device, type and shape."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _check_table(table, cache: TokenCache, device: torch.device, B: int) -> int:
    if not isinstance(table, torch.Tensor) or table.dtype != torch.int32 or table.dim() != 2 or table.shape[0] != B:
        raise ValueError("page_table must be int32 [B, max_pages]")
    if cache.pages.device != device:
        raise ValueError(f"cache must be on {device}")
    return _check(table, "page_table", device, torch.int32, table.shape)


def _check_workspace(ws, device: torch.device, size: int):
    """The given workspace's pointer and size, or a zeroed one of `size` bytes."""
    if ws is None:
        ws = torch.zeros(size, dtype=torch.uint8, device=device)
    elif not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace must be contiguous uint8 on {device}")
    return ws, ws.data_ptr(), ws.numel()


def _scope(device: torch.device, stream):
    """Where the launch and everything it allocates belongs: the tensors' device, and `stream`."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream must be on {device}")
        return torch.cuda.stream(stream)
    if device.index != torch.cuda.current_device():
        return torch.cuda.device(device)
    return _NULL_SCOPE


def _vectors(t, name: str, dims: int, cache: TokenCache) -> torch.device:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dims or t.shape[-1] != cache.d or t.dtype != cache.dtype:
        raise ValueError(f"{name} must have {dims} dimensions and the cache's dtype and d")
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along d")
    return t.device


def _strides(t: torch.Tensor, dims: int):
    """Strides of the leading dimensions; one of a single element has none that matters."""
    return [st if n > 1 else 0 for st, n in zip(t.stride()[:dims], t.shape)]


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
    device = _vectors(k, "k", 3, cache)
    if _vectors(v, "v", 3, cache) != device or v.shape != k.shape:
        raise ValueError("k and v must have the same shape and device")
    n, Hkv, d = k.shape
    if Hkv != cache.Hkv:
        raise ValueError("k and v must have the cache's Hkv heads")
    B = lens.shape[0] if isinstance(lens, torch.Tensor) and lens.dim() == 1 else 0
    if B < 1:
        raise ValueError("lens must be int32 [B]")
    lens_p = _check(lens, "lens", device, torch.int32, (B,))
    table_p = _check_table(page_table, cache, device, B)
    if cu_new is not None:
        cu_p = _check(cu_new, "cu_new", device, torch.int32, (B + 1,))
    elif n % B != 0:
        raise ValueError("without cu_new the rows of k must divide evenly among the sequences")
    else:
        cu_p = None
    (kt, kh), (vt, vh) = _strides(k, 2), _strides(v, 2)
    with _scope(device, stream):
        if new_lens is None:
            new_lens = torch.empty_like(lens)
        new_p = _check(new_lens, "new_lens", device, torch.int32, (B,))
        workspace, ws_p, ws_n = _check_workspace(workspace, device, 256)
        _lib.check(_lib.load().skv_cache_append(
            k.data_ptr(), v.data_ptr(), cache._dtype_code, kt, kh, vt, vh, B, Hkv, d, n, cu_p, cache._format_code,
            cache._ref, table_p, page_table.shape[1], lens_p, new_p, ws_p, ws_n,
            torch.cuda.current_stream(device).cuda_stream), "skv_cache_append")
    return new_lens


def cache_read(cache: TokenCache, page_table: torch.Tensor, first_list, T_list, k: torch.Tensor | None = None,
               v: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Read positions first_list[b] .. first_list[b] + T_list[b] - 1 of every sequence (host lists) into k, v
    [sum_b Hkv * T_b, d] of the cache's dtype, sequence b a contiguous [Hkv, T_b, d] block: what coarsen() takes.
    Returns (k, v)."""
    B = len(T_list)
    if len(first_list) != B or B < 1:
        raise ValueError("first_list and T_list must name the same sequences, at least one")
    device = cache.pages.device
    table_p = _check_table(page_table, cache, device, B)
    rows = (cache.Hkv * sum(int(t) for t in T_list), cache.d)
    if rows[0] < 0:
        raise ValueError("T_list must not be negative")
    ints = ctypes.c_int32 * B
    with _scope(device, stream):
        k = torch.empty(rows, dtype=cache.dtype, device=device) if k is None else k
        v = torch.empty(rows, dtype=cache.dtype, device=device) if v is None else v
        k_p, v_p = (_check(t, name, device, cache.dtype, rows) for t, name in ((k, "k"), (v, "v")))
        workspace, ws_p, ws_n = _check_workspace(workspace, device, 256)
        _lib.check(_lib.load().skv_cache_read(
            cache._ref, cache._dtype_code, cache._format_code, B, cache.Hkv, cache.d, ints(*map(int, first_list)),
            ints(*map(int, T_list)), table_p, page_table.shape[1], k_p, v_p, ws_p, ws_n,
            torch.cuda.current_stream(device).cuda_stream), "skv_cache_read")
    return k, v


def paged_attn_workspace_bytes(B: int, R: int, Hq: int, Hkv: int, d: int, max_pages: int) -> int:
    return int(_lib.load().skv_paged_attn_workspace_bytes(B, R, Hq, Hkv, d, max_pages))


def paged_attn(q: torch.Tensor, cache: TokenCache, page_table: torch.Tensor, lens: torch.Tensor,
               first: torch.Tensor | None = None, window: int = 0, scale: float | None = None, softcap: float = 0.0,
               slopes: torch.Tensor | None = None, prior=None, out: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Attention of q [B, R, Hq, d] (the new token's query rows, at position lens - 1; only d must be contiguous)
    over the cached keys at positions max(first, lens - window) .. lens - 1 (first: int32 [B]; window 0: none).
    scale: None for 1 / sqrt(d). softcap c > 0: logits become c tanh(s / c). slopes: fp32 [Hq], s -= slope *
    distance. prior: (out, lse) of another attention of the same queries, e.g. decode_attn's over the coarsened
    tokens before `first`; the result is then that of one attention over all keys (out may be prior's out, lse
    not prior's lse). A row without keys gives out 0, lse -inf. workspace: paged_attn_workspace_bytes bytes of
    uint8, zeroed once. Returns (out [B, R, Hq, d], lse [B, R, Hq] fp32)."""
    device = _vectors(q, "q", 4, cache)
    B, R, Hq, d = q.shape
    lens_p = _check(lens, "lens", device, torch.int32, (B,))
    table_p = _check_table(page_table, cache, device, B)
    qs = _strides(q, 3)
    opts = _lib.SkvPagedAttnOptions(0.0 if scale is None else scale, softcap, window)
    if scale is not None and scale == 0.0:
        raise ValueError("scale must not be zero")
    if first is not None:
        opts.first = _check(first, "first", device, torch.int32, (B,))
    if slopes is not None:
        opts.slopes = _check(slopes, "slopes", device, torch.float32, (Hq,))
    if prior is not None:
        opts.prior_out = _check(prior[0], "prior out", device, q.dtype, (B, R, Hq, d))
        opts.prior_lse = _check(prior[1], "prior lse", device, torch.float32, (B, R, Hq))
    with _scope(device, stream):
        if out is None:
            out = torch.empty(B, R, Hq, d, dtype=q.dtype, device=device)
        if lse is None:
            lse = torch.empty(B, R, Hq, dtype=torch.float32, device=device)
        out_p = _check(out, "out", device, q.dtype, (B, R, Hq, d))
        lse_p = _check(lse, "lse", device, torch.float32, (B, R, Hq))
        if workspace is None:
            size = paged_attn_workspace_bytes(B, R, Hq, cache.Hkv, d, page_table.shape[1])
            workspace = torch.zeros(max(size, 256), dtype=torch.uint8, device=device)
        workspace, ws_p, ws_n = _check_workspace(workspace, device, 256)
        _lib.check(_lib.load().skv_paged_attn(
            q.data_ptr(), cache._dtype_code, qs[0], qs[1], qs[2], B, R, Hq, cache.Hkv, d, cache._format_code, cache._ref,
            table_p, page_table.shape[1], lens_p, out_p, lse_p, ws_p, ws_n, ctypes.byref(opts),
            torch.cuda.current_stream(device).cuda_stream), "skv_paged_attn")
    return out, lse
