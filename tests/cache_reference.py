"""Plain 64-bit reference of the exact-token cache (numpy, element by element definitions; shares
nothing with the package but the documented page layout), and the error bounds its tests use.

e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f / 0xff are NaN, the largest value is 448.
"""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE, GROUP = 64, 16


def e4m3_table() -> np.ndarray:
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if c & 127 == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -x if c & 128 else x
    return v


TABLE = e4m3_table()


def quantise(x: np.ndarray):
    """Rows [..., d] -> (code values, exponents): nearest e4m3 value of x 2^-e, ties to the even code."""
    ax = np.where(np.isfinite(x), np.abs(x), 0.0)
    a = ax.max(-1)
    e = np.zeros(a.shape, np.int64)
    for i in np.ndindex(a.shape):
        if a[i] > 0:
            k = math.frexp(a[i])[1] - 10
            while a[i] > 448 * 2.0 ** k:
                k += 1
            e[i] = min(max(k, -100), 119)
    y = x * np.ldexp(1.0, -e)[..., None]
    pos = TABLE[:127]                                   # 0 .. 448, increasing
    m = np.minimum(np.where(np.isnan(y), 0, np.abs(y)), 448.0)
    hi = np.searchsorted(pos, m)                        # first value >= m
    lo = np.maximum(hi - 1, 0)
    up = (pos[hi] - m < m - pos[lo]) | ((pos[hi] - m == m - pos[lo]) & (hi % 2 == 0))
    q = np.where(up, pos[hi], pos[lo]) * np.sign(np.where(np.isnan(y), 0, y))
    return np.where(np.isnan(y), np.nan, q), e


def _columns(n: int, d: int, per: int) -> np.ndarray:
    """Stored column of each of the d elements of slot n (per elements to a 16-byte chunk)."""
    f = ((n & 6) ^ ((n & 1) << 2)) & (d // per - 1)
    i = np.arange(d)
    return ((i // per) ^ f) * per + i % per


def _slots(cache, table_row, t: int):
    return int(table_row[t // PAGE]), t % PAGE // GROUP, t % GROUP


def read_rows(cache, table_row, lo: int, hi: int):
    """Values held at positions [lo, hi) of one sequence: (k, v) [hi - lo, Hkv, d], and their scales."""
    k, v = cache.k.double().cpu().numpy(), cache.v.double().cpu().numpy()
    per = 16 if cache.format == "e4m3" else 16 // cache.k.element_size()
    out = [np.empty((hi - lo, cache.Hkv, cache.d)) for _ in range(2)]
    scale = [np.ones((hi - lo, cache.Hkv)) for _ in range(2)]
    exps = [None if x is None else x.cpu().numpy().astype(np.int64) for x in (cache.k_exp, cache.v_exp)]
    for t in range(lo, hi):
        p, g, n = _slots(cache, table_row, t)
        col = _columns(n, cache.d, per)
        for i, src in enumerate((k, v)):
            out[i][t - lo] = src[p, :, g, n][:, col]
            if exps[i] is not None:
                scale[i][t - lo] = np.ldexp(1.0, exps[i][p, :, g, n] - 127)
    return [o * s[..., None] for o, s in zip(out, scale)], scale


def write_rows(cache, table_row, t0: int, k: np.ndarray, v: np.ndarray):
    """Put rows [n, Hkv, d] at positions t0 .. of one sequence (the cache's views are host tensors or not)."""
    per = 16 if cache.format == "e4m3" else 16 // cache.k.element_size()
    for i in range(k.shape[0]):
        p, g, n = _slots(cache, table_row, t0 + i)
        col = torch.from_numpy(_columns(n, cache.d, per)).to(cache.k.device)
        for x, held, ex in ((k[i], cache.k, cache.k_exp), (v[i], cache.v, cache.v_exp)):
            if cache.format == "e4m3":
                x, e = quantise(x)
                ex[p, :, g, n] = torch.from_numpy(e + 127).to(torch.uint8).to(ex.device)
            val = torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).to(held.dtype).to(held.device)
            held[p, :, g, n, :].view(torch.uint8 if held.element_size() == 1 else held.dtype)[:, col] = \
                val.view(torch.uint8) if held.element_size() == 1 else val


class Attn:
    """Attention of one sequence's query rows q [R, Hq, d] over keys k, v [n, Hkv, d] (fp64), with the
    quantities that bound a kernel's error: mass = sum_j p_j |v_j| per output, and per row the largest
    error that fp32 products and sums can put into a logit."""

    def __init__(self, q, k, v, vscale, pos, j0, scale=None, softcap=0.0, slopes=None):
        R, Hq, d = q.shape
        n, Hkv, _ = k.shape
        G = Hq // Hkv
        self.out, self.mass = np.zeros((R, Hq, d)), np.zeros((R, Hq, d))
        self.tiny = np.zeros((R, Hq, d))
        self.lse, self.dlogit = np.full((R, Hq), -np.inf), np.zeros((R, Hq))
        scale = 1 / math.sqrt(d) if scale is None else scale
        if n == 0:
            return
        gap = pos - (j0 + np.arange(n))
        for h in range(Hq):
            kk, vv, vs = k[:, h // G], v[:, h // G], vscale[:, h // G]
            s = scale * (q[:, h] @ kk.T)
            size = abs(scale) * (np.abs(q[:, h]) @ np.abs(kk).T)
            bias = 0.0 if slopes is None else slopes[h] * gap
            if softcap:
                s = softcap * np.tanh(s / softcap)
            s = s - bias
            top = s.max(-1, keepdims=True)
            p = np.exp(s - top)
            z = p.sum(-1, keepdims=True)
            p = p / z
            self.lse[:, h] = (top + np.log(z))[:, 0]
            self.out[:, h] = p @ vv
            self.mass[:, h] = p @ np.abs(vv)
            # a 16-bit weight of 2^-14 of the largest (scaled by its value's scale) or less is off by 2^-25 of it;
            # values of zeros have no scale
            some = np.abs(vv).max(-1) > 0
            self.tiny[:, h] = 2.0 ** -25 * (p * vs * some).max(-1, keepdims=True) * (np.abs(vv) / vs[:, None]).sum(0)
            # d products and sums, the scales, the cap (a few 2^-24 of itself and of the cap) and the bias, each
            # rounded in fp32, and the exponent's base-2 conversion
            self.dlogit[:, h] = (2.0 ** -24 * ((d + 8) * size.max(-1) + 16 * softcap + 8 * np.abs(np.asarray(bias)).max()
                                               + 4 * np.abs(s).max(-1)) + 2.0 ** -21)


def attention_bounds(ref: Attn, dtype, fmt: str):
    """Largest error of (out, lse) against the 64-bit result. Weights: exact exponentials of logits off by
    dlogit (both in the weight and in their sum: 2 dlogit relative), rounded to the matrix product's type (bf16
    caches 2^-8, e4m3 caches 2^-11 plus `tiny`; fp32 not at all), products summed in fp32 (2^-16 relative of the
    mass covers 2^8 sums of sums); one rounding to the output's type."""
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    weight = 0.0 if dtype == torch.float32 else 2.0 ** -11 if fmt == "e4m3" else 2.0 ** -8
    sums = 2.0 ** -18 if dtype == torch.float32 else 2.0 ** -16
    inner = ref.mass * (weight + sums + 2 * ref.dlogit[..., None]) + (ref.tiny if weight else 0.0)
    out = inner * (1 + half) + half * np.abs(ref.out) + 1e-37
    lse = ref.dlogit + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isfinite(ref.lse), ref.lse, 0))
    return out, lse


def check_attention(out, lse, ref: Attn, dtype, fmt, what=""):
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    bo, bl = attention_bounds(ref, dtype, fmt)
    empty = np.isneginf(ref.lse)
    assert np.array_equal(np.isneginf(l), empty), f"{what}: rows without keys differ"
    assert np.all(o[empty] == 0), f"{what}: rows without keys must give zeros"
    with np.errstate(invalid="ignore"):
        le = np.where(empty, 0, np.abs(l - ref.lse))
    assert np.all(le <= bl), f"{what}: lse off by {np.max(le / bl):.2f} bounds"
    err = np.abs(o - ref.out)
    assert np.all(err <= bo), f"{what}: out off by {np.max(err / bo):.2f} bounds"
