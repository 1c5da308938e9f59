"""The exact-token cache as it is measured: append (quantise and write), read (back into the packed
layout that coarsening takes) and paged attention of new query rows over it.

`run` computes each operator in plain torch operations, or, where `own` is true, through this
package's entry points. A page of the cache holds 64 tokens of one sequence for all KV heads, as
[Hkv][4 groups][group]; a group holds 16 tokens: keys [16][d], values [16][d] in the input's type
("raw"), or e4m3 codes of both followed by a scale exponent byte (e + 127) for each key and each value
("e4m3"). Inside the key and value blocks the 16-byte chunk c of slot n is stored at chunk
c ^ (((n & 6) ^ ((n & 1) << 2)) & (chunks - 1)).
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
GROUP = 16
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E_MIN, E_MAX = -100, 119   # scale exponents of an e4m3 row


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _append(name, B, Hq, Hkv, d, dtype, fmt, old, new, pad=0, fused=True):
    return {"name": name, "op": "append", "B": B, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype, "format": fmt,
            "old_lo": old[0], "old_hi": old[1], "new_lo": new[0], "new_hi": new[1], "pad": pad, "fused": fused}


def _read(name, B, Hkv, d, dtype, fmt, length, first=0):
    return {"name": name, "op": "read", "B": B, "Hkv": Hkv, "d": d, "dtype": dtype, "format": fmt,
            "len_lo": length[0], "len_hi": length[1], "first": first}


def _attn(name, B, R, Hq, Hkv, d, dtype, fmt, length, window=0, softcap=0.0, alibi=False, prior=False):
    return {"name": name, "op": "attn", "B": B, "R": R, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype, "format": fmt,
            "len_lo": length[0], "len_hi": length[1], "window": window, "softcap": softcap, "alibi": alibi,
            "prior": prior}


def listed():
    return [
        # one decode step of the 1.5B-shaped model, one sequence: latency only
        _append("append_token_1p5b", 1, 12, 2, 128, "bf16", "e4m3", (10500, 10500), (1, 1)),
        # one decode step of a full batch of the 7B-shaped model, keys and values out of a fused projection
        _append("append_step_7b_b128", 128, 28, 4, 128, "bf16", "e4m3", (1, 2048), (1, 1)),
        # prompts of a batch arriving together, ragged, with rows of padding behind the last one
        _append("append_prompts_7b", 8, 28, 4, 128, "bf16", "e4m3", (0, 0), (1000, 32768), pad=37),
        # a continued prompt kept unquantised in 32 bits, the small model's shape
        _append("append_raw_f32", 3, 2, 1, 64, "f32", "raw", (5, 700), (77, 1024), fused=False),
        # a batch's history read back to be coarsened
        _read("read_7b_e4m3", 8, 4, 128, "bf16", "e4m3", (8192, 32768)),
        # the older part of short unquantised histories, starting inside a page
        _read("read_raw_tail", 5, 2, 64, "bf16", "raw", (129, 4001), first=37),
        # one sequence of the 1.5B-shaped model: few keys, so latency and the split over the length count
        _attn("attn_1p5b", 1, 1, 12, 2, 128, "bf16", "e4m3", (10500, 10500)),
        # the 7B-shaped decode batch over its whole exact history, 8 bit
        _attn("attn_7b_e4m3", 32, 1, 28, 4, 128, "bf16", "e4m3", (32768, 32768)),
        # the same model with an unquantised cache and ragged lengths
        _attn("attn_7b_raw_ragged", 32, 1, 28, 4, 128, "bf16", "raw", (512, 32768)),
        # four query rows per sequence, capped scores, a sliding window, some sequences of a single token
        _attn("attn_rows_cap_window", 48, 4, 28, 4, 128, "bf16", "e4m3", (1, 16384), window=4096, softcap=30.0),
        # the small model's shape in 32 bits
        _attn("attn_f32", 4, 1, 2, 1, 64, "f32", "raw", (100, 1024)),
        # exact recent tokens behind a coarsened prefix: attention from each sequence's start on, with a
        # distance bias, joined with the prefix's output and partition
        _attn("attn_join_alibi", 64, 1, 16, 16, 128, "bf16", "e4m3", (64, 8192), alibi=True, prior=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn"])
    d, dtype, fmt = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "bf16", "f32"]), rng.choice(["raw", "e4m3", "e4m3"])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    G = rng.choice([1, 2, 4, 6, 7, 8])
    B = _log(rng, 1, 128)
    if op == "append":
        top = max(1, min(32768, 65536 // (B * Hkv)))
        hi = rng.choice([1, _log(rng, 1, top)])
        lo = 1 if hi == 1 else rng.randint(0, hi)
        old = _log(rng, 1, 2048)
        return {k: v for k, v in _append("", B, G * Hkv, Hkv, d, dtype, fmt, (rng.randint(0, old), old), (lo, hi),
                                         pad=rng.choice([0, 0, 5]) if hi > 1 else 0, fused=rng.random() < 0.5).items()
                if k != "name"}
    if op == "read":
        top = max(2, min(32768, 262144 // (B * Hkv)))
        hi = _log(rng, 1, top)
        return {k: v for k, v in _read("", B, Hkv, d, dtype, fmt, (rng.randint(1, hi), hi),
                                       first=rng.choice([0, 1, 37, 64])).items() if k != "name"}
    R = rng.choice([1, 1, 1, 2, 4])
    top = max(2, min(32768, (1 << 21) // (B * Hkv)))
    if dtype == "f32":
        top = max(2, top // 8)
    hi = _log(rng, 1, top)
    return {k: v for k, v in _attn("", B, R, G * Hkv, Hkv, d, dtype, fmt, (rng.randint(1, hi), hi),
                                   window=rng.choice([0, 0, _log(rng, 1, 4096)]), softcap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                                   alibi=rng.random() < 0.3, prior=rng.random() < 0.3).items() if k != "name"}


def _spread(lo, hi, n, shift=0.0):
    """n lengths from lo to hi, both among them, spread over their logarithm in a scattered order."""
    if n == 1 or lo == hi:
        return [hi] * n
    u = [(0.5 + shift + b * 0.6180339887498949) % 1.0 for b in range(n)]
    v = [min(hi, max(lo, int((lo + 1) * ((hi + 1) / (lo + 1)) ** x) - 1)) for x in u]
    v[u.index(min(u))], v[u.index(max(u))] = lo, hi
    return v


def _lengths(c):
    """Per sequence: tokens held before, tokens that come, or (attention, read) length and first position."""
    if c["op"] == "append":
        return _spread(c["old_lo"], c["old_hi"], c["B"]), _spread(c["new_lo"], c["new_hi"], c["B"], 0.3)
    lens = [max(1, n) for n in _spread(c["len_lo"], c["len_hi"], c["B"])]
    if c["op"] == "read":
        return lens, [min(c["first"], n) for n in lens]
    first = [0] * c["B"]
    if c["prior"]:   # the coarsened prefix: a quarter of the history, in one sequence of eight all of it
        first = [n if b % 8 == 5 else n // 4 for b, n in enumerate(lens)]
    return lens, first


def _keys(c):
    """Keys that the attention of one query row sees, per sequence."""
    lens, first = _lengths(c)
    return [n - min(n, max(f, n - c["window"] if c["window"] else 0)) for n, f in zip(lens, first)]


def work(case):
    c = case
    el = 2 if c["dtype"] == "bf16" else 4
    d, Hkv = c["d"], c["Hkv"]
    vec = 2 * d * el
    held = 2 * (d + 1) if c["format"] == "e4m3" else vec
    if c["op"] == "append":
        rows = sum(_lengths(c)[1]) * Hkv
        return {"bytes": rows * (vec + held) + 8 * c["B"], "flops": 4 * rows * 2 * d}
    if c["op"] == "read":
        lens, first = _lengths(c)
        rows = sum(n - f for n, f in zip(lens, first)) * Hkv
        return {"bytes": rows * (vec + held), "flops": rows * 2 * d}
    keys, q = sum(_keys(c)), c["B"] * c["R"] * c["Hq"]
    return {"bytes": keys * Hkv * held + q * ((3 if c["prior"] else 2) * d * el + (8 if c["prior"] else 4)),
            "flops": 4 * d * keys * c["R"] * c["Hq"]}


# ---------------------------------------------------------------------------
# the cache's bytes in plain torch
# ---------------------------------------------------------------------------
def _power(e):
    """2^e in 32 bits, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """fp32 rows [..., d] -> e4m3 codes and the exponents of their power-of-two scales."""
    a = torch.where(x.isfinite(), x.abs(), 0).amax(-1)
    m, p = torch.frexp(a)                                   # a = m 2^p, m in [0.5, 1)
    e = torch.where(m > 0.875, p - 8, p - 9)                # 448 = 0.875 2^9
    e = torch.where(a > 0, e, 0).clamp(E_MIN, E_MAX)
    y = x * _power(-e)[..., None]
    return y.clamp(-448, 448).to(torch.float8_e4m3fn), e


def _geometry(c):
    el = 1 if c["format"] == "e4m3" else 2 if c["dtype"] == "bf16" else 4
    row = c["d"] * el
    return el, row, GROUP * row * 2 + (2 * GROUP if c["format"] == "e4m3" else 0)


def _blocks(c, pages):
    """Views of the pages: keys and values as [pages, Hkv, 4, 16, chunks, 16] bytes, and the exponent bytes."""
    _, row, group = _geometry(c)
    p = pages.view(-1, c["Hkv"], PAGE // GROUP, group)
    k, v = (p[..., i * GROUP * row:(i + 1) * GROUP * row].view(*p.shape[:3], GROUP, row // 16, 16) for i in (0, 1))
    ke, ve = (p[..., 2 * GROUP * row + i * GROUP:2 * GROUP * row + (i + 1) * GROUP] for i in (0, 1))
    return k, v, ke, ve


def _typed(c, pages):
    """The values held, as the types they are held in: what a call returns of an updated cache."""
    k, v, ke, ve = _blocks(c, pages)
    t = torch.float8_e4m3fn if c["format"] == "e4m3" else DTYPES[c["dtype"]]
    out = {"k": k.flatten(-2).view(t), "v": v.flatten(-2).view(t)}
    return {**out, "k_exp": ke, "v_exp": ve} if c["format"] == "e4m3" else out


def _place(n, chunks, device):
    """Where chunk 0 .. chunks - 1 of the slots n are stored."""
    f = ((n & 6) ^ ((n & 1) << 2)) & (chunks - 1)
    return torch.arange(chunks, device=device) ^ f[..., None]


def _write(c, pages, k, v, page, pos):
    """Write rows k, v [n, Hkv, d] at the positions pos of the pages `page`."""
    kb, vb, ke, ve = _blocks(c, pages)
    slot = (pos % GROUP).long()
    chunks = kb.shape[-2]
    at = (page.long()[:, None, None], torch.arange(c["Hkv"], device=pages.device)[None, :, None],
          (pos % PAGE // GROUP).long()[:, None, None], slot[:, None, None], _place(slot, chunks, pages.device)[:, None, :])
    for x, b, eb in ((k, kb, ke), (v, vb, ve)):
        if c["format"] == "e4m3":
            x, e = _quantise(x.float())
            eb[at[0][..., 0], at[1][..., 0], at[2][..., 0], at[3][..., 0]] = (e + 127).to(torch.uint8)
        b[at] = x.contiguous().view(torch.uint8).view(*x.shape[:2], chunks, 16)


def _rows(c, blocks, table):
    """fp32 keys and values of whole sequences, [B, Hkv, tokens, d], of the pages in `table`."""
    out = []
    slots = torch.arange(GROUP, device=table.device)
    place = _place(slots, blocks[0].shape[-2], table.device)
    for b, eb in ((blocks[0], blocks[2]), (blocks[1], blocks[3])):
        x = b[table.long()][..., slots[:, None], place, :].flatten(-2)          # [B, np, Hkv, 4, 16, row]
        if c["format"] == "e4m3":
            x = x.view(torch.float8_e4m3fn).float() * _power(eb[table.long()].int() - 127)[..., None]
        else:
            x = x.view(DTYPES[c["dtype"]]).float()
        out.append(x.permute(0, 2, 1, 3, 4, 5).flatten(2, 4))
    return out


# ---------------------------------------------------------------------------
# states
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _vectors(g, n, H, d, dtype):
    """Rows with channels of unequal size, as keys have."""
    gain = torch.exp(0.5 * torch.randn(H, d, generator=g, device="cuda"))
    return (torch.randn(n, H, d, generator=g, device="cuda") * gain).to(dtype)


def prepare(case, seed):
    c, g = case, _generator(seed)
    dtype, B, Hkv, d = DTYPES[c["dtype"]], c["B"], c["Hkv"], c["d"]
    a, b = _lengths(c)
    total = [x + y for x, y in zip(a, b)] if c["op"] == "append" else a
    need = [-(-n // PAGE) for n in total]
    cols, num = max(1, max(need)), sum(need) + 3
    order = list(range(num))
    random.Random(seed).shuffle(order)
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n] + [-1] * (cols - n))
        at += n
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": c, "table": torch.tensor(rows, **i32)}
    s["pages"] = torch.zeros(num, Hkv * (PAGE // GROUP) * _geometry(c)[2], dtype=torch.uint8, device="cuda")
    if c["op"] == "append":
        n = sum(b) + c["pad"]
        # keys and values are slices of the projection's output, or tensors of their own
        x = _vectors(g, n, (c["Hq"] if c["fused"] else 0) + 2 * Hkv, d, dtype)
        s["k"], s["v"] = x[:, -2 * Hkv:-Hkv], x[:, -Hkv:]
        if not c["fused"]:
            s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
        s["lens"], s["new_lens"] = torch.tensor(a, **i32), torch.zeros(B, **i32)
        even = c["new_lo"] == c["new_hi"] == 1
        s["cu"] = None if even else torch.tensor(np.concatenate([[0], np.cumsum(b)]), **i32)
        s["held"] = _typed(c, s["pages"])
    else:
        n = sum(a)
        pos = torch.cat([torch.arange(m, device="cuda") for m in a])
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(a, device="cuda"))
        page = s["table"][seq, pos // PAGE]
        step = max(1, (1 << 26) // (Hkv * d))
        for lo in range(0, n, step):
            at = slice(lo, min(n, lo + step))
            m = at.stop - at.start
            _write(c, s["pages"], _vectors(g, m, Hkv, d, dtype), _vectors(g, m, Hkv, d, dtype), page[at], pos[at])
        s["lens_list"], s["first_list"] = a, b
        s["lens"], s["first"] = torch.tensor(a, **i32), torch.tensor(b, **i32) if any(b) else None
    if c["op"] == "attn":
        R, Hq = c["R"], c["Hq"]
        s["q"] = torch.randn(B, R, Hq, d, generator=g, device="cuda").to(dtype)
        s["slopes"] = (torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq).float() if c["alibi"] else None)
        s["prior"] = None
        if c["prior"]:
            lse = 6.0 + torch.randn(B, R, Hq, generator=g, device="cuda")
            lse[::7] = -math.inf                            # nothing coarsened yet
            out = torch.randn(B, R, Hq, d, generator=g, device="cuda").to(dtype)
            out[::7] = 0
            s["prior"] = (out, lse)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, R, Hq, device="cuda")
    if own:   # the handle and the zeroed workspace that a serving program keeps
        import compressed_decode_attention_equal_b200 as skv
        s["skv"] = skv
        s["cache"] = skv.TokenCache(num, Hkv, d, dtype, format=c["format"], pages=s["pages"])
        size = (skv.paged_attn_workspace_bytes(B, c["R"], c["Hq"], Hkv, d, cols) if c["op"] == "attn" else 256)
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return {"append": _run_append, "read": _run_read, "attn": _run_attn}[state["case"]["op"]](state)


def _run_append(s):
    c = s["case"]
    if own:
        lens = s["skv"].cache_append(s["k"], s["v"], s["cache"], s["table"], s["lens"], cu_new=s["cu"],
                                     new_lens=s["new_lens"], workspace=s["workspace"])
        return {**s["held"], "lens": lens}
    n = s["k"].shape[0] - c["pad"]
    if s["cu"] is None:
        seq, off, new = torch.arange(n, device="cuda"), 0, 1
    else:
        seq = torch.searchsorted(s["cu"], torch.arange(n, device="cuda", dtype=torch.int32), right=True) - 1
        off, new = torch.arange(n, device="cuda") - s["cu"][seq], s["cu"].diff()
    pos = s["lens"][seq] + off
    _write(c, s["pages"], s["k"][:n], s["v"][:n], s["table"][seq, (pos // PAGE).long()], pos)
    return {**s["held"], "lens": (s["lens"] + new).to(torch.int32)}


def _run_read(s):
    c = s["case"]
    count = [n - f for n, f in zip(s["lens_list"], s["first_list"])]
    if own:
        k, v = s["skv"].cache_read(s["cache"], s["table"], s["first_list"], count, workspace=s["workspace"])
        return {"k": k, "v": v}
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    k, v = _rows(c, _blocks(c, s["pages"]), s["table"].clamp(min=0))
    t = torch.arange(k.shape[2], device="cuda")
    keep = (t < s["lens"][:, None]) & (t >= (0 if s["first"] is None else s["first"][:, None]))
    keep = keep[:, None, :].expand(B, Hkv, -1)
    return {"k": k[keep].to(DTYPES[c["dtype"]]), "v": v[keep].to(DTYPES[c["dtype"]])}


def _run_attn(s):
    c = s["case"]
    if own:
        out, lse = s["skv"].paged_attn(s["q"], s["cache"], s["table"], s["lens"], first=s["first"], window=c["window"],
                                       softcap=c["softcap"], slopes=s["slopes"], prior=s["prior"], out=s["out"],
                                       lse=s["lse"], workspace=s["workspace"])
        return {"out": out, "lse": lse}
    B, R, Hq, Hkv, d = c["B"], c["R"], c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    k, v = _rows(c, _blocks(c, s["pages"]), s["table"].clamp(min=0))
    q = s["q"].float().view(B, R, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, R * G, d)
    x = q @ k.transpose(-1, -2) * d ** -0.5
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    t, n = torch.arange(k.shape[2], device="cuda"), s["lens"][:, None]
    if c["alibi"]:
        gap = (n - 1 - t).float()[:, None, None, None, :]
        x = (x.view(B, Hkv, R, G, -1) - s["slopes"].view(Hkv, 1, G, 1) * gap).view_as(x)
    seen = t < n
    if s["first"] is not None:
        seen = seen & (t >= s["first"][:, None])
    if c["window"]:
        seen = seen & (t >= n - c["window"])
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top.isfinite(), top, 0)
    p = torch.exp(x - top)
    z = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(z > 0, z, 1)
    lse = torch.log(z) + top
    out = out.view(B, Hkv, R, G, d).transpose(1, 2).reshape(B, R, Hq, d)
    lse = lse.view(B, Hkv, R, G).transpose(1, 2).reshape(B, R, Hq)
    if c["prior"]:
        both = torch.logaddexp(lse, s["prior"][1])
        w, u = (torch.where(both > -math.inf, torch.exp(l - both), 0)[..., None] for l in (lse, s["prior"][1]))
        out, lse = w * out + u * s["prior"][0].float(), both
    return {"out": out.to(s["q"].dtype), "lse": lse}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_values():
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    v = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = math.nan if code & 127 == 127 else m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(-x if code & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _held_rows(c, pages, table_row, lo, hi):
    """Keys and values of positions [lo, hi) of one sequence in 64 bits, [hi - lo, Hkv, d], byte by byte."""
    el, row, group = _geometry(c)
    Hkv, d = c["Hkv"], c["d"]
    pos = torch.arange(lo, hi, device="cuda")
    base = (table_row.long()[pos // 64] * Hkv)[:, None] + torch.arange(Hkv, device="cuda")   # page and head
    base = (base * 4 + (pos % 64 // 16)[:, None]) * group
    n = pos % 16
    swizzle = torch.where(n % 2 == 1, (n // 2 * 2 % 8) ^ 4, n // 2 * 2 % 8) % (row // 16)
    byte = torch.arange(row, device="cuda")
    inside = ((byte // 16)[None, :] ^ swizzle[:, None]) * 16 + byte % 16
    flat, both = pages.view(-1), []
    for i in (0, 1):
        at = base[:, :, None] + (i * 16 * row + n * row)[:, None, None] + inside[:, None, :]
        raw = flat[at.reshape(-1)].view(len(pos), Hkv, row)
        if c["format"] == "e4m3":
            e = flat[(base + (32 * row + 16 * i + n)[:, None]).reshape(-1)].view(len(pos), Hkv).double() - 127
            both.append(_e4m3_values()[raw.long()] * _two(e)[..., None])
        else:
            both.append(raw.view(DTYPES[c["dtype"]]).view(len(pos), Hkv, d).double())
    return both


def _two(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _to_e4m3(x):
    """64-bit rows to the nearest e4m3 multiples of their scale (ties to even), as code values and exponents."""
    a = x.abs().amax(-1)
    e = torch.ceil(torch.log2(a / 448))
    e = torch.where(a == 0, 0.0, e)
    e = torch.where(a > 448 * _two(e), e + 1, e)
    e = torch.where(a <= 448 * _two(e - 1), e - 1, e)
    e = torch.where(a == 0, 0.0, e).clamp(E_MIN, E_MAX)
    y = x * _two(-e)[..., None]
    step = _two(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448), e


def exact(case, seed):
    c, s = case, prepare(case, seed)
    d, Hkv = c["d"], c["Hkv"]
    a, b = _lengths(c)
    if c["op"] == "append":
        P, row = s["pages"].shape[0], d
        held = {x: torch.zeros(P, Hkv, 4, 16, d, dtype=torch.float64, device="cuda") for x in ("k", "v")}
        per = 16 // _geometry(c)[0]                          # values in a 16-byte chunk
        i = 0
        for q in range(c["B"]):
            pos = torch.arange(a[q], a[q] + b[q], device="cuda")
            n = pos % 16
            swizzle = torch.where(n % 2 == 1, (n // 2 * 2 % 8) ^ 4, n // 2 * 2 % 8) % (d // per)
            page = s["table"][q].long()[pos // 64]
            for x in ("k", "v"):
                val = s[x][i:i + b[q]].double()
                if c["format"] == "e4m3":
                    val = _to_e4m3(val)[0]
                col = torch.arange(d, device="cuda")
                to = ((col // per)[None, :] ^ swizzle[:, None]) * per + col % per
                val = torch.empty_like(val).scatter_(-1, to[:, None, :].expand_as(val), val)
                held[x][page, :, pos % 64 // 16, n] = val
            i += b[q]
        lens = torch.tensor([x + y for x, y in zip(a, b)], dtype=torch.int32, device="cuda")
        none = {"k_exp": None, "v_exp": None} if c["format"] == "e4m3" else {}
        return {**held, **none, "lens": lens}
    if c["op"] == "read":
        got = [_held_rows(c, s["pages"], s["table"][q], b[q], a[q]) for q in range(c["B"])]
        return {x: torch.cat([r[i].transpose(0, 1).reshape(-1, d) for r in got]) for i, x in enumerate(("k", "v"))}
    R, Hq, B = c["R"], c["Hq"], c["B"]
    G = Hq // Hkv
    out = torch.zeros(B, R, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, R, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(_keys(c)):
        if n:
            k, v = _held_rows(c, s["pages"], s["table"][i], a[i] - n, a[i])
            x = torch.einsum("rhgd,thd->rhgt", s["q"][i].double().view(R, Hkv, G, d), k) / math.sqrt(d)
            if c["softcap"]:
                x = torch.tanh(x / c["softcap"]) * c["softcap"]
            if c["alibi"]:
                slope = s["slopes"].double().view(Hkv, G)
                x = x - slope[None, :, :, None] * (n - 1 - torch.arange(n, device="cuda", dtype=torch.float64))
            lse[i] = torch.logsumexp(x, -1).view(R, Hq)
            out[i] = torch.einsum("rhgt,thd->rhgd", torch.softmax(x, -1), v).reshape(R, Hq, d)
        if c["prior"]:
            po, pl = s["prior"][0][i].double(), s["prior"][1][i].double()
            z = torch.logaddexp(lse[i], pl)
            w = torch.where(z > -math.inf, torch.exp(lse[i] - z), 0)
            u = torch.where(z > -math.inf, torch.exp(pl - z), 0)
            out[i], lse[i] = w[..., None] * out[i] + u[..., None] * po, z
    return {"out": out, "lse": lse}
