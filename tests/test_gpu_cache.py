"""The exact-token cache on the GPU: append and read bit for bit against the 64-bit reference, paged
attention within the bounds derived in cache_reference.py, over odd lengths, strides, page orders and options;
unused slots hold NaN everywhere, so that one that leaks into a result fails the test."""
import math

import numpy as np
import pytest
import torch

import cache_reference as ref
import compressed_decode_attention_equal_b200 as skv
import oracle
import workloads
from compressed_decode_attention_equal_b200 import _lib
from gpu_helpers import gpu_units

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(B, Hkv, d, dtype, fmt, total, seed=0, spare=2, cols=0):
    """A cache full of NaN (codes and exponent bytes of ones) and a shuffled page table for `total` tokens each."""
    need = [skv.token_pages_for(t) for t in total]
    num = sum(need) + spare
    order = np.random.RandomState(seed).permutation(num)
    table = np.full((B, max(1, cols, *need)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    c = skv.TokenCache(num, Hkv, d, dtype, format=fmt)
    c.pages.fill_(255)
    return c, torch.from_numpy(table).cuda()


def rand(g, *shape, dtype=BF):
    gain = torch.exp(0.5 * torch.randn(shape[-1], generator=g))
    return (torch.randn(*shape, generator=g) * gain).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def ok(ws):
    st, flags = skv.workspace_error(ws)
    assert st == _lib.SKV_OK, flags


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,fmt", [(BF, "e4m3"), (BF, "raw"), (F32, "e4m3"), (F32, "raw")])
@pytest.mark.parametrize("d,Hkv,fused", [(128, 4, True), (64, 3, False), (128, 5, False), (64, 9, True)])
def test_append_writes_what_the_definition_says(dtype, fmt, d, Hkv, fused):
    old, new, pad = [0, 63, 5, 130, 64], [1, 2, 0, 77, 64], 3
    g = torch.Generator().manual_seed(d + Hkv)
    total = [a + b for a, b in zip(old, new)]
    cache, table = make(5, Hkv, d, dtype, fmt, total, seed=Hkv)
    before = cache.pages.clone()
    n = sum(new) + pad
    x = rand(g, n, (6 if fused else 0) + 2 * Hkv, d, dtype=dtype).cuda()
    k, v = x[:, -2 * Hkv:-Hkv], x[:, -Hkv:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens = i32(old)
    cu = i32(np.concatenate([[0], np.cumsum(new)]))
    got = skv.cache_append(k, v, cache, table, lens, cu_new=cu, workspace=ws)
    ok(ws)
    assert got.tolist() == total and lens.tolist() == old
    # every byte of the cache: the new tokens by the definition, all others as they were
    want = skv.TokenCache(cache.num_pages, Hkv, d, dtype, format=fmt, device="cpu", pages=before.cpu())
    i = 0
    for b, m in enumerate(new):
        ref.write_rows(want, table[b].tolist(), old[b], k[i:i + m].double().cpu().numpy(), v[i:i + m].double().cpu().numpy())
        i += m
    a, w = cache.pages.cpu(), want.pages
    if fmt == "e4m3":   # -0 and +0 are both right where a value rounds to zero
        a, w = (torch.where(t == 128, 0, t) for t in (a, w))
    assert torch.equal(a, w)


@pytest.mark.parametrize("dtype,fmt", [(BF, "e4m3"), (BF, "raw"), (F32, "e4m3")])
@pytest.mark.parametrize("d,Hkv,n", [(128, 4, 24000), (64, 8, 33001), (64, 3, 40007), (128, 1, 50021), (128, 12, 9999)])
def test_append_long_prompts(dtype, fmt, d, Hkv, n):
    """Enough rows that every warp takes several: read back, they are the rows quantised by torch's own e4m3
    conversion (which the host tests compare with the definition)."""
    g = torch.Generator(device="cuda").manual_seed(n)
    cut = n // 3
    cache, table = make(2, Hkv, d, dtype, fmt, [cut + 7, n - cut], seed=1)
    x = (torch.randn(n + 5, Hkv + 1, 2 * d, generator=g, device="cuda") * torch.exp(3 * torch.randn(n + 5, 1, 1, generator=g, device="cuda"))).to(dtype)
    k, v = x[:, :Hkv, :d], x[:, 1:, d:]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = skv.cache_append(k, v, cache, table, i32([7, 0]), cu_new=i32([0, cut, n]), workspace=ws)
    assert got.tolist() == [cut + 7, n - cut]
    rk, rv = skv.cache_read(cache, table, [7, 0], [cut, n - cut], workspace=ws)
    ok(ws)
    for src, have in ((k, rk), (v, rv)):
        want = src[:n].float()
        if fmt == "e4m3":
            a = want.abs().amax(-1)
            m, p = torch.frexp(a)
            e = torch.where(m > 0.875, p - 8, p - 9).clamp(-100, 119)
            two = ((torch.stack([e, -e]).int() + 127) << 23).view(torch.float32)
            want = (want * two[1][..., None]).to(torch.float8_e4m3fn).float() * two[0][..., None]
        want = torch.cat([want[:cut].transpose(0, 1).reshape(-1, d), want[cut:].transpose(0, 1).reshape(-1, d)])
        assert torch.equal(have, want.to(dtype))


def test_append_special_values():
    """Zeros, subnormals, the largest finite values, infinities and NaN; ties go to the even code."""
    d = 64
    rows = np.zeros((8, 1, d), np.float32)
    rows[1, 0, :3] = [1e-40, -3e-42, 2e-44]
    rows[2, 0, :4] = [3e38, -3.3e38, 1e38, 1.0]
    rows[3, 0, :4] = [np.inf, -np.inf, 1.5, -0.25]
    rows[4, 0, :4] = [np.nan, 448.0, -17.0, 19.0]          # 17 and 19 lie between 16, 18 and 20
    rows[5, 0] = np.inf
    rows[6, 0, :4] = [449.0, 448.5, 1.0, 2.0 ** -10]       # one step above 448: the next power
    rows[7, 0, :4] = [2.0 ** -120, 2.0 ** -128, 0, 0]      # below the smallest scale
    cache, table = make(1, 1, d, F32, "e4m3", [8])
    x = torch.from_numpy(rows).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    skv.cache_append(x, x, cache, table, i32([0]), workspace=ws)
    ok(ws)
    (k, v), _ = ref.read_rows(cache, table[0].tolist(), 0, 8)
    q, e = ref.quantise(rows.astype(np.float64))
    want = q * np.ldexp(1.0, e)[..., None]
    assert np.array_equal(k, want, equal_nan=True) and np.array_equal(v, want, equal_nan=True)
    assert want[3, 0, 0] == 448 * 2.0 ** -8 and np.isnan(want[4, 0, 0]) and want[4, 0, 2] == -16 and want[4, 0, 3] == 20
    rk, _ = skv.cache_read(cache, table, [0], [8])
    assert np.array_equal(rk.double().cpu().numpy(), want[:, 0], equal_nan=True)


@pytest.mark.parametrize("Hkv", [1, 4, 6])
def test_append_token_by_token_in_place(Hkv):
    """One token per sequence and call, lens updated in place, across page ends; equal to one call with all."""
    B, d, steps = 3, 128, 70
    g = torch.Generator().manual_seed(5)
    k, v = rand(g, steps, B, Hkv, d).cuda(), rand(g, steps, B, Hkv, d).cuda()
    start = [0, 60, 127]
    one, table = make(B, Hkv, d, BF, "e4m3", [s + steps for s in start])
    lens, ws = i32(start), torch.zeros(256, dtype=torch.uint8, device="cuda")
    for i in range(steps):
        assert skv.cache_append(k[i], v[i], one, table, lens, new_lens=lens, workspace=ws) is lens
    assert lens.tolist() == [s + steps for s in start]
    all_, _ = make(B, Hkv, d, BF, "e4m3", [s + steps for s in start])
    skv.cache_append(k.transpose(0, 1).flatten(0, 1), v.transpose(0, 1).flatten(0, 1), all_, table, i32(start),
                     cu_new=i32([0, steps, 2 * steps, 3 * steps]), workspace=ws)
    ok(ws)
    assert torch.equal(one.pages, all_.pages)


def test_append_nothing_and_errors_are_reported():
    B, Hkv, d = 3, 2, 64
    cache, table = make(B, Hkv, d, BF, "e4m3", [128] * 3)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    e = torch.zeros(0, Hkv, d, dtype=BF, device="cuda")
    assert skv.cache_append(e, e, cache, table, i32([3, 0, 128]), workspace=ws).tolist() == [3, 0, 128]
    before = cache.pages.clone()
    x = torch.ones(6, Hkv, d, dtype=BF, device="cuda")
    # above the capacity (the part that fits is written), below zero, above it before the call
    got = skv.cache_append(x, x, cache, table, i32([127, -1, 129]), workspace=ws)
    assert skv.workspace_error(ws) == (_lib.SKV_ERR_DEVICE, _lib.FLAG_BAD_LENS)
    assert got.tolist() == [128, -1, 129]
    p = int(table[0, 1])
    assert cache.k[p, 0, 3, 15].float().eq(256.0).all()     # 1 = 256 * 2^-8
    changed = (cache.pages != before).any(1).nonzero().flatten().tolist()
    assert changed == [p]
    # offsets that run down or past the rows: those sequences get nothing
    cache.pages.copy_(before)
    got = skv.cache_append(x, x, cache, table, i32([1, 2, 3]), cu_new=i32([0, 4, 2, 9]), workspace=ws)
    assert skv.workspace_error(ws) == (_lib.SKV_ERR_DEVICE, _lib.FLAG_BAD_LENS)
    assert got.tolist() == [5, 2, 3]
    # a page outside the cache: skipped and reported
    bad = table.clone()
    bad[1, 0], bad[2, 0] = cache.num_pages, -7
    cache.pages.copy_(before)
    assert skv.cache_append(x, x, cache, bad, i32([0, 0, 0]), workspace=ws).tolist() == [2, 2, 2]
    assert skv.workspace_error(ws) == (_lib.SKV_ERR_DEVICE, _lib.FLAG_BAD_PAGE)
    changed = (cache.pages != before).any(1).nonzero().flatten().tolist()
    assert changed == [int(table[0, 0])]
    ok(ws)


@pytest.mark.parametrize("dtype,fmt", [(BF, "e4m3"), (BF, "raw"), (F32, "e4m3"), (F32, "raw")])
@pytest.mark.parametrize("d,Hkv", [(128, 3), (64, 2)])
def test_read_returns_what_is_held(dtype, fmt, d, Hkv):
    total = [0, 1, 64, 200, 79, 33]
    first = [0, 0, 63, 17, 79, 5]
    T = [0, 1, 1, 150, 0, 28]
    g = torch.Generator().manual_seed(7)
    cache, table = make(6, Hkv, d, dtype, fmt, total, seed=3)
    x = rand(g, sum(total), Hkv, d, dtype=dtype).cuda()
    y = rand(g, sum(total), Hkv, d, dtype=dtype).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    skv.cache_append(x, y, cache, table, i32([0] * 6), cu_new=i32(np.concatenate([[0], np.cumsum(total)])), workspace=ws)
    k, v = skv.cache_read(cache, table, first, T, workspace=ws)
    ok(ws)
    at = 0
    for b in range(6):
        (kk, vv), _ = ref.read_rows(cache, table[b].tolist(), first[b], first[b] + T[b])
        n = Hkv * T[b]
        assert np.array_equal(k[at:at + n].double().cpu().numpy(), kk.transpose(1, 0, 2).reshape(n, d))
        assert np.array_equal(v[at:at + n].double().cpu().numpy(), vv.transpose(1, 0, 2).reshape(n, d))
        at += n
    if fmt == "raw":
        assert torch.equal(k[Hkv:2 * Hkv], x[1 + 63])
    # nothing to read, and a page outside the cache
    k0, v0 = skv.cache_read(cache, table, [0] * 6, [0] * 6, workspace=ws)
    assert k0.shape == v0.shape == (0, d)
    bad = table.clone()
    bad[3, 1] = cache.num_pages
    k, v = skv.cache_read(cache, bad, [0, 0, 0, 60, 0, 0], [0, 0, 0, 10, 0, 0], workspace=ws)
    assert skv.workspace_error(ws) == (_lib.SKV_ERR_DEVICE, _lib.FLAG_BAD_PAGE)
    k = k.view(Hkv, 10, d)
    assert not k[:, 4:].any() and k[:, :4].any()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def filled(B, Hkv, d, dtype, fmt, lens, seed=0, **kw):
    cache, table = make(B, Hkv, d, dtype, fmt, lens, seed=seed, **kw)
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    if n:
        skv.cache_append(rand(g, n, Hkv, d, dtype=dtype).cuda(), rand(g, n, Hkv, d, dtype=dtype).cuda(), cache, table,
                         i32([0] * B), cu_new=i32(np.concatenate([[0], np.cumsum(lens)])))
    return cache, table, g


def reference(q, cache, table, lens, b, first=0, window=0, **kw):
    n = lens[b]
    lo = min(n, max(0, first, n - window if window else 0))
    (k, v), (_, vs) = ref.read_rows(cache, table[b].tolist(), lo, n)
    return ref.Attn(q[b].double().cpu().numpy(), k, v, vs, n - 1, lo, **kw)


LENS = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 300, 777]


@pytest.mark.parametrize("dtype,fmt", [(BF, "e4m3"), (BF, "raw"), (F32, "e4m3"), (F32, "raw")])
@pytest.mark.parametrize("d,Hkv,G,R", [(128, 2, 7, 1), (64, 1, 6, 1), (128, 1, 1, 1), (128, 2, 3, 5), (64, 2, 8, 2),
                                       (128, 1, 7, 4), (64, 1, 9, 4), (128, 1, 12, 6)])
def test_attention_lengths_and_rows(dtype, fmt, d, Hkv, G, R):
    B = len(LENS)
    cache, table, g = filled(B, Hkv, d, dtype, fmt, LENS, seed=d + G)
    q = torch.randn(B, R, G * Hkv, d, generator=g).to(dtype).cuda()
    ws = torch.zeros(skv.paged_attn_workspace_bytes(B, R, G * Hkv, Hkv, d, table.shape[1]), dtype=torch.uint8, device="cuda")
    out, lse = skv.paged_attn(q, cache, table, i32(LENS), workspace=ws)
    ok(ws)
    for b in range(B):
        ref.check_attention(out[b], lse[b], reference(q, cache, table, LENS, b), dtype, fmt, f"len {LENS[b]}")
    again, lse2 = skv.paged_attn(q, cache, table, i32(LENS), workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,fmt", [(BF, "e4m3"), (BF, "raw"), (F32, "raw"), (F32, "e4m3")])
@pytest.mark.parametrize("window,softcap,alibi,scale", [(1, 0.0, False, None), (16, 0.0, True, None), (100, 20.0, False, None),
                                                        (0, 5.0, True, 0.3), (17, 30.0, True, -0.05)])
def test_attention_options(dtype, fmt, window, softcap, alibi, scale):
    d, Hkv, G, R = 128, 2, 4, 1
    lens = [500, 1, 0, 97, 64, 260, 40, 18]
    first = [123, 0, 5, 97, 63, -4, 1000, 2]
    B = len(lens)
    cache, table, g = filled(B, Hkv, d, dtype, fmt, lens, seed=window + 1)
    q = torch.randn(B, R, G * Hkv, d, generator=g).to(dtype).cuda()
    slopes = torch.exp2(-torch.arange(1, G * Hkv + 1).float()).cuda() if alibi else None
    out, lse = skv.paged_attn(q, cache, table, i32(lens), first=i32(first), window=window, softcap=softcap, slopes=slopes,
                              scale=scale)
    sl = None if slopes is None else slopes.double().cpu().numpy()
    for b in range(B):
        r = reference(q, cache, table, lens, b, first=first[b], window=window, softcap=softcap, slopes=sl, scale=scale)
        ref.check_attention(out[b], lse[b], r, dtype, fmt, f"sequence {b}")


@pytest.mark.parametrize("dtype,fmt", [(BF, "e4m3"), (F32, "raw")])
def test_attention_joins_a_prior(dtype, fmt):
    """Attention over the first part, then over the rest with the first as prior, equals the formula of the join on
    the separately computed halves; with a prior of no keys it is the attention itself, bit for bit."""
    d, Hkv, G, R = 128, 2, 7, 1
    lens, cut = [400, 64, 90, 33, 0], [150, 64, 0, 20, 0]
    B = len(lens)
    cache, table, g = filled(B, Hkv, d, dtype, fmt, lens, seed=2)
    q = torch.randn(B, R, G * Hkv, d, generator=g).to(dtype).cuda()
    head, head_lse = skv.paged_attn(q, cache, table, i32(cut))
    tail, tail_lse = skv.paged_attn(q, cache, table, i32(lens), first=i32(cut))
    both, both_lse = skv.paged_attn(q, cache, table, i32(lens), first=i32(cut), prior=(head, head_lse))
    a, b, la, lb = (t.double() for t in (head, tail, head_lse, tail_lse))
    z = torch.logaddexp(la, lb)
    w, u = (torch.where(z > -math.inf, torch.exp(x - z), 0.0)[..., None] for x in (la, lb))
    want = w * a + u * b
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    # the tail enters unrounded (half an ulp of its own rounding), the sum is rounded once; weights in fp32
    bound = half * (u * b.abs() + want.abs()) + 2.0 ** -20 * (w * a.abs() + u * b.abs()) + 1e-37
    assert torch.all((both.double() - want).abs() <= bound * (1 + half))
    fin = z > -math.inf
    assert torch.all((both_lse.double() - z).abs()[fin] <= 2.0 ** -21 + 2.0 ** -22 * z.abs()[fin])
    assert torch.equal(both_lse == -math.inf, z == -math.inf) and not both[4].any()
    none = (torch.full_like(head, math.nan), torch.full_like(head_lse, -math.inf))
    same, same_lse = skv.paged_attn(q, cache, table, i32(lens), first=i32(cut), prior=none)
    assert torch.equal(same, tail) and torch.equal(same_lse, tail_lse)
    # the outputs may replace the prior's
    keep = head.clone()
    skv.paged_attn(q, cache, table, i32(lens), first=i32(cut), prior=(keep, head_lse), out=keep)
    assert torch.equal(keep, both)
    with pytest.raises(skv.SkvError):
        skv.paged_attn(q, cache, table, i32(lens), prior=(head, head_lse), lse=head_lse)


@pytest.mark.parametrize("fmt", ["e4m3", "raw"])
def test_attention_long_ragged_batch_and_determinism(fmt):
    """Units of very unequal length over the whole grid: pieces, joins and one-piece units; the same bits again."""
    d, Hkv, G, R = 128, 3, 7, 1
    lens = [9000, 1, 4097, 33, 0, 2500, 640, 12]
    B = len(lens)
    cache, table, g = filled(B, Hkv, d, BF, fmt, lens, seed=9)
    q = torch.randn(B, R, G * Hkv, d, generator=g).bfloat16().cuda()
    ws = torch.zeros(skv.paged_attn_workspace_bytes(B, R, G * Hkv, Hkv, d, table.shape[1]), dtype=torch.uint8, device="cuda")
    out, lse = skv.paged_attn(q, cache, table, i32(lens), workspace=ws)
    for b in (0, 1, 2, 3, 4, 6):
        ref.check_attention(out[b], lse[b], reference(q, cache, table, lens, b), BF, fmt, f"len {lens[b]}")
    for _ in range(3):
        o, l = skv.paged_attn(q, cache, table, i32(lens), workspace=ws)
        assert torch.equal(o, out) and torch.equal(l, lse)
    # a larger page table changes nothing that is seen
    wide = torch.full((B, table.shape[1] + 37), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    o, l = skv.paged_attn(q, cache, wide, i32(lens))
    assert torch.equal(o, out) and torch.equal(l, lse)
    ok(ws)


@pytest.mark.parametrize("dtype,fmt", [(BF, "e4m3"), (BF, "raw"), (F32, "raw")])
@pytest.mark.parametrize("d,B,Hkv,G", [(64, 260, 63, 1), (128, 512, 24, 1), (128, 150, 40, 20)])
def test_attention_many_short_units(dtype, fmt, d, B, Hkv, G):
    """Far more (sequence, head) units than CTAs, so that a CTA lays its pieces out several times over; the sequences
    share a few pages (one prefix), and each must give what a batch of its own gives."""
    lens = [(7 * b) % 41 for b in range(B)]
    g = torch.Generator().manual_seed(B)
    cache, _ = make(1, Hkv, d, dtype, fmt, [64])
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    x = rand(g, 2 * 41, Hkv, d, dtype=dtype).cuda()
    skv.cache_append(x[:41], x[41:], cache, table[:1], i32([0]))
    q = torch.randn(B, 1, G * Hkv, d, generator=g).to(dtype).cuda()
    ws = torch.zeros(skv.paged_attn_workspace_bytes(B, 1, G * Hkv, Hkv, d, 1), dtype=torch.uint8, device="cuda")
    out, lse = skv.paged_attn(q, cache, table, i32(lens), workspace=ws)
    ok(ws)
    for b in list(range(0, B, 37)) + [B - 1]:
        ref.check_attention(out[b], lse[b], reference(q, cache, table, lens, b), dtype, fmt, f"sequence {b}")
    # the rest against the same rows in plain torch, all at once
    (k, v), _ = ref.read_rows(cache, [0], 0, 41)
    check_shared(out, lse, q, *(torch.from_numpy(t).cuda().permute(1, 0, 2) for t in (k, v)), lens, dtype, fmt)


def check_shared(out, lse, q, k, v, lens, dtype, fmt):
    """Sequences that share their keys k, v [Hkv, t, d] (fp64), each seeing the first lens[b], within the bounds of
    cache_reference.attention_bounds, row by row (the 2^-25 of tiny weights goes into 2^-15)."""
    B, _, Hq, d = q.shape
    Hkv, T, _ = k.shape
    x = q.double().view(B, Hkv, Hq // Hkv, d)
    seen = torch.arange(T, device="cuda") < i32(lens)[:, None, None, None]
    s = (torch.einsum("bhgd,htd->bhgt", x, k) / math.sqrt(d)).masked_fill(~seen, -math.inf)
    size = torch.einsum("bhgd,htd->bhgt", x.abs(), k.abs()).amax(-1) / math.sqrt(d)
    dlogit = (2.0 ** -24 * (d + 12) * size + 2.0 ** -21).reshape(B, 1, -1)
    want = torch.logsumexp(s, -1).view(B, 1, -1)
    fin = want > -math.inf
    assert torch.equal(lse > -math.inf, fin)
    assert torch.all(((lse.double() - want).abs() <= dlogit + 2.0 ** -20 + 2.0 ** -22 * want.abs())[fin])
    p = torch.nan_to_num(torch.softmax(s, -1))
    o = torch.einsum("bhgt,htd->bhgd", p, v).reshape(B, 1, -1, d)
    mass = torch.einsum("bhgt,htd->bhgd", p, v.abs()).reshape(B, 1, -1, d)
    weight = 0.0 if dtype == F32 else 2.0 ** -11 if fmt == "e4m3" else 2.0 ** -8
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    assert torch.all((out.double() - o).abs() <= mass * (weight + 2.0 ** -15 + 2 * dlogit[..., None]) * (1 + half) + half * o.abs() + 1e-30)


@pytest.mark.parametrize("dtype,fmt,d,G", [(BF, "e4m3", 128, 1), (BF, "raw", 128, 7), (BF, "e4m3", 64, 8), (BF, "e4m3", 128, 12),
                                           (BF, "raw", 64, 28), (F32, "raw", 64, 2), (F32, "e4m3", 128, 3)])
def test_attention_many_long_units(dtype, fmt, d, G):
    """Pieces of more groups than a warp looks page ids up for at once: 48 sequences of up to 8,192 tokens that share
    their pages (one prefix), 8 KV heads."""
    B, Hkv, T = 48, 8, 8192
    lens = [T - 61 * b for b in range(B)]
    cache, table = make(1, Hkv, d, dtype, fmt, [T], seed=4)
    g = torch.Generator(device="cuda").manual_seed(d + G)
    k, v = (torch.randn(T, Hkv, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    skv.cache_append(k, v, cache, table, i32([0]))
    k, v = skv.cache_read(cache, table, [0], [T])
    q = torch.randn(B, 1, G * Hkv, d, generator=g, device="cuda").to(dtype)
    out, lse = skv.paged_attn(q, cache, table.expand(B, -1).contiguous(), i32(lens))
    check_shared(out, lse, q, k.view(Hkv, T, d).double(), v.view(Hkv, T, d).double(), lens, dtype, fmt)


@pytest.mark.parametrize("dtype,fmt,d", [(BF, "e4m3", 128), (BF, "raw", 64), (F32, "e4m3", 64)])
@pytest.mark.parametrize("B,Hkv,G", [(1, 1, 7), (1, 2, 28), (1, 5, 1), (2, 3, 4), (3, 3, 12)])
def test_attention_few_long_units(dtype, fmt, d, B, Hkv, G):
    """Units of tens to hundreds of pieces, joined in one step or two; a second call on the same workspace finds its
    counters as the first did."""
    T = 50000
    lens = [T - 7777 * b for b in range(B)]
    cache, table = make(1, Hkv, d, dtype, fmt, [T], seed=4)
    g = torch.Generator(device="cuda").manual_seed(d + G)
    k, v = (torch.randn(T, Hkv, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    skv.cache_append(k, v, cache, table, i32([0]))
    k, v = skv.cache_read(cache, table, [0], [T])
    q = torch.randn(B, 1, G * Hkv, d, generator=g, device="cuda").to(dtype)
    table = table.expand(B, -1).contiguous()
    ws = torch.zeros(skv.paged_attn_workspace_bytes(B, 1, G * Hkv, Hkv, d, table.shape[1]), dtype=torch.uint8, device="cuda")
    out, lse = skv.paged_attn(q, cache, table, i32(lens), workspace=ws)
    ok(ws)
    check_shared(out, lse, q, k.view(Hkv, T, d).double(), v.view(Hkv, T, d).double(), lens, dtype, fmt)
    again, lse2 = skv.paged_attn(q, cache, table, i32(lens), workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fmt", ["e4m3", "raw"])
def test_attention_peaked_and_unequal_scales(fmt):
    """One key far above the others, values of very unequal size, equal keys: the running maximum and the value
    scales meet their extremes."""
    d, Hkv, G = 128, 1, 7
    n = 500
    g = torch.Generator().manual_seed(4)
    k, v = rand(g, n, Hkv, d), rand(g, n, Hkv, d)
    k[321] *= 30
    k[17] = k[18]
    v *= torch.exp2(torch.randint(-12, 13, (n, 1, 1), generator=g).float()).bfloat16()
    v[40:60] = 0
    q = torch.randn(3, 1, G, d, generator=g).bfloat16()
    q[1] *= 8
    q[2] = 0
    cache, table = make(3, Hkv, d, BF, fmt, [n] * 3)
    for b in range(3):
        skv.cache_append(k.cuda(), v.cuda(), cache, table[b:b + 1], i32([0]))
    q = q.cuda()
    out, lse = skv.paged_attn(q, cache, table, i32([n] * 3))
    for b in range(3):
        ref.check_attention(out[b], lse[b], reference(q, cache, table, [n] * 3, b), BF, fmt, f"row {b}")


@pytest.mark.parametrize("dtype,fmt", [(BF, "e4m3"), (BF, "raw"), (F32, "e4m3")])
@pytest.mark.parametrize("d,G,size", [(128, 7, 2.0 ** -30), (64, 2, 2.0 ** -60), (128, 12, 2.0 ** -10), (64, 28, 2.0 ** 40)])
def test_values_of_zeros_leave_small_values_alone(dtype, fmt, d, G, size):
    """Keys with the largest logits whose values are all zeros (of either sign) beside values far below and above 1: the
    zeros add to the partition and to nothing else."""
    n, Hkv = 333, 1
    g = torch.Generator().manual_seed(d + G)
    k, v = torch.randn(n, Hkv, d, generator=g), torch.randn(n, Hkv, d, generator=g) * size
    q = torch.randn(2, 1, G, d, generator=g)
    q[0] = q[0, 0, 0]
    k[[0, 50, 200]] = 0.3 * q[0, 0, 0]                      # far above the others for the first sequence's rows
    v[[0, 50, 120, 200, 332]] = 0.0
    v[200] = -v[200]
    cache, table = make(2, Hkv, d, dtype, fmt, [n] * 2)
    for b in range(2):
        skv.cache_append(k.to(dtype).cuda(), v.to(dtype).cuda(), cache, table[b:b + 1], i32([0]))
    q = q.to(dtype).cuda()
    out, lse = skv.paged_attn(q, cache, table, i32([n] * 2))
    for b in range(2):
        ref.check_attention(out[b], lse[b], reference(q, cache, table, [n] * 2, b), dtype, fmt, f"sequence {b}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,G", [(128, 7), (64, 12)])
@pytest.mark.parametrize("at", [0, 20, 299])
@pytest.mark.parametrize("gap,top,rest", [(80, 0.0, 1.0), (200, 0.0, 1.0), (180, 2.0 ** -100, 2.0 ** 110), (5, 2.0 ** 110, 2.0 ** -90)])
def test_values_of_scales_far_apart(dtype, d, G, at, gap, top, rest):
    """One key whose logit is `gap` above the others', which are about equal, and values of scales at the two ends of the
    format's range, or zeros: finite results, none of them lost."""
    n = 300
    g = torch.Generator().manual_seed(at + G)
    k, v = torch.randn(n, 1, d, generator=g) / 64, torch.randn(n, 1, d, generator=g) * rest
    q = torch.ones(1, 1, G, d)
    k[at] = gap / math.sqrt(d)
    v[at] = torch.randn(1, d, generator=g) * top
    cache, table = make(1, 1, d, dtype, "e4m3", [n])
    skv.cache_append(k.to(dtype).cuda(), v.to(dtype).cuda(), cache, table, i32([0]))
    q = q.to(dtype).cuda()
    out, lse = skv.paged_attn(q, cache, table, i32([n]))
    ref.check_attention(out[0], lse[0], reference(q, cache, table, [n], 0), dtype, "e4m3")


@pytest.mark.parametrize("dtype,fmt", [(BF, "e4m3"), (BF, "raw"), (F32, "raw")])
def test_nan_stays_where_it_is_seen(dtype, fmt):
    """A NaN key or value poisons the rows that see it and no other; behind the window, before `first` and behind
    the length it is never read into a result."""
    d, Hkv, G, n = 64, 2, 4, 100
    cache, table, g = filled(1, Hkv, d, dtype, fmt, [n], seed=1)
    q = torch.randn(1, 1, Hkv * G, d, generator=g).to(dtype).cuda()
    clean, clean_lse = skv.paged_attn(q, cache, table, i32([n]), first=i32([41]))
    bad = torch.full((1, Hkv, d), math.nan, dtype=dtype, device="cuda")
    bad[0, 1] = 1.0
    skv.cache_append(bad, bad, cache, table, i32([40]))
    for kw in (dict(first=i32([41])), dict(window=n - 41)):
        o, l = skv.paged_attn(q, cache, table, i32([n]), **kw)
        assert torch.equal(o, clean) and torch.equal(l, clean_lse)
    o, l = skv.paged_attn(q, cache, table, i32([n]))
    assert o[:, :, :G].isnan().all() and l[:, :, :G].isnan().all() and o[:, :, G:].isfinite().all()


def test_attention_device_errors_are_reported():
    d, Hkv, G, lens = 128, 2, 7, [200, 130]
    cache, table, g = filled(2, Hkv, d, BF, "e4m3", lens, seed=1)
    q = torch.randn(2, 1, Hkv * G, d, generator=g).bfloat16().cuda()
    ws = torch.zeros(skv.paged_attn_workspace_bytes(2, 1, 14, 2, d, table.shape[1]), dtype=torch.uint8, device="cuda")
    bad = table.clone()
    bad[0, 1] = cache.num_pages
    out, lse = skv.paged_attn(q, cache, bad, i32(lens), workspace=ws)
    assert skv.workspace_error(ws) == (_lib.SKV_ERR_DEVICE, _lib.FLAG_BAD_PAGE)
    (k, v), (_, vs) = ref.read_rows(cache, table[0].tolist(), 0, 200)   # the page's 64 tokens are skipped
    keep = np.r_[0:64, 128:200]
    r = ref.Attn(q[0].double().cpu().numpy(), k[keep], v[keep], vs[keep], 199, 0)
    ref.check_attention(out[0], lse[0], r, BF, "e4m3", "page skipped")
    ref.check_attention(out[1], lse[1], reference(q, cache, table, lens, 1), BF, "e4m3")
    out, lse = skv.paged_attn(q, cache, table, i32([-5, 130]), workspace=ws)
    assert skv.workspace_error(ws) == (_lib.SKV_ERR_DEVICE, _lib.FLAG_BAD_LENS)
    assert not out[0].any() and torch.all(lse[0] == -math.inf)
    ref.check_attention(out[1], lse[1], reference(q, cache, table, lens, 1), BF, "e4m3")
    ok(ws)


def test_host_values_are_checked():
    cache, table, _ = filled(1, 1, 64, BF, "raw", [9])
    q = torch.zeros(1, 1, 1, 64, dtype=BF, device="cuda")
    for kw in (dict(window=-1), dict(window=(1 << 32) + 1), dict(scale=0.0)):
        with pytest.raises(ValueError):
            skv.paged_attn(q, cache, table, i32([9]), **kw)
    for first, T in (([0], [-1]), ([-1], [1]), ([0], [(1 << 32) + 3]), ([1 << 33], [1]), ([0, 0], [1])):
        with pytest.raises(ValueError):
            skv.cache_read(cache, table, first, T)
    with pytest.raises(skv.SkvError):
        skv.cache_read(cache, table, [0], [65])
    k, _ = skv.cache_read(cache, table, np.array([1]), np.array([3]))
    assert k.shape == (3, 64)
    bad = torch.zeros(2, 1, 64, dtype=BF, device="cuda")
    for args in ((bad[:, :, :32], bad[:, :, :32]), (bad, bad[:1]), (bad.float(), bad.float()), (bad.transpose(0, 2), bad.transpose(0, 2))):
        with pytest.raises(ValueError):
            skv.cache_append(*args, cache, table, i32([9]))
    with pytest.raises(ValueError):
        skv.cache_append(bad, bad, cache, table, torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        skv.cache_append(bad, bad, cache, table.long(), i32([9]))
    with pytest.raises(skv.SkvError):   # rows that do not start on 16 bytes
        x = torch.zeros(2, 2, 68, dtype=BF, device="cuda")[:, :1, 2:66]
        skv.cache_append(x, x, cache, table, i32([9]))


def test_strided_queries_other_stream_and_shared_workspace():
    d, Hkv, G, R, lens = 128, 2, 4, 2, [300, 77, 5]
    B, Hq = 3, 8
    cache, table, g = filled(B, Hkv, d, BF, "e4m3", lens, seed=6)
    x = torch.randn(B, R, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    q = x[:, :, :Hq]
    others = ((64, 1, 1, 64, 40), (1, 8, 4, 128, 3000))
    size = max([skv.paged_attn_workspace_bytes(B, R, Hq, Hkv, d, table.shape[1])] +
               [skv.paged_attn_workspace_bytes(B2, R2, H2, 1, d2, skv.token_pages_for(n)) for B2, R2, H2, d2, n in others])
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = skv.paged_attn(q.contiguous(), cache, table, i32(lens), workspace=ws)
    got = skv.paged_attn(q, cache, table, i32(lens), workspace=ws)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = skv.paged_attn(q, cache, table, i32(lens), stream=s)   # everything it allocates belongs to that stream
    s.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    # other shapes through the same workspace, and the first again
    for B2, R2, H2, d2, n in others:
        c2, t2, _ = filled(B2, 1, d2, BF, "raw", [n] * B2, seed=n)
        q2 = torch.randn(B2, R2, H2, d2, generator=g).bfloat16().cuda()
        a = skv.paged_attn(q2, c2, t2, i32([n] * B2), workspace=ws)
        b = skv.paged_attn(q2, c2, t2, i32([n] * B2))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        got = skv.paged_attn(q, cache, table, i32(lens), workspace=ws)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    ok(ws)


def test_append_and_attention_in_a_replayed_graph():
    """A captured decode step (append in place, attend) replayed over page ends equals the same calls made one by one."""
    B, Hkv, G, d, steps = 2, 2, 7, 128, 40
    start = [50, 127]
    cache, table = make(B, Hkv, d, BF, "e4m3", [256, 256], seed=8)
    g = torch.Generator().manual_seed(8)
    pre = rand(g, sum(start), Hkv, d).cuda()
    xs, qs = rand(g, steps, B, Hkv, d).cuda(), torch.randn(steps, B, 1, Hkv * G, d, generator=g).bfloat16().cuda()
    ws = torch.zeros(skv.paged_attn_workspace_bytes(B, 1, Hkv * G, Hkv, d, 4), dtype=torch.uint8, device="cuda")
    x, q, lens = xs[0].clone(), qs[0].clone(), i32(start)

    def begin():
        cache.pages.fill_(255)
        skv.cache_append(pre, pre, cache, table, i32([0, 0]), cu_new=i32([0, start[0], sum(start)]), workspace=ws)
        lens.copy_(i32(start))

    begin()
    want = []
    for i in range(steps):
        skv.cache_append(xs[i], xs[i], cache, table, lens, new_lens=lens, workspace=ws)
        want.append([t.clone() for t in skv.paged_attn(qs[i], cache, table, lens, workspace=ws)])
    begin()
    out, lse = torch.empty_like(q), torch.empty(B, 1, Hkv * G, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        skv.cache_append(x, x, cache, table, lens, new_lens=lens, workspace=ws)
        skv.paged_attn(q, cache, table, lens, out=out, lse=lse, workspace=ws)
    for i in range(steps):
        x.copy_(xs[i])
        q.copy_(qs[i])
        graph.replay()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), f"step {i}"
    assert lens.tolist() == [s + steps for s in start]
    ok(ws)


def test_offsets_beyond_32_bits():
    """Pages that lie more than 4 GiB into the cache."""
    Hkv, d = 8, 128
    num = 34000
    cache = skv.TokenCache(num, Hkv, d, BF, format="e4m3")
    assert cache.nbytes() > 1 << 32
    table = i32([[num - 1, 5, num - 2, num // 2 + 9]])
    g = torch.Generator().manual_seed(3)
    k, v = rand(g, 200, Hkv, d).cuda(), rand(g, 200, Hkv, d).cuda()
    skv.cache_append(k, v, cache, table, i32([0]))
    small, t2 = make(1, Hkv, d, BF, "e4m3", [200])
    skv.cache_append(k, v, small, t2, i32([0]))
    for a, b in zip(skv.cache_read(cache, table, [0], [200]), skv.cache_read(small, t2, [0], [200])):
        assert torch.equal(a, b)
    q = torch.randn(1, 1, 16, d, generator=g).bfloat16().cuda()
    a, b = skv.paged_attn(q, cache, table, i32([200])), skv.paged_attn(q, small, t2, i32([200]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------------------
# as they are used together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["e4m3", "raw"])
def test_cache_then_coarsen_then_join(fmt):
    """A history kept in the cache, its older part read back and coarsened, and decode steps that append a token and
    attend over both: outputs and partitions are those of one attention over the nodes and the exact tokens."""
    B, Hq, Hkv, d = 2, 14, 2, 128
    T, cut = [700, 431], [512, 300]
    w = workloads.Workload("cache", 5, B=B, Hq=Hq, Hkv=Hkv, d=d, R=1, dtype="bf16", T=0, regimes=6)
    ks, vs, _ = workloads.make_kv(w, torch.device("cuda"), T_list=T)
    cache, table = make(B, Hkv, d, BF, fmt, [t + 8 for t in T], seed=2)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    rows = [torch.stack([workloads.unit_rows(x, T, Hkv, b, h) for h in range(Hkv)], 1) for x in (ks, vs) for b in range(B)]
    lens = skv.cache_append(torch.cat(rows[:B]), torch.cat(rows[B:]), cache, table, i32([0] * B),
                            cu_new=i32([0, T[0], sum(T)]), workspace=ws)
    k, v = skv.cache_read(cache, table, [0] * B, cut, workspace=ws)
    N, S, W = [40, 25], 4, 16
    pages = [skv.pages_for(t, n, S, W) for t, n in zip(cut, N)]
    ntable, num = workloads.page_assignment(B, Hkv, pages, True, 1)
    pool = skv.NodePool(num, d, BF)
    nlens = skv.coarsen(k, v, Hkv, cut, N, S, W, 3, pool, ntable.cuda())
    g = torch.Generator().manual_seed(2)
    aws = torch.zeros(skv.paged_attn_workspace_bytes(B, 1, Hq, Hkv, d, table.shape[1]), dtype=torch.uint8, device="cuda")
    for step in range(3):
        x = rand(g, 2 * B, Hkv, d).cuda()
        skv.cache_append(x[:B], x[B:], cache, table, lens, new_lens=lens, workspace=ws)
        q = torch.randn(B, 1, Hq, d, generator=g).bfloat16().cuda()
        prior = skv.decode_attn(q, Hkv, pool, ntable.cuda(), nlens)
        out, lse = skv.paged_attn(q, cache, table, lens, first=i32(cut), prior=prior, workspace=aws)
        units = gpu_units(pool, ntable.cuda(), nlens, B, Hkv)
        node_out, node_lse = oracle.decode(q.double().cpu().numpy(), units)
        for b in range(B):
            r = reference(q, cache, table, lens.tolist(), b, first=cut[b])
            z = np.logaddexp(r.lse, node_lse[b])
            a, c = np.exp(r.lse - z)[..., None], np.exp(node_lse[b] - z)[..., None]
            want = a * r.out + c * node_out[b]
            o, l = out[b].double().cpu().numpy(), lse[b].double().cpu().numpy()
            bo, bl = ref.attention_bounds(r, BF, fmt)
            # decode_attn's own bars (2e-2 absolute on outputs, 1e-3 on lse) weighted by its share, and one rounding
            dz = c[..., 0] * 1e-3 + bl
            shift = 2 * dz[..., None] * (a * np.abs(r.out) + c * np.abs(node_out[b]))
            assert np.all(np.abs(l - z) <= dz + 2.0 ** -20)
            assert np.all(np.abs(o - want) <= a * bo + c * (2e-2 + 2.0 ** -8 * np.abs(node_out[b])) + shift
                          + 2.0 ** -8 * np.abs(want))
    ok(ws)
    ok(aws)
