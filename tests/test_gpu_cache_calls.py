"""Calls of the exact-token cache that its documentation allows, beyond the ordinary ones: offsets in any order, options
with every kind of row tile, joins of many rows and passes, and arguments at the ends of their ranges."""
import math

import numpy as np
import pytest
import torch

import cache_reference as ref
import compressed_decode_attention_equal_b200 as skv
from compressed_decode_attention_equal_b200 import _lib
from test_gpu_cache import BF, F32, filled, i32, make, ok, rand, reference

pytestmark = pytest.mark.gpu


def granted(cu, n):
    """Rows of each sequence by the documented rule: upwards within n, and behind the rows of the sequences before."""
    end, got = 0, []
    for c0, c1 in zip(cu, cu[1:]):
        fine = end <= c0 <= c1 <= n
        got.append((c0, c1) if fine else None)
        end = c1 if fine else end
    return got


OFFSETS = [([0, 5, 3, 8], 8), ([0, 5, 3, 6], 6), ([3, 1, 4, 4, 9], 9), ([-2, 3, 5, 7], 7), ([0, 4, 20, 6, 8], 8), ([8, 0, 8], 8),
           ([2, 2, 2], 5), ([0, 9], 8), ([5, 2, 7, 3, 7, 7, 9], 12), ([0, 3, 6, 1, 6, 6, 11], 11)]


@pytest.mark.parametrize("d,Hkv,dtype,fmt", [(128, 4, BF, "e4m3"), (64, 3, F32, "raw"), (128, 1, BF, "raw")])
@pytest.mark.parametrize("cu,n", OFFSETS + [("random", 400)])
def test_offsets_in_any_order_never_count_what_was_not_written(d, Hkv, dtype, fmt, cu, n):
    g = torch.Generator().manual_seed(n)
    if cu == "random":
        up = np.sort(np.random.RandomState(1).randint(0, n + 1, 151))
        up[[20, 77, 78, 140]] = up[[90, 10, 150, 0]]        # a few out of place
        cu = up.tolist()
    B = len(cu) - 1
    got = granted(cu, n)
    old = [(7 * b) % 70 for b in range(B)]
    want_lens = [o + (r[1] - r[0] if r else 0) for o, r in zip(old, got)]
    cache, table = make(B, Hkv, d, dtype, fmt, [o + n for o in old], seed=5)
    want = skv.TokenCache(cache.num_pages, Hkv, d, dtype, format=fmt, device="cpu", pages=cache.pages.cpu().clone())
    k, v = rand(g, n, Hkv, d, dtype=dtype), rand(g, n, Hkv, d, dtype=dtype)
    for b, r in enumerate(got):
        if r:
            ref.write_rows(want, table[b].tolist(), old[b], k[r[0]:r[1]].double().numpy(), v[r[0]:r[1]].double().numpy())
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens = i32(old)
    assert skv.cache_append(k.cuda(), v.cuda(), cache, table, lens, cu_new=i32(cu), new_lens=lens, workspace=ws).tolist() == want_lens
    if None in got:
        assert skv.workspace_error(ws) == (_lib.SKV_ERR_DEVICE, _lib.FLAG_BAD_LENS)
    ok(ws)
    a, w = cache.pages.cpu(), want.pages
    if fmt == "e4m3":   # -0 and +0 are both right where a value rounds to zero
        a, w = (torch.where(t == 128, 0, t) for t in (a, w))
    assert torch.equal(a, w)


@pytest.mark.parametrize("dtype,fmt", [(BF, "e4m3"), (BF, "raw"), (F32, "raw"), (F32, "e4m3")])
@pytest.mark.parametrize("d,Hkv,G,R", [(64, 2, 4, 1), (64, 1, 6, 2), (128, 2, 3, 5), (128, 1, 9, 4), (64, 2, 7, 4), (128, 1, 5, 9)])
@pytest.mark.parametrize("window,softcap,alibi,scale", [(0, 0.0, True, None), (47, 4.0, False, 0.2), (0, 30.0, True, -0.05)])
def test_options_with_every_row_tile(dtype, fmt, d, Hkv, G, R, window, softcap, alibi, scale):
    """Window, start, cap, bias and scale with one, two and four tiles of rows and with several passes; starts and ends in
    both halves of the two groups that are copied at once at d = 64."""
    lens = [500, 1, 97, 64, 260, 40, 30, 333, 48, 300, 80, 32]
    first = [123, 0, 97, 63, -4, 1000, 17, 240, 16, 31, 48, 0]
    B = len(lens)
    cache, table, g = filled(B, Hkv, d, dtype, fmt, lens, seed=d + window)
    q = torch.randn(B, R, G * Hkv, d, generator=g).to(dtype).cuda()
    slopes = torch.exp2(-torch.arange(1, G * Hkv + 1).float() / 2).cuda() if alibi else None
    ws = torch.zeros(skv.paged_attn_workspace_bytes(B, R, G * Hkv, Hkv, d, table.shape[1]), dtype=torch.uint8, device="cuda")
    out, lse = skv.paged_attn(q, cache, table, i32(lens), first=i32(first), window=window, softcap=softcap, slopes=slopes,
                              scale=scale, workspace=ws)
    ok(ws)
    sl = None if slopes is None else slopes.double().cpu().numpy()
    for b in range(B):
        r = reference(q, cache, table, lens, b, first=first[b], window=window, softcap=softcap, slopes=sl, scale=scale)
        ref.check_attention(out[b], lse[b], r, dtype, fmt, f"sequence {b}")


@pytest.mark.parametrize("dtype,fmt,d,Hkv,G,R", [(BF, "e4m3", 128, 2, 7, 4), (BF, "raw", 64, 1, 6, 3), (BF, "e4m3", 64, 2, 4, 9),
                                                 (BF, "raw", 128, 1, 28, 2), (F32, "raw", 64, 2, 3, 5), (F32, "e4m3", 128, 1, 9, 1)])
def test_join_of_many_rows_and_passes(dtype, fmt, d, Hkv, G, R):
    """Both halves of a history joined, with several rows per sequence and several passes, over units cut into pieces:
    one attention over all of it, within the bounds of one."""
    lens, cut = [4000, 64, 90, 33, 7], [1500, 64, 0, 20, 3]
    B = len(lens)
    cache, table, g = filled(B, Hkv, d, dtype, fmt, lens, seed=2)
    q = torch.randn(B, R, G * Hkv, d, generator=g).to(dtype).cuda()
    head = skv.paged_attn(q, cache, table, i32(cut))
    out, lse = skv.paged_attn(q, cache, table, i32(lens), first=i32(cut), prior=head)
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    for b in range(B):
        r = reference(q, cache, table, lens, b)
        bo, bl = ref.attention_bounds(r, dtype, fmt)
        # the head's share enters rounded to the dtype: half a step of it, at most of the mass of all keys
        bo = bo + half * r.mass
        assert np.all(np.abs(out[b].double().cpu().numpy() - r.out) <= bo)
        assert np.all(np.abs(lse[b].double().cpu().numpy() - r.lse) <= 2 * bl + 2.0 ** -20)


@pytest.mark.parametrize("dtype,fmt,d,G,R", [(BF, "e4m3", 128, 4, 1), (BF, "raw", 64, 3, 4), (F32, "raw", 128, 2, 1)])
@pytest.mark.parametrize("softcap,scale", [(0.0, None), (5.0, 0.3)])
def test_join_under_cap_and_bias(dtype, fmt, d, G, R, softcap, scale):
    """A prior of the same scale, cap and bias joins as documented: its distances counted from its own last token, so that
    slope * (lens - n) comes off its partition. The result is one attention over all keys."""
    Hkv, lens, cut = 2, [900, 70, 64, 33], [400, 70, 1, 0]
    B = len(lens)
    cache, table, g = filled(B, Hkv, d, dtype, fmt, lens, seed=4)
    q = torch.randn(B, R, G * Hkv, d, generator=g).to(dtype).cuda()
    slopes = torch.exp2(-torch.arange(1, G * Hkv + 1).float()).cuda()
    kw = dict(softcap=softcap, scale=scale, slopes=slopes)
    head, head_lse = skv.paged_attn(q, cache, table, i32(cut), **kw)
    head_lse = head_lse - slopes * (i32(lens) - i32(cut))[:, None, None]
    out, lse = skv.paged_attn(q, cache, table, i32(lens), first=i32(cut), prior=(head, head_lse), **kw)
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    for b in range(B):
        r = reference(q, cache, table, lens, b, softcap=softcap, scale=scale, slopes=slopes.double().cpu().numpy())
        bo, bl = ref.attention_bounds(r, dtype, fmt)
        # the head's share enters rounded to the dtype; its shifted partition is one more fp32 sum of up to |lse| + bias
        bl = 2 * bl + 2.0 ** -20 + 2.0 ** -22 * float(slopes[0]) * lens[b]
        bo = bo + half * r.mass + 2 * bl[..., None] * r.mass
        assert np.all(np.abs(out[b].double().cpu().numpy() - r.out) <= bo)
        assert np.all(np.abs(lse[b].double().cpu().numpy() - r.lse) <= bl)


@pytest.mark.parametrize("kw", [dict(scale=0.0), dict(scale=-0.0), dict(scale=1e-46), dict(scale=-1e-50), dict(softcap=1e-46)])
def test_a_scale_or_cap_that_is_zero_in_32_bits_is_refused(kw):
    """Zero stands for the defaults below the binding: 1 / sqrt(d) and no cap, the opposite of what was asked for."""
    cache, table, g = filled(1, 1, 64, BF, "raw", [9])
    q = torch.randn(1, 1, 1, 64, generator=g).bfloat16().cuda()
    with pytest.raises(ValueError, match="zero in 32 bits"):
        skv.paged_attn(q, cache, table, i32([9]), **kw)
    out, _ = skv.paged_attn(q, cache, table, i32([9]), **{k: math.copysign(1e-44, v) for k, v in kw.items()})
    (_, v), _ = ref.read_rows(cache, table[0].tolist(), 0, 9)
    assert np.all(np.abs(out[0, 0, 0].double().cpu().numpy() - v.mean(0)[0]) <= 2.0 ** -8 * np.abs(v).mean(0)[0] + 2.0 ** -14)


@pytest.mark.parametrize("dtype,fmt,d,G,R", [(BF, "e4m3", 128, 7, 1), (BF, "raw", 64, 9, 5), (F32, "raw", 128, 3, 4)])
def test_the_outputs_may_take_the_queries_place(dtype, fmt, d, G, R):
    """out = q, with units that are cut into pieces, several passes and short units among them."""
    Hkv, lens = 2, [9000, 0, 3, 700, 64]
    cache, table, g = filled(5, Hkv, d, dtype, fmt, lens, seed=7)
    q = torch.randn(5, R, G * Hkv, d, generator=g).to(dtype).cuda()
    want = skv.paged_attn(q, cache, table, i32(lens))
    out, lse = skv.paged_attn(q, cache, table, i32(lens), out=q)
    assert out is q and torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype,fmt,d,G", [(BF, "e4m3", 64, 7), (BF, "raw", 128, 12), (F32, "e4m3", 128, 2)])
def test_positions_at_the_end_of_the_range(dtype, fmt, d, G):
    """A sequence of 2^30 tokens, the most there may be, of which the last few hundred are appended, read and attended to
    through a start or a window: the bits of the same tokens at the same places of a short sequence."""
    Hkv, n, T = 2, 300, 1 << 30
    g = torch.Generator().manual_seed(d)
    x = rand(g, 2 * n, Hkv, d, dtype=dtype).cuda()
    q = torch.randn(1, 1, G * Hkv, d, generator=g).to(dtype).cuda()
    slopes = torch.exp2(-torch.arange(1, G * Hkv + 1).float()).cuda()
    skip = -n % 64                                          # both runs start at the same place of a page
    small, table = make(1, Hkv, d, dtype, fmt, [skip + n])
    far = torch.full((1, T // 64), -1, dtype=torch.int32, device="cuda")
    far[:, -table.shape[1]:] = table
    got = []
    for end, tab in ((skip + n, table), (T, far)):
        small.pages.fill_(255)
        ws = torch.zeros(skv.paged_attn_workspace_bytes(1, 1, G * Hkv, Hkv, d, tab.shape[1]), dtype=torch.uint8, device="cuda")
        lens = skv.cache_append(x[:n], x[n:], small, tab, i32([end - n]), workspace=ws)
        assert lens.tolist() == [end]
        read = skv.cache_read(small, tab, [end - n], [n], workspace=ws)
        a = skv.paged_attn(q, small, tab, lens, first=i32([end - n]), slopes=slopes, workspace=ws)
        b = skv.paged_attn(q, small, tab, lens, window=n, slopes=slopes, workspace=ws)
        ok(ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        got.append((*read, *a))
    for u, w in zip(*got):
        assert torch.equal(u, w)
    with pytest.raises(skv.SkvError):
        skv.cache_read(small, far, [T - 1], [2])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert skv.cache_append(x[:1], x[:1], small, far, i32([T]), workspace=ws).tolist() == [T]
    assert skv.workspace_error(ws) == (_lib.SKV_ERR_DEVICE, _lib.FLAG_BAD_LENS)


def test_two_captured_graphs_share_a_workspace():
    """Calls of different shapes captured into two graphs over one workspace and replayed in turns, eager calls between."""
    g = torch.Generator().manual_seed(12)
    calls = []
    for B, Hkv, G, R, d, dtype, fmt, n in ((1, 2, 7, 4, 128, BF, "e4m3", 20000), (40, 3, 1, 1, 64, F32, "raw", 500), (2, 8, 2, 1, 128, BF, "raw", 3000)):
        cache, table, _ = filled(B, Hkv, d, dtype, fmt, [n - b for b in range(B)], seed=n)
        q = torch.randn(B, R, G * Hkv, d, generator=g).to(dtype).cuda()
        calls.append((q, cache, table, i32([n - b for b in range(B)])))
    size = max(skv.paged_attn_workspace_bytes(q.shape[0], q.shape[1], q.shape[2], c.Hkv, c.d, t.shape[1]) for q, c, t, _ in calls)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = [skv.paged_attn(*c) for c in calls]
    graphs = []
    torch.cuda.synchronize()
    for order in ((0, 1, 2), (2, 0)):
        graph, outs = torch.cuda.CUDAGraph(), []
        with torch.cuda.graph(graph):
            for i in order:
                outs.append((i, *skv.paged_attn(*calls[i], workspace=ws)))
        graphs.append((graph, outs))
    for turn in range(6):
        graph, outs = graphs[turn % 2]
        for _, o, l in outs:
            o.fill_(math.nan), l.fill_(math.nan)
        graph.replay()
        o, l = skv.paged_attn(*calls[turn % 3], workspace=ws)
        assert torch.equal(o, want[turn % 3][0]) and torch.equal(l, want[turn % 3][1])
        for i, o, l in outs:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]), (turn, i)
    ok(ws)
