"""Paged attention held to bounds in which every rounding is counted one by one: what the products, the weights and
the output's type can each put into a result, and nothing for what the formula computes exactly."""
import math

import numpy as np
import pytest
import torch

import cache_reference as ref
import compressed_decode_attention_equal_b200 as skv
from test_gpu_cache import BF, F32, i32, make, reference

pytestmark = pytest.mark.gpu


def put(k, v, dtype, fmt, B=1):
    """A cache whose B sequences share the pages of rows k, v [n, Hkv, d]."""
    n, Hkv, d = k.shape
    cache, table = make(1, Hkv, d, dtype, fmt, [n])
    skv.cache_append(k.to(dtype).cuda(), v.to(dtype).cuda(), cache, table, i32([0]))
    return cache, table.expand(B, -1).contiguous()


@pytest.mark.parametrize("d,Hkv,G,R", [(128, 2, 7, 1), (64, 1, 4, 1), (128, 1, 1, 1), (128, 1, 12, 1), (64, 2, 7, 4), (128, 1, 28, 1)])
def test_weights_of_raw_caches_keep_sixteen_bits(d, Hkv, G, R):
    """The second product's weights are a bf16 number and the rest as another: 2^-16 of a weight, not bf16's 2^-8. With
    values of both signs many outputs are far smaller than the sum of their magnitudes, where 2^-8 of a weight shows
    and the output's own rounding does not. Bound: weights 2^-16, twice the logits' error, fp32 sums 2^-16 of the mass,
    and half a step of the output."""
    lens = [2, 3, 17, 40, 64, 100]
    g = torch.Generator().manual_seed(d + G)
    k, v = (torch.randn(100, Hkv, d, generator=g) for _ in range(2))
    cache, table = put(k, v, BF, "raw", len(lens))
    q = (torch.randn(len(lens), R, G * Hkv, d, generator=g) / 4).bfloat16().cuda()
    out, _ = skv.paged_attn(q, cache, table, i32(lens))
    for b in range(len(lens)):
        r = reference(q, cache, table, lens, b)
        inner = r.mass * (2.0 ** -16 + 2.0 ** -16 + 2 * r.dlogit[..., None])
        bound = inner * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(r.out) + 1e-37
        err = np.abs(out[b].double().cpu().numpy() - r.out)
        assert np.all(err <= bound), f"len {lens[b]}: {np.max(err / bound):.2f} bounds"


@pytest.mark.parametrize("dtype,d,G", [(BF, 128, 7), (BF, 64, 12), (BF, 128, 28), (F32, 64, 2)])
def test_an_infinite_value_that_is_seen_stays_infinite(dtype, d, G):
    """Raw caches hold infinities: with a weight above zero they are the output, of either sign; their neighbours in
    other dimensions and the rows that do not see them stay finite."""
    n = 77
    g = torch.Generator().manual_seed(3)
    k, v = torch.randn(n, 1, d, generator=g) / 4, torch.randn(n, 1, d, generator=g)
    v[20, 0, 3], v[61, 0, d - 1] = math.inf, -math.inf
    cache, table = put(k, v, dtype, "raw", 2)
    q = (torch.randn(2, 1, G, d, generator=g) / 4).to(dtype).cuda()
    out, lse = skv.paged_attn(q, cache, table, i32([n, n]), first=i32([0, 62]))
    assert torch.all(out[0, ..., 3] == math.inf) and torch.all(out[0, ..., d - 1] == -math.inf)
    rest = out.clone()
    rest[0, ..., 3] = rest[0, ..., d - 1] = 0
    assert rest.isfinite().all() and lse.isfinite().all()


@pytest.mark.parametrize("d,G,Hkv,B", [(128, 1, 8, 512), (128, 12, 8, 256), (64, 28, 8, 256)])
def test_many_small_weights_beside_a_large_one(d, G, Hkv, B):
    """e4m3 pages, one key 2^26 above 4,095 equal others: each of these weighs less than half of fp16's smallest step
    beside a weight of 1, and together they are the whole output in the dimensions where the large one's value is zero.
    (More units than CTAs, so that one warp sees the large key and hundreds of others.) Bound: a weight is off by
    2^-11 of itself or by 2^-32 of the largest."""
    n = 4096
    k, v = torch.zeros(n, Hkv, d), torch.ones(n, Hkv, d)
    k[0] = 26 * math.log(2) / math.sqrt(d)                  # q of ones: logit 26 ln 2
    v[0] = 0
    v[:, :, 0] = 0
    v[0, :, 0] = 1
    cache, table = put(k, v, BF, "e4m3", B)
    q = torch.ones(B, 1, G * Hkv, d, dtype=BF, device="cuda")
    lens = [n - b % 7 for b in range(B)]
    out, lse = skv.paged_attn(q, cache, table, i32(lens))
    for b in (0, 1, B // 2, B - 1):
        r = reference(q, cache, table, lens, b)
        inner = r.mass * (2.0 ** -11 + 2.0 ** -16 + 2 * r.dlogit[..., None]) + 2.0 ** -7 * r.tiny
        bound = inner * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(r.out) + 1e-37
        err = np.abs(out[b].double().cpu().numpy() - r.out)
        assert np.all(err <= bound), f"sequence {b}: {np.max(err / bound):.2f} bounds"
    assert torch.equal(out, out[:, :, :1].expand_as(out))   # equal rows over equal keys


@pytest.mark.parametrize("dtype,fmt", [(BF, "e4m3"), (BF, "raw"), (F32, "e4m3"), (F32, "raw")])
@pytest.mark.parametrize("cap", [1e-40, 1e-3, 0.5, 6.0, 30.0, 1e3, 1e6, 1e8, 3e38])
@pytest.mark.parametrize("d,G", [(128, 3), (64, 13), (64, 25)])
def test_caps_of_every_size(dtype, fmt, cap, d, G):
    """c tanh(s / c) for any finite c > 0: tiny (the sign of s alone is left), in the range of the logits, and so large
    that nothing is capped. A capped logit is off by its own product's error and 2^-20 of itself, not of the cap."""
    n = 211
    g = torch.Generator().manual_seed(G)
    k, v = torch.randn(n, 1, d, generator=g) * 2, torch.randn(n, 1, d, generator=g)
    cache, table = put(k, v, dtype, fmt)
    q = torch.randn(1, 1, G, d, generator=g).to(dtype).cuda()
    out, lse = skv.paged_attn(q, cache, table, i32([n]), softcap=cap)
    (kk, vv), (_, vs) = ref.read_rows(cache, table[0].tolist(), 0, n)
    cap = float(np.float32(cap))
    x = q[0].double().cpu().numpy()
    r = ref.Attn(x, kk, vv, vs, n - 1, 0, softcap=cap)
    top = np.abs(x[0] @ kk[:, 0].T).max(-1) / math.sqrt(d)
    r.dlogit = ref.Attn(x, kk, vv, vs, n - 1, 0).dlogit + 2.0 ** -20 * np.minimum(cap, top)
    ref.check_attention(out[0], lse[0], r, dtype, fmt, f"cap {cap}")


@pytest.mark.parametrize("dtype,fmt", [(BF, "raw"), (BF, "e4m3"), (F32, "raw")])
@pytest.mark.parametrize("d,G", [(128, 7), (64, 12), (128, 28)])
def test_a_weight_of_zero_takes_nothing_of_a_huge_value(dtype, fmt, d, G):
    """Keys so far below the others that their weights are zero in 32 bits, with values of 2^120: the output is that of the
    others, whatever the weights are made of. (In 64 bits the huge ones add e^-400 2^120, nothing.)"""
    n = 90
    g = torch.Generator().manual_seed(G)
    k, v = torch.randn(n, 1, d, generator=g) / 64, torch.randn(n, 1, d, generator=g)
    k[1::2] -= 400 / math.sqrt(d)                            # q of ones: logits of about 0 and -400
    v[1::2] = 2.0 ** 120
    cache, table = put(k, v, dtype, fmt)
    q = torch.ones(1, 1, G, d).to(dtype).cuda()
    out, lse = skv.paged_attn(q, cache, table, i32([n]))
    r = reference(q, cache, table, [n], 0)
    r.tiny = r.tiny * 0                                     # that term takes a weight's scale from its value's
    ref.check_attention(out[0], lse[0], r, dtype, fmt)
