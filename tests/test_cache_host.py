"""The exact-token cache's host side (not gpu): page arithmetic and views, the reference's own
quantisation against torch's e4m3 conversion, and every refusal of the binding and of the C ABI before a
launch."""
import ctypes

import numpy as np
import pytest
import torch

import cache_reference as ref
import compressed_decode_attention_equal_b200 as skv
from compressed_decode_attention_equal_b200 import _lib

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    from compressed_decode_attention_equal_b200 import build
    build.build()
    return _lib.load()


@pytest.mark.parametrize("dtype,fmt,d,group", [(BF, "raw", 128, 8192), (BF, "raw", 64, 4096), (F32, "raw", 128, 16384),
                                               (BF, "e4m3", 128, 4128), (F32, "e4m3", 64, 2080)])
def test_page_bytes_and_views(lib, dtype, fmt, d, group):
    c = skv.TokenCache(3, 5, d, dtype, device="cpu", format=fmt)
    assert c.page_bytes == 5 * 4 * group == skv.cache_page_bytes(dtype, 5, d, fmt)
    assert c.k.shape == c.v.shape == (3, 5, 4, 16, d)
    assert c.k.dtype == (torch.float8_e4m3fn if fmt == "e4m3" else dtype)
    c.pages.zero_()
    c.v[2, 3, 1, 7, 0] = 1.0
    at = int(c.pages[2].nonzero()[0])
    row = d * c.k.element_size()
    assert (3 * 4 + 1) * group + 16 * row + 7 * row <= at < (3 * 4 + 1) * group + 16 * row + 8 * row
    if fmt == "e4m3":
        c.pages.zero_()
        c.v_exp[1, 4, 3, 15] = 9
        assert int(c.pages[1].nonzero()[0]) == c.page_bytes - 1
    assert [skv.token_pages_for(t) for t in (0, 1, 64, 65)] == [0, 1, 1, 2]
    assert lib.skv_cache_page_bytes(1, 1, 0, 128) == lib.skv_cache_page_bytes(1, 2, 1, 128) == 0
    assert lib.skv_cache_page_bytes(1, 1, 1, 96) == lib.skv_cache_page_bytes(2, 0, 1, 64) == 0


def test_the_reference_quantises_as_torch_does_and_scales_by_the_smallest_power():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(400, 64, generator=g) * torch.exp(torch.randn(400, 1, generator=g) * 8)).bfloat16().double().numpy()
    q, e = ref.quantise(x)
    a = np.abs(x).max(-1)
    assert np.all(a <= 448 * np.ldexp(1.0, e)) and np.all(a > 448 * np.ldexp(1.0, e - 1))
    y = torch.from_numpy(x * np.ldexp(1.0, -e)[:, None]).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(q, y)
    normal = np.abs(x * np.ldexp(1.0, -e)[:, None]) >= 2.0 ** -6
    assert np.all(np.abs(q * np.ldexp(1.0, e)[:, None] - x)[normal] <= 2.0 ** -4 * np.abs(x)[normal])


def test_construction_is_checked():
    with pytest.raises(ValueError, match="format"):
        skv.TokenCache(1, 1, 128, BF, device="cpu", format="int8")
    with pytest.raises(TypeError):
        skv.TokenCache(1, 1, 128, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="d must"):
        skv.TokenCache(1, 1, 96, BF, device="cpu")
    with pytest.raises(ValueError, match="pages"):
        skv.TokenCache(1, 1, 128, BF, device="cpu", pages=torch.zeros(1, 5, dtype=torch.uint8))


@pytest.mark.parametrize("call", ["append", "read", "attn"])
def test_host_tensors_are_refused(call):
    c = skv.TokenCache(2, 2, 128, BF, device="cpu")
    t = torch.zeros(1, 2, dtype=torch.int32)
    lens = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 128, dtype=BF)
    with pytest.raises(ValueError, match="CUDA tensor"):
        if call == "append":
            skv.cache_append(x, x, c, t, lens)
        elif call == "read":
            skv.cache_read(c, t, [0], [1])
        else:
            skv.paged_attn(torch.zeros(1, 1, 4, 128, dtype=BF), c, t, lens)


P = ctypes.c_void_p


def _append(lib, **kw):
    a = dict(k=P(4096), v=P(8192), dtype=1, kt=512, kh=128, vt=512, vh=128, B=2, Hkv=4, d=128, n=2, cu=None, fmt=1,
             pool=_lib.SkvTokenCache(4096, 9), table=P(256), mp=4, lens=P(512), new=P(768), ws=P(1024), wsn=256)
    a.update(kw)
    return lib.skv_cache_append(a["k"], a["v"], a["dtype"], a["kt"], a["kh"], a["vt"], a["vh"], a["B"], a["Hkv"], a["d"],
                                a["n"], a["cu"], a["fmt"], ctypes.byref(a["pool"]) if a["pool"] else None, a["table"],
                                a["mp"], a["lens"], a["new"], a["ws"], a["wsn"], None)


INV, UNS, WSP = _lib.SKV_ERR_INVALID_ARG, _lib.SKV_ERR_UNSUPPORTED, _lib.SKV_ERR_WORKSPACE


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), INV), (dict(B=513), INV), (dict(Hkv=0), INV), (dict(mp=0), INV), (dict(fmt=2), INV), (dict(n=-2), INV),
    (dict(n=3), INV), (dict(k=None), INV), (dict(v=P(8200)), INV), (dict(table=None), INV), (dict(lens=None), INV),
    (dict(new=None), INV), (dict(new=P(516)), INV), (dict(pool=None), INV), (dict(pool=_lib.SkvTokenCache(8, 9)), INV),
    (dict(pool=_lib.SkvTokenCache(None, 9)), INV), (dict(pool=_lib.SkvTokenCache(4096, -1)), INV), (dict(kt=-512), INV),
    (dict(vh=130), INV), (dict(d=96), UNS), (dict(dtype=2), UNS), (dict(mp=1 << 25), UNS), (dict(Hkv=65536), UNS),
    (dict(n=1 << 30, Hkv=2), UNS), (dict(ws=None), WSP), (dict(ws=P(1040)), WSP), (dict(wsn=255), WSP)])
def test_append_refuses(lib, kw, want):
    assert _append(lib, **kw) == want


@pytest.mark.parametrize("first,T,mp,kw,want", [
    ([0, -1], [1, 1], 4, {}, INV), ([0, 0], [1, -1], 4, {}, INV), ([0, 200], [1, 57], 4, {}, INV),
    ([0, 0], [1, 1], 4, dict(k=None), INV), ([0, 0], [1, 1], 4, dict(v=P(8)), INV), ([0, 0], [1, 1], 4, dict(ws=None), WSP),
    ([0, 0], [1, 1], 4, dict(d=32), UNS), ([0, 0], [1 << 30, 1 << 30], 1 << 24, dict(Hkv=64), UNS),
    ([0, 0], [1, 1], 4, dict(table=None), INV), ([0, 0], [1, 1], 4, dict(fmt=-1), INV)])
def test_read_refuses(lib, first, T, mp, kw, want):
    a = dict(k=P(4096), v=P(8192), d=128, Hkv=4, fmt=1, table=P(256), ws=P(1024))
    a.update(kw)
    ints = ctypes.c_int32 * 2
    pool = _lib.SkvTokenCache(4096, 9)
    assert lib.skv_cache_read(ctypes.byref(pool), 1, a["fmt"], 2, a["Hkv"], a["d"], ints(*first), ints(*T), a["table"], mp,
                              a["k"], a["v"], a["ws"], 256, None) == want


def _attn(lib, opts=None, **kw):
    a = dict(q=P(4096), dtype=1, qs=(512, 512, 128), B=2, R=1, Hq=8, Hkv=4, d=128, fmt=1, pool=_lib.SkvTokenCache(4096, 9),
             table=P(256), mp=4, lens=P(512), out=P(65536), lse=P(131072), ws=P(1024), wsn=1 << 30)
    a.update(kw)
    return lib.skv_paged_attn(a["q"], a["dtype"], *a["qs"], a["B"], a["R"], a["Hq"], a["Hkv"], a["d"], a["fmt"],
                              ctypes.byref(a["pool"]), a["table"], a["mp"], a["lens"], a["out"], a["lse"], a["ws"], a["wsn"],
                              ctypes.byref(opts) if opts else None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), INV), (dict(R=0), INV), (dict(Hq=0), INV), (dict(Hq=6), UNS), (dict(d=80), UNS), (dict(dtype=7), UNS),
    (dict(fmt=3), INV), (dict(q=None), INV), (dict(q=P(4104)), INV), (dict(qs=(512, 512, 4)), INV),
    (dict(qs=(512, -512, 128)), INV), (dict(out=None), INV), (dict(out=P(65544)), INV), (dict(lse=None), INV),
    (dict(table=None), INV), (dict(lens=None), INV), (dict(pool=_lib.SkvTokenCache(None, 1)), INV), (dict(mp=1 << 25), UNS),
    (dict(R=1 << 20), UNS), (dict(B=512, Hkv=512, Hq=512), UNS), (dict(Hkv=4096, Hq=4096, B=1, mp=1 << 24), UNS),
    (dict(ws=None), WSP), (dict(ws=P(1000)), WSP), (dict(wsn=4096), WSP)])
def test_attention_refuses(lib, kw, want):
    assert _attn(lib, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(scale=float("nan")), dict(softcap=-1.0), dict(softcap=float("inf")), dict(window=-1), dict(first=2), dict(slopes=6),
    dict(prior_out=1 << 20), dict(prior_lse=1 << 20), dict(prior_out=(1 << 20) + 8, prior_lse=1 << 21),
    dict(prior_out=65536 + 256, prior_lse=1 << 21),     # overlaps out without being it
    dict(prior_out=65536, prior_lse=131072),            # the partitions may not be replaced in place
    dict(prior_out=65536, prior_lse=131072 + 16 * 4 - 4)])
def test_attention_options_refused(lib, kw):
    assert _attn(lib, opts=_lib.SkvPagedAttnOptions(**kw)) == INV
    bad = _lib.SkvPagedAttnOptions()
    bad.reserved[2] = 1
    assert _attn(lib, opts=bad) == INV


def test_workspace_query(lib):
    q = skv.paged_attn_workspace_bytes
    assert q(32, 1, 28, 4, 128, 512) > 256 and q(1, 1, 1, 1, 64, 1) > 256
    assert q(32, 1, 28, 5, 128, 512) == q(0, 1, 1, 1, 128, 1) == q(1, 1, 1, 1, 96, 1) == q(513, 1, 1, 1, 128, 1) == 0
