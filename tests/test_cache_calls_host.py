"""The exact-token cache's arguments on the host (not gpu): where the calls' pointers come from, and calls that are
refused before a launch."""
import ctypes

import pytest
import torch

import compressed_decode_attention_equal_b200 as skv
from compressed_decode_attention_equal_b200 import _lib
from test_cache_host import BF, INV, P, _append, _attn, lib  # noqa: F401


def test_the_pages_are_where_they_are_now():
    """The address is asked for at each call: storage given anew in place is followed, never the one that was freed;
    another tensor cannot take the pages' place, since the views would stay with the old one."""
    c = skv.TokenCache(3, 2, 64, BF, device="cpu", format="e4m3")
    assert c.struct()._obj.pages == c.pages.data_ptr() and c.struct()._obj.num_pages == 3
    c.pages.data = torch.ones_like(c.pages)
    assert c.struct()._obj.pages == c.pages.data_ptr()
    with pytest.raises(AttributeError):
        c.pages = torch.zeros_like(c.pages)
    c.pages.data = torch.zeros(1, c.page_bytes, dtype=torch.uint8)
    with pytest.raises(ValueError, match="another size"):
        c.struct()


@pytest.mark.parametrize("kw", [
    dict(cu=P(768)), dict(cu=P(760)), dict(cu=P(772)),          # the new lengths in the offsets
    dict(new=P(256)), dict(new=P(256 + 28)), dict(new=P(252)),  # in the page table, 2 x 4 ids at 256
])
def test_new_lengths_may_not_lie_in_what_is_read(lib, kw):
    assert _append(lib, **kw) == INV


@pytest.mark.parametrize("v", [4096, 4096 + 2032, 4096 - 2032])
def test_keys_and_values_are_not_read_into_one_place(lib, v):
    ints, pool = ctypes.c_int32 * 2, _lib.SkvTokenCache(4096, 9)   # 2 x 4 rows of 256 bytes

    def read(v, T=1):
        return lib.skv_cache_read(ctypes.byref(pool), 1, 1, 2, 4, 128, ints(0, 0), ints(T, T), P(256), 4, P(4096), P(v), None,
                                  256, None)
    assert read(v) == INV
    assert read(4096 + 2048) == read(4096 - 2048) == _lib.SKV_ERR_WORKSPACE   # side by side: on to the next check


@pytest.mark.parametrize("kw,opts", [
    (dict(lse=P(65536)), None), (dict(lse=P(65536 + 4092)), None), (dict(lse=P(65536 - 60)), None),
    ({}, dict(prior_out=1 << 20, prior_lse=65536 + 4092)), ({}, dict(prior_out=65536, prior_lse=65536))])
def test_outputs_and_partitions_stay_apart(lib, kw, opts):
    assert _attn(lib, opts=_lib.SkvPagedAttnOptions(**opts) if opts else None, **kw) == INV
    assert _attn(lib, lse=P(65536 + 4096), ws=None) == _lib.SKV_ERR_WORKSPACE
