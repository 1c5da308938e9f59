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
