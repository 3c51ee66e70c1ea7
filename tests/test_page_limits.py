"""Limits of the page calls and of the cache's pages, checked before anything is launched."""
import ctypes

import pytest

import exact_attention_138_b200 as ea

F = ctypes.c_void_p(1 << 20)        # an aligned address that is never read: the call is refused first


@pytest.mark.parametrize("pages", [2**31 - 8192, 2**31 - 4000, 2**31 - 258, 2**31 - 1])
def test_pages_whose_scan_would_pass_32_bits(pages):
    # the scans go on by tiles of 4096 pages in 32 bits, past the last page by up to one tile
    assert ea.attn_pages_reserve(F, F, F, F, F, F, pages, 4, 3, 16, 2, None) == ea.ATTN_ERR_INVALID
    assert ea.attn_pages_fork(F, F, F, F, F, F, F, pages, 4, 3, 16, 2, None) == ea.ATTN_ERR_INVALID
    assert ea.attn_pages_free(F, F, F, F, pages, 4, 3, 16, 2, -1, 0, None) == ea.ATTN_ERR_INVALID
    assert ea.attn_pages_compact(F, F, F, F, F, pages, 4, 3, F, 1 << 40, None) == ea.ATTN_ERR_INVALID
