"""Limits of the page calls and of the cache's pages, checked before anything is launched."""
import ctypes

import pytest
import torch

import stream_ref as ref
from test_gpu_kv4_paths import _i32, _randn, attend, cache, check

import exact_attention_138_b200 as ea

F = ctypes.c_void_p(1 << 20)        # an aligned address that is never read: the call is refused first


@pytest.mark.parametrize("pages", [2**31 - 8192, 2**31 - 4000, 2**31 - 258, 2**31 - 1])
def test_pages_whose_scan_would_pass_32_bits(pages):
    # the scans go on by tiles of 4096 pages in 32 bits, past the last page by up to one tile
    assert ea.attn_pages_reserve(F, F, F, F, F, F, pages, 4, 3, 16, 2, None) == ea.ATTN_ERR_INVALID
    assert ea.attn_pages_fork(F, F, F, F, F, F, F, pages, 4, 3, 16, 2, None) == ea.ATTN_ERR_INVALID
    assert ea.attn_pages_free(F, F, F, F, pages, 4, 3, 16, 2, -1, 0, None) == ea.ATTN_ERR_INVALID
    assert ea.attn_pages_compact(F, F, F, F, F, pages, 4, 3, F, 1 << 40, None) == ea.ATTN_ERR_INVALID


@pytest.mark.gpu
def test_pages_of_more_than_65536_tokens(cuda_device):
    # any multiple of 16 is a page size: appending, reading back and attending across such a page's end
    page, lens = 65552 * 2, [65552 * 2 + 100, 7]
    pool, table = cache(lens, page, 1, 32, 3)
    assert pool.shape[2] == ea.attn_kv4_page_bytes(page, 1, 32)
    q = _randn((2, 2, 1, 32), 5)
    for window, sinks in ((None, 0), ((300, 0), 20)):
        got = ea.kv4_attend(q.cuda(), pool, _i32(table), _i32(lens), window=window, sinks=sinks)
        wl, wr = window or (-1, 0)
        check(got, attend(ref.f64(q), pool.cpu().numpy(), table, lens, [0, 1], wl, wr, sinks))
    k, _ = ea.kv4_gather(pool, _i32(table), _i32([page - 3, 2]), 9, 32)
    x = _randn((2, 1, max(lens), 32), 4)
    x[..., :2] *= 6
    for i, at in enumerate((page - 3, 2)):
        n = min(9, lens[i] - at)
        q4, s, lo = ref.quantise(ref.f64(x[i, :, at:at + n]))
        assert torch.equal(k[i, :, :n].cpu(), torch.from_numpy(ref.value(q4, s, lo)).float().bfloat16())
