"""The binding's treatment of bounds that a C int cannot hold, and refusals before any C call."""
import pytest
import torch

import exact_attention_138_b200 as ea


@pytest.mark.parametrize("window,want", [
    ((5, 0), (5, 0)), ((-3, -1), (-1, -1)), ((2**31 - 1, 7), (2**31 - 1, 7)), ((2**31, 2**31), (-1, -1)),
    ((2**32 + 5, 0), (-1, 0)), ((5, 2**32 + 1), (5, -1)), ((-2**40, 3), (-1, 3))])
def test_windows_beyond_32_bits_are_open(window, want):
    assert ea._window(False, window) == want
    assert ea._window(True, window) == (want[0], 0)


def test_the_cache_passes_bounds_on_whole(monkeypatch):
    """kv4_attend and pages_free on host tensors, with the device checks and the C calls taken out."""
    from exact_attention_138_b200 import kvcache
    seen = {}
    monkeypatch.setattr(kvcache, "_tensors", lambda where, *ts: 0)
    monkeypatch.setattr(kvcache, "_raw_stream", lambda *a: None)
    monkeypatch.setattr(kvcache._lib, "attn_kv4_attend", lambda *a: seen.update(attend=a[17:20]) or 0)
    monkeypatch.setattr(kvcache._lib, "attn_pages_free", lambda *a: seen.update(free=a[9:11]) or 0)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)                         # noqa: E731
    q, pool = torch.zeros((1, 2, 1, 32), dtype=torch.bfloat16), torch.zeros((3, 2, 640), dtype=torch.uint8)
    for window, want in ((None, (-1, 0)), ((2**32 + 5, 0), (-1, 0)), ((9, 2**32), (9, -1)), ((7, 1), (7, 1))):
        ea.kv4_attend(q, pool, i(1, 3), i(1), window=window, sinks=2)
        assert seen["attend"] == (*want, 2)
    for window, left in ((None, -1), ((9, 0), 9), ((2**32 + 5, 0), None), ((-1, 0), None)):
        seen.pop("free", None)
        ea.pages_free(i(4, 3), i(4), i(9), 16, i(2), window=window, sinks=3)
        assert seen.get("free") == (None if left is None else (left, 3))     # an open window frees nothing


def test_refusals_are_value_errors():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)                         # noqa: E731
    q, pool = torch.zeros((1, 2, 1, 32), dtype=torch.bfloat16), torch.zeros((3, 2, 640), dtype=torch.uint8)
    for f in (lambda: ea.kv4_attend(q, pool[:, :0], i(1, 3), i(1)), lambda: ea.kv4_gather(pool, i(1, 3), i(), 4, 32),
              lambda: ea.pages_reserve(i(4, 3), i(4), i(9), 16, i(), i()),
              lambda: ea.pages_free(i(4, 3), i(4), i(9), 16, i())):
        with pytest.raises(ValueError):
            f()
