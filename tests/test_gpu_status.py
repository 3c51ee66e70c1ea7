"""The device status: a refused page call, which a full cache meets in ordinary use, neither hides a fault
that a kernel reports after it nor is lost behind one that was reported before it. Freeing rows out of range,
which is reported in the same way, serves the others."""
import pytest
import torch

import exact_attention_138_b200 as ea


def _refused():
    """A page call that finds no free page."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")     # noqa: E731
    start = ea.pages_reserve(i32([[-1, -1]]), i32([0]), i32([1, 1]), 16, i32([0]), i32([5]))
    assert start.tolist() == [-1]


def _expired():
    """The self-test of the bounded wait: a wait of 200 us that nothing ends."""
    assert ea.attn_selftest_wait_timeout(200, torch.cuda.current_stream().cuda_stream) == ea.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["refused first", "expired first", "refused twice"])
def test_a_refusal_and_a_fault_are_both_reported(cuda_device, order):
    ea.device_status()
    if order == "expired first":
        _expired()
    _refused()
    if order == "refused twice":
        _refused()
    if order != "expired first":
        _expired()
    assert [ea.device_status() for _ in range(3)] == [ea.ATTN_ERR_TIMEOUT, ea.ATTN_ERR_PAGES, ea.ATTN_OK]


@pytest.mark.gpu
@pytest.mark.parametrize("what,code", [(_refused, ea.ATTN_ERR_PAGES), (_expired, ea.ATTN_ERR_TIMEOUT)])
def test_each_alone_is_reported_once(cuda_device, what, code):
    ea.device_status()
    what()
    assert [ea.device_status() for _ in range(2)] == [code, ea.ATTN_OK]


@pytest.mark.gpu
@pytest.mark.parametrize("window", [None, (0, 0)])
def test_freeing_passes_over_rows_out_of_range_and_reports_them(cuda_device, window):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")     # noqa: E731
    table, lens, refs = i32([[0, 1], [2, -1], [3, -1]]), i32([32, 16, 16]), i32([1, 1, 1, 1, 0])
    ea.device_status()
    ea.pages_free(table, lens, refs, 16, i32([0, 3, 1, -1]), window=window)
    assert ea.device_status() == ea.ATTN_ERR_PAGES and ea.device_status() == ea.ATTN_OK
    assert table.tolist() == [[-1, -1], [-1, -1], [3, -1]] and refs.tolist() == [0, 0, 0, 1, 0]
    assert lens.tolist() == ([0, 0, 16] if window is None else [32, 16, 16])
