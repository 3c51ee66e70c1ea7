"""A paged K/V cache in 4 bits: quantising rows into it, reading them back, attending to it
(attn_kv4_* of include/attn.h, csrc/kv4.cu) and its pages (attn_pages_*, csrc/pages.cu). Like the rest of the package this module only marshals
arguments; device memory and streams come from PyTorch.

    pool = kv4_pool(pages, kv_heads, page_size, d)            # uint8 (pages, kv_heads, bytes)
    table: int32 (slots, max_pages), the page of every page_size tokens of a sequence, -1: none
    kv4_append(pool, table, start, k, v)                      # rows of k, v -> tokens start + row
    o, lse = kv4_attend(q, pool, table, lens, window=(1024, 0), sinks=4)

Pages: with lens (slots,) and refs (pages,), int32 like the table and all of it on the device,

    start = pages_reserve(table, lens, refs, page_size, seqs, counts)     # room for new tokens
    pages_copy(pool, *pages_fork(table, lens, refs, page_size, src, dst)) # sequences that share pages
    pages_free(table, lens, refs, page_size, seqs)                        # they end
    pages_free(table, lens, refs, page_size, seqs, window=(1024, 0), sinks=4)  # what no query sees
    pages_copy(pool, *pages_compact(table, refs))                         # pages in use come first

A reserve or fork that cannot be served changes nothing, and pages_free passes over rows out of range;
`device_status()` then says ATTN_ERR_PAGES.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import AttnError, _fill, _lib, _sinks, _torch_stream, _window

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_lib.attn_kv4_page_bytes.restype = _sz
_lib.attn_kv4_page_bytes.argtypes = [_i, _i, _i]
_lib.attn_kv4_append.restype = _i
_lib.attn_kv4_append.argtypes = [_vp] * 7 + [_i] * 8 + [_vp]
_lib.attn_kv4_gather.restype = _i
_lib.attn_kv4_gather.argtypes = [_vp] * 7 + [_i] * 8 + [_vp]
_lib.attn_kv4_workspace_bytes.restype = _sz
_lib.attn_kv4_workspace_bytes.argtypes = [_i] * 4
_lib.attn_kv4_attend.restype = _i
_lib.attn_kv4_attend.argtypes = [_vp] * 7 + [_i] * 9 + [_f, _i, _i, _i, _vp, _sz, _vp]
_lib.attn_pages_reserve.restype = _i
_lib.attn_pages_reserve.argtypes = [_vp] * 6 + [_i] * 5 + [_vp]
_lib.attn_pages_fork.restype = _i
_lib.attn_pages_fork.argtypes = [_vp] * 7 + [_i] * 5 + [_vp]
_lib.attn_pages_free.restype = _i
_lib.attn_pages_free.argtypes = [_vp] * 4 + [_i] * 7 + [_vp]
_lib.attn_pages_workspace_bytes.restype = _sz
_lib.attn_pages_workspace_bytes.argtypes = [_i]
_lib.attn_pages_compact.restype = _i
_lib.attn_pages_compact.argtypes = [_vp] * 5 + [_i] * 3 + [_vp, _sz, _vp]
_lib.attn_pages_copy.restype = _i
_lib.attn_pages_copy.argtypes = [_vp] * 4 + [_i, _i, ctypes.c_longlong, _i, _vp]


# ---------------------------------------------------------------- raw C entry points
def attn_kv4_page_bytes(page_size, Hkv, d) -> int:
    return _lib.attn_kv4_page_bytes(page_size, Hkv, d)


def attn_kv4_append(pool, table, seqs, start, counts, k, v, pages, slots, max_pages, page_size, B,
                    Hkv, n, d, stream) -> int:
    return _lib.attn_kv4_append(pool, table, seqs, start, counts, k, v, pages, slots, max_pages,
                                page_size, B, Hkv, n, d, stream)


def attn_kv4_gather(pool, table, seqs, start, counts, k, v, pages, slots, max_pages, page_size, B,
                    Hkv, n, d, stream) -> int:
    return _lib.attn_kv4_gather(pool, table, seqs, start, counts, k, v, pages, slots, max_pages,
                                page_size, B, Hkv, n, d, stream)


def attn_kv4_workspace_bytes(H, Hkv, nq, d) -> int:
    return _lib.attn_kv4_workspace_bytes(H, Hkv, nq, d)


def attn_kv4_attend(q, pool, table, seqs, lens, o, lse, pages, slots, max_pages, page_size, B, H, Hkv,
                    nq, d, scale, window_left, window_right, n_sink, workspace, ws_bytes, stream) -> int:
    return _lib.attn_kv4_attend(q, pool, table, seqs, lens, o, lse, pages, slots, max_pages,
                                page_size, B, H, Hkv, nq, d, scale, window_left, window_right, n_sink,
                                workspace, ws_bytes, stream)


def attn_pages_reserve(table, lens, refs, seqs, counts, start, pages, slots, max_pages, page_size, n,
                       stream) -> int:
    return _lib.attn_pages_reserve(table, lens, refs, seqs, counts, start, pages, slots, max_pages,
                                   page_size, n, stream)


def attn_pages_fork(table, lens, refs, src, dst, from_, to, pages, slots, max_pages, page_size, n,
                    stream) -> int:
    return _lib.attn_pages_fork(table, lens, refs, src, dst, from_, to, pages, slots, max_pages,
                                page_size, n, stream)


def attn_pages_free(table, lens, refs, seqs, pages, slots, max_pages, page_size, n, window_left, n_sink,
                    stream) -> int:
    return _lib.attn_pages_free(table, lens, refs, seqs, pages, slots, max_pages, page_size, n,
                                window_left, n_sink, stream)


def attn_pages_workspace_bytes(pages) -> int:
    return _lib.attn_pages_workspace_bytes(pages)


def attn_pages_compact(table, refs, from_, to, count, pages, slots, max_pages, workspace, ws_bytes,
                       stream) -> int:
    return _lib.attn_pages_compact(table, refs, from_, to, count, pages, slots, max_pages, workspace,
                                   ws_bytes, stream)


def attn_pages_copy(pool, from_, to, count, layers, pages, page_bytes, n, stream) -> int:
    return _lib.attn_pages_copy(pool, from_, to, count, layers, pages, page_bytes, n, stream)


# ---------------------------------------------------------------- torch-tensor wrappers
def _tensors(where, *ts):
    """Packed CUDA tensors on the current device: kernels are launched there, and a host or a strided
    tensor's pointer must never reach one."""
    dev = torch.cuda.current_device() if ts[0].is_cuda else -2
    for t in ts:
        if t is not None and not (t.get_device() == dev and t.is_contiguous()):     # -1: host memory
            raise ValueError(f"{where}: tensors must be contiguous and on the current CUDA device")
    return dev


def _is(where, name, t, dtype, *shape):
    """t must have this dtype and shape (None: any size of that dimension)."""
    have = t.shape
    if t.dtype is dtype and (have == shape or len(have) == len(shape) and all(
            s is None or s == x for s, x in zip(shape, have))):
        return
    raise ValueError(f"{where}: {name} must be {dtype} {shape}, got {t.dtype} {tuple(have)}")


def _raw_stream(stream, dev, *written):
    """The stream's handle; what the call writes is not reused before `stream` is done with it."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    for t in written:
        t.record_stream(_torch_stream(stream))
    return stream.cuda_stream


def _at(t):
    return None if t is None else t.data_ptr()


def _page_size(where, pool, d):
    """Tokens of a page of the pool (pages, kv_heads, bytes)."""
    if pool.dtype != torch.uint8 or pool.dim() != 3:
        raise ValueError(f"{where}: the pool must be uint8 (pages, kv_heads, bytes)")
    if d not in (32, 64, 128):
        raise AttnError(2, where)
    if pool.shape[2] < 1 or pool.shape[2] % (20 * d):
        raise ValueError(f"{where}: a page and head of {pool.shape[2]} bytes holds no blocks of {20 * d}")
    return pool.shape[2] // (20 * d) * 16


def _rows(where, pool, table, d, B, start, counts, seqs):
    page = _page_size(where, pool, d)
    if table.dtype is not torch.int32 or table.dim() != 2:
        _is(where, "table", table, torch.int32, None, None)
    _is(where, "start", start, torch.int32, B)
    if counts is not None:
        _is(where, "counts", counts, torch.int32, B)
    if seqs is not None:
        _is(where, "seqs", seqs, torch.int32, B)
    return page


def kv4_pool(pages, kv_heads, page_size, d, device=None):
    """An uninitialised pool: uint8 (pages, kv_heads, page_size / 16 * 20 d)."""
    each = attn_kv4_page_bytes(page_size, 1, d)
    if not each or pages < 1 or kv_heads < 1:
        raise ValueError("page_size must be a multiple of 16, d 32, 64 or 128, counts 1 or more")
    return torch.empty((pages, kv_heads, each), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def kv4_append(pool, table, start, k, v, counts=None, seqs=None, stream=None):
    """Quantises rows [0, counts[i]) (all, without counts) of k, v (B, kv_heads, n, d) bf16 into tokens
    start[i] + row of table row seqs[i] (i, without seqs). A negative start leaves its entry out, tokens
    on no page are dropped, and no other token's bits change."""
    where = "kv4_append"
    if k.dim() != 4:
        raise ValueError(f"{where}: k and v must be (B, kv_heads, n, d)")
    B, Hkv, n, d = k.shape
    page = _rows(where, pool, table, d, B, start, counts, seqs)
    _is(where, "k", k, torch.bfloat16, B, pool.shape[1], n, d)
    _is(where, "v", v, torch.bfloat16, B, Hkv, n, d)
    dev = _tensors(where, pool, table, start, k, v, counts, seqs)
    rc = _lib.attn_kv4_append(pool.data_ptr(), table.data_ptr(), _at(seqs), start.data_ptr(),
                              _at(counts), k.data_ptr(), v.data_ptr(), pool.shape[0], table.shape[0],
                              table.shape[1], page, B, Hkv, n, d, _raw_stream(stream, dev))
    if rc:
        raise AttnError(rc, "attn_kv4_append")


def kv4_gather(pool, table, start, n, d, counts=None, seqs=None, k=None, v=None, stream=None):
    """The values that tokens start[i] .. start[i] + n - 1 of table row seqs[i] stand for, rounded to
    bf16: k, v (B, kv_heads, n, d). Rows at or beyond counts[i], of entries with a negative start and
    on no page are zeros."""
    where = "kv4_gather"
    if start.dim() != 1:
        _is(where, "start", start, torch.int32, None)
    B = start.shape[0]
    page = _rows(where, pool, table, d, B, start, counts, seqs)
    if n < 1:
        raise ValueError(f"{where}: n must be 1 or more")
    dev = _tensors(where, pool, table, start, counts, seqs, k, v)
    shape = (B, pool.shape[1], n, d)
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _is(where, name, t, torch.bfloat16, *shape)
    make = lambda: pool.new_empty(shape, dtype=torch.bfloat16)          # noqa: E731
    k, v = _fill(stream, (k, make), (v, make))
    rc = _lib.attn_kv4_gather(pool.data_ptr(), table.data_ptr(), _at(seqs), start.data_ptr(),
                              _at(counts), k.data_ptr(), v.data_ptr(), pool.shape[0],
                              table.shape[0], table.shape[1], page, B, shape[1], n, d,
                              _raw_stream(stream, dev, k, v))
    if rc:
        raise AttnError(rc, "attn_kv4_gather")
    return k, v


def kv4_attend(q, pool, table, lens, window=None, sinks=0, scale=None, seqs=None, out=None, lse=None,
               workspace=None, stream=None):
    """O, LSE of q (B, H, nq, d) bf16 over the lens[row] tokens of table row seqs[i] (i, without
    seqs), for the newest tokens of a sequence: query t sits at key position lens - nq + t. window =
    (left, right) as in `forward`; None is causal, (-1, 0). The first `sinks` tokens stay visible
    beyond the left bound. Tokens on no page are not seen; a row that sees none gets O = 0, LSE =
    -inf."""
    where = "kv4_attend"
    if q.dim() != 4:
        raise ValueError(f"{where}: q must be (B, H, nq, d)")
    B, H, nq, d = q.shape
    page = _page_size(where, pool, d)
    pages, Hkv, _ = pool.shape
    if Hkv < 1 or H % Hkv:
        raise ValueError(f"{where}: H must be a multiple of the pool's K/V heads")
    if q.dtype is not torch.bfloat16 or table.dtype is not torch.int32 or table.dim() != 2:
        _is(where, "q", q, torch.bfloat16, B, H, nq, d)
        _is(where, "table", table, torch.int32, None, None)
    slots, width = table.shape
    _is(where, "lens", lens, torch.int32, slots)
    if seqs is not None:
        _is(where, "seqs", seqs, torch.int32, B)
    wl, wr = _window(window is None, window)
    sinks = _sinks(sinks)
    dev = _tensors(where, q, pool, table, lens, seqs, out, lse, workspace)
    if out is not None:
        _is(where, "out", out, torch.bfloat16, B, H, nq, d)
    if lse is not None:
        _is(where, "lse", lse, torch.float32, B, H, nq)
    out, lse, workspace = _fill(
        stream, (out, lambda: torch.empty_like(q)), (lse, lambda: q.new_empty((B, H, nq), dtype=torch.float32)),
        (workspace, lambda: pool.new_empty(_lib.attn_kv4_workspace_bytes(H, Hkv, nq, d))))
    rc = _lib.attn_kv4_attend(q.data_ptr(), pool.data_ptr(), table.data_ptr(), _at(seqs),
                              lens.data_ptr(), out.data_ptr(), lse.data_ptr(), pages, slots, width,
                              page, B, H, Hkv, nq, d, 1.0 / math.sqrt(d) if scale is None else float(scale),
                              wl, wr, sinks, workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(),
                              _raw_stream(stream, dev, out, lse, workspace))
    if rc:
        raise AttnError(rc, "attn_kv4_attend")
    return out, lse


def _page_state(where, table, lens, refs, *ts):
    """Checks the state and the int32 vectors of one call; (pages, slots, max_pages, device)."""
    if table.dtype is not torch.int32 or table.dim() != 2:
        _is(where, "table", table, torch.int32, None, None)
    slots, width = table.shape
    if lens is not None:
        _is(where, "lens", lens, torch.int32, slots)
    if refs.dtype is not torch.int32 or refs.dim() != 1:
        _is(where, "refs", refs, torch.int32, None)
    for t in ts:
        _is(where, "rows and counts", t, torch.int32, ts[0].shape[0] if ts[0].dim() else None)
    return refs.shape[0], slots, width, _tensors(where, table, lens, refs, *ts)


def pages_reserve(table, lens, refs, page_size, seqs, counts, stream=None):
    """Sequences seqs[i] grow by counts[i] tokens: pages are taken for them and lens follows. Returns
    start (n,), the first new token of each (its length before), or -1 throughout if the call was
    refused: pages or table columns ran out, or a row is out of range or given twice."""
    where = "pages_reserve"
    pages, slots, width, dev = _page_state(where, table, lens, refs, seqs, counts)
    start, = _fill(stream, (None, lambda: torch.empty_like(seqs)))
    rc = _lib.attn_pages_reserve(table.data_ptr(), lens.data_ptr(), refs.data_ptr(), seqs.data_ptr(),
                                 counts.data_ptr(), start.data_ptr(), pages, slots, width, page_size,
                                 seqs.shape[0], _raw_stream(stream, dev, start))
    if rc:
        raise AttnError(rc, "attn_pages_reserve")
    return start


def pages_fork(table, lens, refs, page_size, src, dst, stream=None):
    """The empty sequences dst[i] become src[i] and share its full pages; a partly filled last page gets
    a page of its own. Returns (from, to) (n,) int32 for `pages_copy`, -1 where there is nothing to copy
    or the call was refused (pages ran out, a dst not empty, given twice or also a src)."""
    where = "pages_fork"
    pages, slots, width, dev = _page_state(where, table, lens, refs, src, dst)
    frm, to = _fill(stream, *[(None, lambda: torch.empty_like(src))] * 2)
    rc = _lib.attn_pages_fork(table.data_ptr(), lens.data_ptr(), refs.data_ptr(), src.data_ptr(),
                              dst.data_ptr(), frm.data_ptr(), to.data_ptr(), pages, slots, width, page_size,
                              src.shape[0], _raw_stream(stream, dev, frm, to))
    if rc:
        raise AttnError(rc, "attn_pages_fork")
    return frm, to


def pages_free(table, lens, refs, page_size, seqs, window=None, sinks=0, stream=None):
    """Without a window the sequences end: their pages lose a reference, their rows and lengths are
    cleared. With window=(left, right) only pages are given back whose tokens no query from the next
    token on sees under that window and these sinks; their entries become -1. Rows out of range are passed
    over (and reported by `device_status()`), the others served."""
    where = "pages_free"
    pages, slots, width, dev = _page_state(where, table, lens, refs, seqs)
    sinks = _sinks(sinks)
    left = _window(False, window)[0]
    if window is not None and left < 0:
        return                                  # an open window: every token stays visible
    rc = _lib.attn_pages_free(table.data_ptr(), lens.data_ptr(), refs.data_ptr(), seqs.data_ptr(), pages,
                              slots, width, page_size, seqs.shape[0], left, sinks,
                              _raw_stream(stream, dev))
    if rc:
        raise AttnError(rc, "attn_pages_free")


def pages_compact(table, refs, workspace=None, stream=None):
    """Renumbers the pages in use to 0 .. L-1. Returns (from, to, count) for `pages_copy`: page from[r]
    becomes to[r] for r < count[0], -1 behind."""
    where = "pages_compact"
    pages, slots, width, dev = _page_state(where, table, None, refs)
    if workspace is not None:
        _tensors(where, workspace)
    need = (pages + 4) * 4
    half = max(pages // 2, 1)
    out, workspace = _fill(
        stream, (None, lambda: torch.empty(2 * half + 1, dtype=torch.int32, device=refs.device)),
        (workspace, lambda: torch.empty(need, dtype=torch.uint8, device=refs.device)))
    frm, to, count = out[:half], out[half:2 * half], out[2 * half:]
    rc = _lib.attn_pages_compact(table.data_ptr(), refs.data_ptr(), frm.data_ptr(), to.data_ptr(),
                                 count.data_ptr(), pages, slots, width, workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(),
                                 _raw_stream(stream, dev, out, workspace))
    if rc:
        raise AttnError(rc, "attn_pages_compact")
    return frm, to, count


def pages_copy(pool, frm, to, count=None, layered=False, stream=None):
    """Copies the contents of page frm[i] to page to[i] for i < count[0] (all, without count); pairs with
    a number outside the pool are skipped. pool: (pages, ...) of any type, or (layers, pages, ...) with
    layered=True (the same pages of every layer). No page may be both copied from and to."""
    where = "pages_copy"
    if pool.dim() < (2 if layered else 1):
        raise ValueError(f"{where}: the pool needs a dimension of pages")
    if frm.dtype is not torch.int32 or frm.dim() != 1:
        _is(where, "frm", frm, torch.int32, None)
    _is(where, "to", to, torch.int32, frm.shape[0])
    if count is not None:
        _is(where, "count", count, torch.int32, 1)
    dev = _tensors(where, pool, frm, to, count)
    layers, pages = (pool.shape[0], pool.shape[1]) if layered else (1, pool.shape[0])
    if layers < 1 or pages < 1:
        raise ValueError(f"{where}: the pool is empty")
    each = pool.numel() // (layers * pages) * pool.element_size()
    rc = _lib.attn_pages_copy(pool.data_ptr(), frm.data_ptr(), to.data_ptr(), _at(count), layers, pages, each,
                              frm.shape[0], _raw_stream(stream, dev))
    if rc:
        raise AttnError(rc, "attn_pages_copy")
