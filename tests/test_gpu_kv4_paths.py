"""Attention over the 4-bit cache where its work is cut up in other ways than small batches reach: more
entries than a block has threads, enough tiles that beginning a segment counts as places of its own, blocks
of 16 rows under windows with sinks, and a line of more than 2^22 places. Also the compaction of pages
whose table takes a launch of its own. References in fp64."""
import numpy as np
import pytest
import torch

import stream_ref as ref
from test_gpu_pages import Device, Model

import exact_attention_138_b200 as ea


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def _randn(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).bfloat16()


def unpack(pool, d):
    """K, V (pages, Hkv, page_size, d) fp64 that a pool stands for, and s of V's groups (..., d / 32)."""
    pages, Hkv, each = pool.shape
    blk = pool.reshape(pages, Hkv, each // (20 * d), 20 * d)
    out = []
    for data, par, isk in ((0, 16 * d, True), (8 * d, 18 * d, False)):
        n4 = np.stack([ref.nibble_at(t, d, isk) for t in range(16)])                   # (16, d)
        q = blk[..., data + n4 // 2] >> (4 * (n4 % 2)).astype(np.uint8) & 15
        w = np.ascontiguousarray(blk[..., par:par + 2 * d]).view(np.uint16).astype(np.uint32)
        ch = np.arange(d) // 32
        with np.errstate(invalid="ignore"):
            f = (w << 16).view(np.float32).astype(np.float64).reshape(*blk.shape[:3], 16, d // 32, 2)
            x = f[..., ch, 1] + f[..., ch, 0] * q
        out.append((x.reshape(pages, Hkv, -1, d), f[..., 0].reshape(pages, Hkv, -1, d // 32)))
    return out[0][0], out[1][0], out[1][1]


def attend(q, pool, table, lens, seqs, wl, wr, ns):
    """(O, LSE, bounds of both) in fp64. The kernel rounds P s to fp16: by 2^-11 of itself, or by 2^-25 /
    f, f a power of two that brings the row's largest P s above 2^2, so by 2^-27 of that; each
    such error counts up to 15 times. Then P as lo's weight and all sums are fp32, scores too, and O is
    rounded to bf16."""
    B, H, nq, d = q.shape
    K, V, S = unpack(pool, d)
    page = K.shape[2]
    o, lse = np.zeros(q.shape), np.full((B, H, nq), -np.inf)
    eo, el = np.zeros(q.shape), np.zeros((B, H, nq))
    for b in range(B):
        r = int(seqs[b])
        n = int(lens[r]) if 0 <= r < len(lens) else 0
        j = np.arange(n)
        pg = table[r][j // page] if n else np.zeros(0, int)
        vis = ref.visible(nq, n, wl, wr, ns) & ((pg >= 0) & (pg < K.shape[0]))[None]
        some = vis.any(0) if n else np.zeros(0, bool)
        if not some.any():
            continue
        j, pg, vis = j[some], pg[some], vis[:, some]
        k, v, s = (np.moveaxis(x[pg, :, j % page], 0, 1)[None] for x in (K, V, S))
        scale = ref.default_scale(d)
        p, l = ref.probabilities(q[b:b + 1], k, vis, scale)
        ve, ke, se = (ref._expand(x, H) for x in (v, k, s))
        o[b], lse[b] = (p @ ve)[0], l[0]
        size = scale * np.einsum("bhid,bhjd->bhij", np.abs(q[b:b + 1]), np.abs(ke)).max(-1)[0]
        el[b] = 2.0 ** -20 * size + 4e-6
        spread = np.abs(ve) + np.abs(ve).max(-1, keepdims=True)            # s q <= |value| + |lo|
        ps = (p * se.max(-1)[:, :, None, :]).max(-1)[0]                    # the row's largest P s
        eo[b] = (ref.BF16 * np.abs(o[b]) + (p @ spread)[0] * (2.0 ** -11 + 2 * el[b][..., None]) +
                 15 * 2.0 ** -27 * vis.sum(1)[None, :, None] * ps[..., None]) * 1.02 + 1e-38
    return o, lse, eo, el


def check(got, want):
    (o, lse), (ro, rl, eo, el) = got, want
    none = np.isneginf(rl)
    gl = ref.f64(lse)
    assert np.array_equal(np.isneginf(gl), none)
    off = np.abs(np.where(none, 0, gl) - np.where(none, 0, rl)) - el
    assert off.max() <= 0, ("lse", float(off.max()), np.unravel_index(off.argmax(), off.shape))
    off = np.abs(ref.f64(o) - ro) - eo
    assert off.max() <= 0, ("o", float(off.max()), np.unravel_index(off.argmax(), off.shape))
    assert not np.any(ref.f64(o)[none])


def cache(lens, page, Hkv, d, seed):
    """A pool filled by kv4_append and its table: pages in a random order, NaN behind the last tokens."""
    held = [-(-n // page) for n in lens]
    order = np.random.default_rng(seed).permutation(sum(held) + 2)
    table = np.full((len(lens), max(held) + 1), -1, np.int32)
    at = np.cumsum([0] + held)
    for i, n in enumerate(held):
        table[i, :n] = order[at[i]:at[i] + n]
    pool = torch.full((sum(held) + 2, Hkv, page // 16 * 20 * d), 255, dtype=torch.uint8).cuda()
    n = max(max(lens), 1)
    k, v = _randn((len(lens), Hkv, n, d), seed + 1), _randn((len(lens), Hkv, n, d), seed + 2)
    k[..., :2] *= 6
    ea.kv4_append(pool, _i32(table), _i32([0] * len(lens)), k.cuda(), v.cuda(), counts=_i32(lens))
    return pool, table


def _ragged(n, most, seed, empty=0.15):
    rng = np.random.default_rng(seed)
    return [0 if rng.random() < empty else int(x) for x in rng.integers(1, most + 1, n)]


# (H, Hkv, nq, d, page, lens, window_left, window_right, sinks)
CASES = [
    # enough tiles that segments' beginnings count (4 per block of the grid): runs that begin in such
    # places, hold several segments, or cut one in the middle; empty sequences among them
    (32, 8, 1, 128, 32, _ragged(64, 1000, 1), -1, 0, 0),
    (16, 8, 1, 64, 16, _ragged(64, 700, 2), -1, 0, 0),
    (8, 8, 1, 32, 64, _ragged(70, 900, 3), -1, 0, 0),
    (32, 8, 4, 128, 64, _ragged(50, 700, 4), -1, 0, 0),                  # blocks of 16 rows
    (16, 4, 5, 64, 16, _ragged(48, 600, 5), 300, 0, 20),                 # 20 rows: two blocks, windowed
    # more entries than threads: with and without those places, and nearly all empty
    (4, 2, 1, 128, 16, _ragged(130, 60, 6), -1, 0, 0),
    (4, 4, 1, 64, 32, _ragged(200, 500, 7), -1, 0, 0),
    (8, 4, 3, 32, 16, _ragged(300, 200, 8), 50, 0, 3),
    (2, 1, 1, 64, 16, [0] * 700 + [33] + [0] * 70 + [1], -1, 0, 0),
    # blocks of 16 rows, one and several, under windows with sinks
    (16, 1, 1, 128, 16, [900, 77, 20], 100, 0, 4),
    (8, 2, 4, 128, 32, [700, 3, 129], 64, 0, 1),
    (12, 1, 3, 64, 16, [500, 40], 16, 0, 40),
    (8, 1, 5, 64, 16, [333, 48, 0], 30, 7, 2),
    (8, 2, 20, 32, 48, [400, 15], 0, 0, 17),
    (4, 1, 30, 128, 16, [200, 31], 25, 0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "H{}on{}_q{}_d{}_p{}_B{}_w{}_{}_s{}".format(
    *c[:5], len(c[5]), *c[6:]))
def test_attend(cuda_device, case):
    H, Hkv, nq, d, page, lens, wl, wr, ns = case
    pool, table = cache(lens, page, Hkv, d, 11)
    q = _randn((len(lens), H, nq, d), 12)
    got = ea.kv4_attend(q.cuda(), pool, _i32(table), _i32(lens), window=(wl, wr), sinks=ns)
    assert ea.device_status() == ea.ATTN_OK
    check(got, attend(ref.f64(q), pool.cpu().numpy(), table, lens, range(len(lens)), wl, wr, ns))


@pytest.mark.gpu
def test_a_line_of_more_than_2_to_22_places(cuda_device):
    # K = 0 and V = 1 everywhere: every weight is 1, the sums count keys and are exact in fp32, so LSE =
    # log(len) to within log2's two steps at 20, the product's and the result's rounding: 4e-6. One tile
    # (64 keys) too few or too many moves it by 6e-5.
    d, page, width = 32, 1024, 1024
    lens = [width * page, width * page - 187, 700001, 5, 0]
    pool = ea.kv4_pool(1, 1, page, d)
    k = torch.zeros((1, 1, page, d), dtype=torch.bfloat16, device="cuda")
    ea.kv4_append(pool, _i32([[0]]), _i32([0]), k, k + 1)
    table = torch.zeros((5, width), dtype=torch.int32, device="cuda")
    seqs = [(0, 1, 0, 2, 0, 3, 1, 4)[i % 8] for i in range(420)]
    assert sum(lens[s] // 64 for s in seqs) > 1 << 22
    o, lse = ea.kv4_attend(_randn((420, 1, 1, d), 1).cuda(), pool, table, _i32(lens), seqs=_i32(seqs))
    assert ea.device_status() == ea.ATTN_OK
    n = np.array([lens[s] for s in seqs])
    lse, o = ref.f64(lse).ravel(), ref.f64(o)[:, 0, 0]
    assert np.all(np.isneginf(lse[n == 0])) and not np.any(o[n == 0])
    assert np.abs(lse[n > 0] - np.log(n[n > 0])).max() <= 4e-6
    assert np.all(o[n > 0] == 1)


@pytest.mark.gpu
@pytest.mark.parametrize("pages,slots,width", [(3000, 300, 100), (40000, 200, 1000)])
def test_compaction_of_a_large_table(cuda_device, pages, slots, width):
    # more than 16 table entries per thread of the plan's launch: the table follows in a second one
    rng = np.random.default_rng(pages)
    m = Model(pages, slots, width, 16)
    assert m.reserve(list(range(slots)), [int(x) for x in rng.integers(0, 16 * pages // slots - 16, slots)])
    m.free([int(x) for x in rng.permutation(slots)[:slots // 2]])
    empty = np.nonzero(m.lens == 0)[0][:20]
    full = rng.choice(np.nonzero(m.lens)[0], len(empty))
    assert m.fork([int(x) for x in full], [int(x) for x in empty])
    d = Device(m)
    for _ in range(2):                                   # the second one finds nothing to move
        a, b, c = ea.pages_compact(d.t[0], d.t[2])
        frm, to = m.compact()
        assert int(c) == len(frm)
        assert a.cpu().tolist() == frm.tolist() + [-1] * (a.shape[0] - len(frm))
        assert b.cpu().tolist() == to.tolist() + [-1] * (b.shape[0] - len(to))
        d.same(m)
    assert ea.device_status() == ea.ATTN_OK
