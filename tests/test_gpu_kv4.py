"""The 4-bit paged cache against its fp64 reference: the bytes that appending writes (and leaves), what
reading back gives, attention over the cache for the newest tokens, and the refusals. Ragged and empty
sequences, pages of every size, tokens that end inside a block, windows with sinks, missing pages,
garbage and NaN behind the last token, captured calls, another stream."""
import ctypes

import numpy as np
import pytest
import torch

import stream_ref as ref

import exact_attention_138_b200 as ea


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _randn(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).bfloat16()


def _table(lens, page, width, seed, spare=3):
    """Rows of distinct page numbers in a random order, -1 behind each sequence's last page."""
    held = [-(-n // page) for n in lens]
    pages = sum(held) + spare
    order = np.random.default_rng(seed).permutation(pages)
    t = np.full((len(lens), width), -1, np.int32)
    at = 0
    for i, n in enumerate(held):
        t[i, :n] = order[at:at + n]
        at += n
    return t, pages


def _noise(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)


APPENDS = [
    # (Hkv, d, page, starts, counts, n)
    (2, 128, 16, [0], [1], 1),
    (1, 32, 16, [5, 0], [40, 16], 40),
    (3, 64, 32, [31, 1, 16], [1, 20, 33], 33),
    (2, 128, 64, [63, 100, 7], [70, 0, 16], 70),
    (1, 128, 48, [47, -1], [50, 50], 50),              # the second entry is left out
    (2, 64, 128, [129], [14], 20),
]


def _scale_ties(sign):
    """(32, 32) bf16: groups whose range is 15 m for odd m of 9 bits, so that a 15th of it lies midway
    between two bf16 values. Greatest and least have 8 bits at most."""
    rows = []
    for i in range(32):
        m = 2 * (128 + 4 * i + i % 4) + 1                    # 9 bits, odd
        width = 15 * m
        step = 16 if width < 4096 else 32
        hi, lo = width // step * step, -(width % step)
        between = [lo + (hi - lo) * (x + 0.5) / 30 for x in range(30)]
        rows.append([hi, lo] + between)
    return sign * torch.tensor(rows).bfloat16()


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1, -1])
def test_append_rounds_exact_ties_of_the_scale_to_even(cuda_device, sign):
    k = _scale_ties(sign)
    x = ref.f64(k)
    fifteenth = (x.max(-1) - x.min(-1)) / 15
    s = ref.quantise(x)[1][:, 0]
    other = 2 * fifteenth - s                                # the neighbour that is as near
    assert (s != other).all() and np.array_equal(ref.bf16(other), other)
    k = k.view(1, 1, 32, 32)
    pool = torch.zeros((2, 1, 20 * 32), dtype=torch.uint8)
    want = pool.numpy().copy()
    for t in range(32):
        ref.store(want, t // 16, 0, t % 16, ref.f64(k[0, 0, t]), ref.f64(k[0, 0, t]))
    dev = pool.cuda()
    ea.kv4_append(dev, _i32([[0, 1]]), _i32([0]), k.cuda(), k.cuda())
    assert np.array_equal(dev.cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("case", APPENDS, ids=str)
def test_append_writes_exactly_its_tokens(cuda_device, case):
    Hkv, d, page, starts, counts, n = case
    B = len(starts)
    ends = [max(0, s + c) for s, c in zip(starts, counts)]
    table, pages = _table([e + 20 for e in ends], page, 12, 1)
    k, v = _randn((B, Hkv, n, d), 2), _randn((B, Hkv, n, d), 3)
    k[0, 0, 0, :32] = 1.25                                  # a constant group
    k[0, -1, 0, :32] = torch.arange(32).bfloat16() / 2      # values on borders: ties
    pool = _noise((pages, Hkv, page // 16 * 20 * d), 4)
    want = pool.numpy().copy()
    for i in range(B):
        for t in range(counts[i] if starts[i] >= 0 else 0):
            pos = starts[i] + t
            for h in range(Hkv):
                ref.store(want, table[i][pos // page], h, pos % page, ref.f64(k[i, h, t]), ref.f64(v[i, h, t]))
    dev = pool.cuda()
    ea.kv4_append(dev, _i32(table), _i32(starts), k.cuda(), v.cuda(), counts=_i32(counts))
    assert np.array_equal(dev.cpu().numpy(), want)
    gk, gv = ea.kv4_gather(dev, _i32(table), _i32(starts), n, d, counts=_i32(counts))
    for i in range(B):
        c = counts[i] if starts[i] >= 0 else 0
        for got, x in ((gk, k), (gv, v)):
            exp = torch.zeros_like(x[i])
            if c:
                q, s, lo = ref.quantise(ref.f64(x[i, :, :c]))
                exp[:, :c] = torch.from_numpy(ref.value(q, s, lo)).float().bfloat16()
            assert torch.equal(got[i].cpu(), exp)


@pytest.mark.gpu
def test_append_through_rows_and_off_the_table(cuda_device):
    # rows of the table in another order; an entry outside it, a start beyond it and a page that is
    # not there write nothing
    d, page = 64, 16
    table = np.array([[0, 1, -1], [2, 3, 99], [4, 5, 6]], np.int32)
    pool = _noise((7, 1, 20 * d), 1)
    k, v = _randn((4, 1, 20, d), 2), _randn((4, 1, 20, d), 3)
    seqs, start = [2, 0, 7, 1], [3, 20, 0, 40]
    want = pool.numpy().copy()
    for i, (r, s) in enumerate(zip(seqs, start)):
        for t in range(20):
            m = (s + t) // page
            if r < 3 and m < 3 and 0 <= table[r][m] < 7:
                ref.store(want, table[r][m], 0, (s + t) % page, ref.f64(k[i, 0, t]), ref.f64(v[i, 0, t]))
    dev = pool.cuda()
    ea.kv4_append(dev, _i32(table), _i32(start), k.cuda(), v.cuda(), seqs=_i32(seqs))
    assert np.array_equal(dev.cpu().numpy(), want)
    gk, _ = ea.kv4_gather(dev, _i32(table), _i32(start), 20, d, seqs=_i32(seqs))
    assert not torch.any(gk[2]) and not torch.any(gk[1, :, 12:]) and torch.any(gk[1, :, :12])


@pytest.mark.gpu
def test_groups_that_are_not_finite_and_far_apart(cuda_device):
    d, page = 32, 16
    k = _randn((1, 1, 6, d), 1)
    k[0, 0, 0, 3] = float("nan")
    k[0, 0, 1, 3] = float("inf")
    k[0, 0, 2] = 1e-38                                       # spread below 2^-100
    k[0, 0, 3, 0], k[0, 0, 3, 1:] = -1e30, 1e30
    k[0, 0, 4] *= 1e-20
    pool = ea.kv4_pool(1, 1, page, d)
    table = _i32([[0]])
    ea.kv4_append(pool, table, _i32([0]), k.cuda(), k.cuda())
    gk, gv = ea.kv4_gather(pool, table, _i32([0]), 6, d)
    assert torch.isnan(gk[0, 0, :2]).all() and torch.isnan(gv[0, 0, :2]).all()
    q, s, lo = ref.quantise(ref.f64(k[0, 0, 2:]))
    want = torch.from_numpy(ref.value(q, s, lo)).float().bfloat16()
    assert torch.equal(gk[0, 0, 2:].cpu(), want) and torch.equal(gv[0, 0, 2:].cpu(), want)


# (H, Hkv, nq, d, page, lens, window_left, window_right, sinks)
ATTENDS = [
    (1, 1, 1, 32, 16, [1], -1, 0, 0),
    (4, 1, 1, 128, 16, [0, 1, 15, 16, 17, 200], -1, 0, 0),
    (8, 2, 1, 128, 64, [1000, 3, 130], -1, 0, 0),
    (2, 2, 3, 64, 32, [2, 300, 64, 1], -1, 0, 0),               # fewer tokens than queries
    (8, 1, 5, 128, 64, [333, 48], -1, 0, 0),                    # 40 rows of one head: three blocks
    (16, 1, 1, 64, 48, [777], -1, 0, 0),                        # 16 rows: one block of 16
    (6, 2, 4, 32, 128, [129, 500], -1, 0, 0),                   # 12 rows
    (4, 4, 1, 128, 16, [500, 90, 17], 64, 0, 4),
    (4, 2, 4, 64, 16, [600, 100, 31], 0, 0, 1),
    (4, 2, 2, 128, 32, [900, 70], 200, 0, 70),
    (2, 1, 3, 64, 16, [400], 20, 5, 3),                         # keys behind the query
    (2, 1, 6, 32, 16, [300], -1, -1, 0),                        # all of them
    (8, 8, 1, 128, 64, [5000, 1, 2500], -1, 0, 0),              # many runs
    (3, 1, 1, 64, 32, [20000], -1, 0, 0),
]


def _case(case, seed=5, scale_v=1.0):
    H, Hkv, nq, d, page, lens = case[:6]
    B = len(lens)
    table, pages = _table(lens, page, max(-(-max(lens) // page), 1) + 1, seed)
    pool = torch.full((pages, Hkv, page // 16 * 20 * d), 255, dtype=torch.uint8).cuda()   # NaN parameters
    n = max(max(lens), 1)
    k, v = _randn((B, Hkv, n, d), seed + 1), _randn((B, Hkv, n, d), seed + 2)
    k[..., :2] *= 6
    v = (v.float() * scale_v).bfloat16()
    ea.kv4_append(pool, _i32(table), _i32([0] * B), k.cuda(), v.cuda(), counts=_i32(lens))
    return _randn((B, H, nq, d), seed + 3), pool, table


def _check(got, want):
    o, lse = got
    ro, rl, eo, el = want
    none = np.isneginf(rl)
    gl = ref.f64(lse)
    assert np.array_equal(np.isneginf(gl), none)
    off = np.abs(np.where(none, 0, gl) - np.where(none, 0, rl)) - el
    assert off.max() <= 0, ("lse", float(off.max()))
    off = np.abs(ref.f64(o) - ro) - eo
    assert off.max() <= 0, ("o", float(off.max()), np.unravel_index(off.argmax(), off.shape))
    assert not np.any(ref.f64(o)[none])


@pytest.mark.gpu
@pytest.mark.parametrize("case", ATTENDS, ids=str)
def test_attend(cuda_device, case):
    q, pool, table = _case(case)
    H, Hkv, nq, d, page, lens, wl, wr, ns = case
    got = ea.kv4_attend(q.cuda(), pool, _i32(table), _i32(lens), window=(wl, wr), sinks=ns)
    assert ea.device_status() == ea.ATTN_OK
    _check(got, ref.attend(ref.f64(q), pool.cpu().numpy(), table, lens, range(len(lens)), page, wl, wr, ns))


@pytest.mark.gpu
@pytest.mark.parametrize("scale_v", [1e-34, 1e-12, 1e20, 1e34])
def test_attend_values_of_any_size(cuda_device, scale_v):
    case = (4, 1, 1, 64, 16, [300, 40], -1, 0, 0)
    q, pool, table = _case(case, scale_v=scale_v)
    got = ea.kv4_attend(q.cuda(), pool, _i32(table), _i32(case[5]))
    _check(got, ref.attend(ref.f64(q), pool.cpu().numpy(), table, case[5], range(2), 16, -1, 0, 0))


@pytest.mark.gpu
def test_attend_value_sizes_that_grow_along_the_keys(cuda_device):
    # the power of two on P s has to follow the largest s; small ones before it keep their weight
    case = (2, 1, 1, 32, 16, [600], -1, 0, 0)
    q, pool, table = _case(case)
    k, v = _randn((1, 1, 600, 32), 8), _randn((1, 1, 600, 32), 9)
    v = (v.float() * torch.logspace(-20, 10, 600)[None, None, :, None]).bfloat16()
    ea.kv4_append(pool, _i32(table), _i32([0]), k.cuda(), v.cuda())
    got = ea.kv4_attend(q.cuda(), pool, _i32(table), _i32([600]))
    _check(got, ref.attend(ref.f64(q), pool.cpu().numpy(), table, [600], [0], 16, -1, 0, 0))


@pytest.mark.gpu
def test_attend_rows_missing_pages_and_rows_off_the_table(cuda_device):
    case = (4, 2, 2, 64, 16, [200, 90, 33], 30, 0, 5)
    q, pool, table = _case(case)
    table[0, 2:9] = -1                      # behind the window: freed
    table[1, 4] = -1                        # and one inside it
    table[2, 1] = 1 << 20                   # no page of the pool
    seqs = [2, 0, 0, 1, 3, -1]              # the same row twice, rows outside the table
    q = torch.cat((q, q + 1))
    got = ea.kv4_attend(q.cuda(), pool, _i32(table), _i32(case[5]), window=(30, 0), sinks=5, seqs=_i32(seqs))
    _check(got, ref.attend(ref.f64(q), pool.cpu().numpy(), table, case[5], seqs, 16, 30, 0, 5))


@pytest.mark.gpu
def test_attend_nan_where_it_is_not_seen_and_where_it_is(cuda_device):
    case = (2, 1, 3, 64, 16, [100], 20, 0, 2)
    q, pool, table = _case(case)
    k = _randn((1, 1, 100, 64), 3)
    k[0, 0, 40:60] = float("nan")           # behind every query's window
    k[0, 0, 78] = float("nan")              # query 0 (at 97) sees 77 .. 97, query 2 (at 99) 79 .. 99
    ea.kv4_append(pool, _i32(table), _i32([0]), k.cuda(), k.cuda())
    o, lse = ea.kv4_attend(q.cuda(), pool, _i32(table), _i32([100]), window=(20, 0), sinks=2)
    assert torch.isnan(o[:, :, :2]).all() and torch.isnan(lse[:, :, :2]).all()
    ro, rl, eo, el = ref.attend(ref.f64(q[:, :, 2:]), pool.cpu().numpy(), table, [100], [0], 16, 20, 0, 2)
    _check((o[:, :, 2:], lse[:, :, 2:]), (ro, rl, eo, el))


@pytest.mark.gpu
def test_one_captured_call_serves_a_growing_sequence(cuda_device):
    case = (4, 2, 1, 128, 16, [700, 50], -1, 0, 0)
    q, pool, table = _case(case)
    qd, td, lens = q.cuda(), _i32(table), _i32([3, 1])
    start = lens - 1
    k, v = (x[:, :, :1].contiguous().cuda() for x in (_randn((2, 2, 2, 128), 1), _randn((2, 2, 2, 128), 2)))
    args = dict(out=torch.empty_like(qd), lse=torch.empty(2, 4, 1, device="cuda"))
    ea.kv4_attend(qd, pool, td, lens, **args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ea.kv4_append(pool, td, start, k, v)
        ea.kv4_attend(qd, pool, td, lens, **args)
    for n in ([3, 1], [64, 50], [699, 49], [0, 5]):
        lens.copy_(_i32(n))
        start.copy_(_i32(n) - 1)
        for t in args.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        _check((args["out"], args["lse"]), ref.attend(ref.f64(q), pool.cpu().numpy(), table, n, [0, 1], 16, -1, 0, 0))


@pytest.mark.gpu
def test_another_stream_and_repeatability(cuda_device):
    case = (8, 2, 1, 128, 32, [4000, 77, 1500], 900, 0, 4)
    q, pool, table = _case(case)
    args = (q.cuda(), pool, _i32(table), _i32(case[5]))
    kw = dict(window=(900, 0), sinks=4)
    first = ea.kv4_attend(*args, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    others = [ea.kv4_attend(*args, stream=s, **kw) for _ in range(3)]
    s.synchronize()
    for o, l in others:
        assert torch.equal(o, first[0]) and torch.equal(l, first[1])


@pytest.mark.gpu
def test_attend_agrees_with_the_forward_on_what_the_cache_stands_for(cuda_device):
    # a prompt's last rows through the prefill kernel on the gathered cache, and through the cache
    case = (4, 2, 4, 128, 64, [500], 100, 0, 6)
    q, pool, table = _case(case)
    k, v = ea.kv4_gather(pool, _i32(table), _i32([0]), 500, 128)
    a, la = ea.forward(q.cuda(), k, v, window=(100, 0), sinks=6)
    b, lb = ea.kv4_attend(q.cuda(), pool, _i32(table), _i32([500]), window=(100, 0), sinks=6)
    # K and V rounded to bf16: scores move by 2^-8 sum |q k| scale, O by that and 2 roundings of P and V
    ke, ve = ref._expand(ref.f64(k), 4), ref._expand(ref.f64(v), 4)
    shift = ref.BF16 * np.einsum("bhid,bhjd->bhij", np.abs(ref.f64(q)), np.abs(ke)).max() * 128 ** -0.5
    assert np.abs(ref.f64(la) - ref.f64(lb)).max() <= shift
    assert np.abs(ref.f64(a) - ref.f64(b)).max() <= (2 * shift + 4 * ref.BF16) * np.abs(ve).max()


FAKE = 1 << 20


def _attend_code(**kw):
    a = dict(q=FAKE, pool=FAKE, table=FAKE, lens=FAKE, o=FAKE, lse=FAKE, ws=FAKE, pages=4, slots=2, width=3,
             page=16, B=2, H=4, Hkv=2, nq=1, d=64, scale=0.1, ns=0, bytes=1 << 40, seqs=0)
    a.update(kw)
    p = lambda n: ctypes.c_void_p(a[n])                                  # noqa: E731
    return ea.attn_kv4_attend(p("q"), p("pool"), p("table"), p("seqs"), p("lens"), p("o"), p("lse"), a["pages"],
                              a["slots"], a["width"], a["page"], a["B"], a["H"], a["Hkv"], a["nq"], a["d"],
                              a["scale"], 5, 0, a["ns"], p("ws"), a["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(pool=0), 1), (dict(table=0), 1), (dict(lens=0), 1), (dict(o=0), 1), (dict(lse=0), 1),
    (dict(ws=0), 1), (dict(ws=FAKE + 16), 1), (dict(pool=FAKE + 8), 1), (dict(q=FAKE + 2), 1), (dict(page=8), 1),
    (dict(page=24), 1), (dict(pages=0), 1), (dict(slots=0), 1), (dict(width=0), 1), (dict(B=0), 1), (dict(B=3), 1),
    (dict(B=70000, seqs=FAKE), 1), (dict(H=3), 1), (dict(Hkv=0), 1), (dict(nq=0), 1), (dict(scale=0.0), 1),
    (dict(ns=-1), 1), (dict(lens=FAKE + 2), 1), (dict(table=FAKE + 1), 1), (dict(seqs=FAKE + 2), 1), (dict(width=1 << 28), 1), (dict(d=48), 2), (dict(bytes=100), 5)])
def test_attend_refusals(kw, code):
    assert _attend_code(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(start=0), 1), (dict(k=0), 1), (dict(v=FAKE + 4), 1), (dict(n=0), 1), (dict(page=17), 1), (dict(d=256), 2),
    (dict(B=3), 1), (dict(Hkv=0), 1)])
def test_rows_refusals(kw, code):
    a = dict(start=FAKE, k=FAKE, v=FAKE, n=4, page=16, d=64, B=2, Hkv=1)
    a.update(kw)
    p = lambda x: ctypes.c_void_p(x)                                     # noqa: E731
    for f in (ea.attn_kv4_append, ea.attn_kv4_gather):
        assert f(p(FAKE), p(FAKE), None, p(a["start"]), None, p(a["k"]), p(a["v"]), 4, 2, 3, a["page"], a["B"],
                 a["Hkv"], a["n"], a["d"], None) == code


def test_page_bytes_and_workspace_sizes():
    assert ea.attn_kv4_page_bytes(64, 8, 128) == 4 * 8 * 20 * 128
    assert ea.attn_kv4_page_bytes(24, 8, 128) == 0 == ea.attn_kv4_page_bytes(16, 1, 48)
    assert ea.attn_kv4_workspace_bytes(32, 8, 1, 128) > 0
    assert ea.attn_kv4_workspace_bytes(3, 2, 1, 128) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    k = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    pool = torch.zeros((3, 2, 20 * 64), dtype=torch.uint8)
    table, one = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16)
    bad = [lambda: ea.kv4_append(pool, table, one, k, k), lambda: ea.kv4_gather(pool, table, one, 4, 64),
           lambda: ea.kv4_attend(q, pool, table, one),                   # host tensors
           lambda: ea.kv4_append(pool, table, one, k[:, :1], k),
           lambda: ea.kv4_append(pool, table.long(), one, k, k),
           lambda: ea.kv4_append(pool, table, one, k.float(), k.float()),
           lambda: ea.kv4_append(pool, table, one, k, k, counts=torch.zeros(2, dtype=torch.int32)),
           lambda: ea.kv4_append(pool[..., :1279], table, one, k, k),
           lambda: ea.kv4_attend(q[:, :3], pool, table, one), lambda: ea.kv4_attend(q[0], pool, table, one),
           lambda: ea.kv4_attend(q, pool, table, one, sinks=-2), lambda: ea.kv4_gather(pool, table, one, 0, 64)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ea.AttnError):
        ea.kv4_gather(pool, table, one, 4, 48)
