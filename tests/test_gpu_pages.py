"""Pages of the K/V cache against a plain model of their state: reserving, forking, freeing (whole and
behind a window), compacting and copying, one by one, in long random sequences, and together with the
cache and the attention that read them; calls that have to be refused, and the refusals before launch."""
import ctypes

import numpy as np
import pytest
import torch

import stream_ref as ref

import exact_attention_138_b200 as ea


class Model:
    """The state as lists; every operation either succeeds as a whole or returns None."""

    def __init__(self, pages, slots, width, page):
        self.page, self.width = page, width
        self.table = np.full((slots, width), -1, np.int32)
        self.lens = np.zeros(slots, np.int32)
        self.refs = np.zeros(pages, np.int32)

    def up(self, n):
        return -(-int(n) // self.page)

    def reserve(self, seqs, counts):
        slots = len(self.lens)
        if len(set(seqs)) < len(seqs) or any(not 0 <= s < slots for s in seqs) or min(counts) < 0:
            return None
        if any(self.lens[s] + c > self.width * self.page for s, c in zip(seqs, counts)):
            return None
        need = [self.up(self.lens[s] + c) - self.up(self.lens[s]) for s, c in zip(seqs, counts)]
        free = np.nonzero(self.refs == 0)[0]
        if sum(need) > len(free):
            return None
        start, at = [], 0
        for s, c, m in zip(seqs, counts, need):
            have = self.up(self.lens[s])
            self.table[s, have:have + m] = free[at:at + m]
            at += m
            start.append(int(self.lens[s]))
            self.lens[s] += c
        self.refs[free[:at]] = 1
        return start

    def fork(self, src, dst):
        slots = len(self.lens)
        if any(not 0 <= s < slots for s in list(src) + list(dst)) or len(set(dst)) < len(dst):
            return None
        if set(src) & set(dst) or any(self.lens[d] for d in dst):
            return None
        part = [int(self.lens[s]) % self.page > 0 for s in src]
        free = np.nonzero(self.refs == 0)[0]
        if sum(part) > len(free):
            return None
        frm, to, at = [], [], 0
        for s, d, p in zip(src, dst, part):
            full = int(self.lens[s]) // self.page
            self.table[d, :full] = self.table[s, :full]
            for pg in self.table[s, :full]:
                if pg >= 0:
                    self.refs[pg] += 1
            old = self.table[s, full] if p else -1
            if p:
                self.table[d, full] = free[at]
                self.refs[free[at]] = 1
                at += 1
            frm.append(int(old))
            to.append(int(self.table[d, full]) if p and old >= 0 else -1)
            self.lens[d] = self.lens[s]
        return frm, to

    def free(self, seqs, window=None, sinks=0):
        for s in seqs:
            if not 0 <= s < len(self.lens):
                continue
            n = int(self.lens[s])
            for m in range(self.up(n)):
                seen = window is not None and (m * self.page < sinks or (m + 1) * self.page > n - window)
                if not seen and self.table[s, m] >= 0:
                    self.refs[self.table[s, m]] -= 1
                    self.table[s, m] = -1
            if window is None:
                self.lens[s] = 0

    def compact(self):
        live = np.nonzero(self.refs)[0]
        low = len(live)
        frm = live[live >= low]
        to = np.nonzero(self.refs[:low] == 0)[0]
        now = np.arange(len(self.refs))
        now[frm] = to
        self.table = np.where(self.table >= 0, now[np.maximum(self.table, 0)], -1).astype(np.int32)
        self.refs[to] = self.refs[frm]
        self.refs[frm] = 0
        return frm, to


class Device:
    def __init__(self, m):
        self.t = [torch.from_numpy(x.copy()).cuda() for x in (m.table, m.lens, m.refs)]
        self.page = m.page

    def state(self):
        return (*self.t, self.page)

    def same(self, m):
        for got, want, name in zip(self.t, (m.table, m.lens, m.refs), ("table", "lens", "refs")):
            got = got.cpu().numpy()
            assert np.array_equal(got, want), (name, np.argwhere(got != want)[:5])


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


SIZES = [(40, 12, 6, 4), (300, 40, 16, 16), (20000, 64, 300, 64), (70000, 30, 3000, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("pages,slots,width,page", SIZES)
def test_random_sequences_of_calls(cuda_device, pages, slots, width, page):
    rng = np.random.default_rng(pages)
    m = Model(pages, slots, width, page)
    d = Device(m)
    refused = 0
    for step in range(60):
        kind = rng.choice(["reserve", "reserve", "fork", "free", "evict", "compact"])
        n = int(rng.integers(1, max(2, slots // 3)))
        seqs = [int(x) for x in rng.permutation(slots)[:n]]
        if kind == "reserve":
            most = int(rng.choice([3, page * 2, width * page // 2]))
            counts = [int(x) for x in rng.integers(0, most, n)]
            want = m.reserve(seqs, counts)
            got = ea.pages_reserve(*d.state(), _i32(seqs), _i32(counts)).cpu().tolist()
            assert got == (want if want is not None else [-1] * n)
        elif kind == "fork":
            full, empty = np.nonzero(m.lens)[0], np.nonzero(m.lens == 0)[0]
            if not len(full) or not len(empty):
                continue
            dst = [int(x) for x in rng.permutation(empty)[:n]]
            src = [int(x) for x in rng.choice(full, len(dst))]
            want = m.fork(src, dst)
            got = [x.cpu().tolist() for x in ea.pages_fork(*d.state(), _i32(src), _i32(dst))]
            assert got == (list(want) if want is not None else [[-1] * len(dst)] * 2)
        elif kind == "free":
            twice = seqs + seqs[:2]
            m.free(seqs)
            ea.pages_free(*d.state(), _i32(twice))
            want = ()
        elif kind == "evict":
            w, s = int(rng.integers(0, width * page)), int(rng.integers(0, 3 * page))
            m.free(seqs, w, s)
            ea.pages_free(*d.state(), _i32(seqs), window=(w, 0), sinks=s)
            want = ()
        else:
            frm, to = m.compact()
            a, b, c = ea.pages_compact(d.t[0], d.t[2])
            assert int(c) == len(frm)
            assert a.cpu().tolist() == frm.tolist() + [-1] * (a.shape[0] - len(frm))
            assert b.cpu().tolist() == to.tolist() + [-1] * (b.shape[0] - len(to))
            want = ()
        assert ea.device_status() == (ea.ATTN_ERR_PAGES if want is None else ea.ATTN_OK)
        refused += want is None
        d.same(m)
    held = np.bincount(m.table[m.table >= 0], minlength=pages)
    assert np.array_equal(held, m.refs)
    assert pages > 1000 or refused > 0


@pytest.mark.gpu
@pytest.mark.parametrize("call", [
    lambda d: ea.pages_reserve(*d.state(), _i32([1, 1]), _i32([1, 1])),          # the same row twice
    lambda d: ea.pages_reserve(*d.state(), _i32([0, 9]), _i32([1, 1])),          # outside the table
    lambda d: ea.pages_reserve(*d.state(), _i32([0, -1]), _i32([1, 1])),
    lambda d: ea.pages_reserve(*d.state(), _i32([0, 1]), _i32([1, -1])),
    lambda d: ea.pages_reserve(*d.state(), _i32([0, 1]), _i32([1, 2**31 - 1])),  # no such columns
    lambda d: ea.pages_reserve(*d.state(), _i32([2, 3]), _i32([48, 17])),        # 5 pages, 4 are free
    lambda d: ea.pages_fork(*d.state(), _i32([0, 0]), _i32([2, 2])),
    lambda d: ea.pages_fork(*d.state(), _i32([0]), _i32([1])),                   # not empty
    lambda d: ea.pages_fork(*d.state(), _i32([0, 2]), _i32([2, 3])),             # copied and replaced
    lambda d: ea.pages_fork(*d.state(), _i32([0, 4]), _i32([2, 3])),
    lambda d: ea.pages_fork(*d.state(), _i32([0, 1]), _i32([2, -5])),
])
def test_refused_calls_change_nothing(cuda_device, call):
    m = Model(7, 4, 3, 16)
    m.reserve([0, 1], [20, 16])
    d = Device(m)
    ea.device_status()
    out = call(d)
    for t in (out if isinstance(out, tuple) else (out,)):
        assert bool((t == -1).all())
    assert ea.device_status() == ea.ATTN_ERR_PAGES and ea.device_status() == ea.ATTN_OK
    d.same(m)
    # the last free page can still be taken, and an empty request is served
    assert m.reserve([2, 3], [64 - 16, 1]) == ea.pages_reserve(*d.state(), _i32([2, 3]), _i32([48, 1])).cpu().tolist()
    assert m.reserve([0], [0]) == ea.pages_reserve(*d.state(), _i32([0]), _i32([0])).cpu().tolist()
    d.same(m)
    assert ea.device_status() == ea.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("shape,dtype,layered", [
    ((50, 3, 1280), torch.uint8, False), ((9, 50, 40), torch.float32, True), ((50, 70000), torch.bfloat16, False),
    ((2, 50, 16), torch.uint8, True)])
def test_copy(cuda_device, shape, dtype, layered):
    g = torch.Generator().manual_seed(1)
    pool = torch.randint(-100, 100, shape, generator=g).to(dtype)
    frm = [4, -1, 6, 49, 60, 7, 8, 4]
    to = [10, 11, -1, 0, 12, 50, 13, 14]
    dev = pool.cuda()
    ea.pages_copy(dev, _i32(frm), _i32(to), layered=layered)
    want = pool.clone()
    for a, b in zip(frm, to):
        if 0 <= a < 50 and 0 <= b < 50:
            if layered:
                want[:, b] = pool[:, a]
            else:
                want[b] = pool[a]
    assert torch.equal(dev.cpu(), want)
    dev = pool.cuda()                                # count: the first entry alone, then none
    ea.pages_copy(dev, _i32(frm), _i32(to), count=_i32([1]), layered=layered)
    want = pool.clone()
    if layered:
        want[:, 10] = pool[:, 4]
    else:
        want[10] = pool[4]
    assert torch.equal(dev.cpu(), want)
    ea.pages_copy(dev, _i32(to), _i32(frm), count=_i32([0]), layered=layered)
    assert torch.equal(dev.cpu(), want)


@pytest.mark.gpu
def test_a_generation_from_prompt_to_forks_and_eviction(cuda_device):
    """The operators as they are used together: prompts of three sequences are reserved, quantised and
    attended to; two beams fork from one; every beam decodes under a window with sinks while pages behind
    it are given back; one sequence ends, the pool is compacted; results always as the model's."""
    Hkv, H, d, page, wl, ns = 2, 4, 64, 16, 40, 3
    m = Model(60, 8, 20, page)
    dev = Device(m)
    pool = torch.full((60, Hkv, page // 16 * 20 * d), 255, dtype=torch.uint8).cuda()
    host = pool.cpu().numpy().copy()
    g = torch.Generator().manual_seed(7)
    draw = lambda *s: torch.randn(s, generator=g).bfloat16()              # noqa: E731

    def grow(seqs, counts):
        n = max(counts)
        k, v = draw(len(seqs), Hkv, n, d), draw(len(seqs), Hkv, n, d)
        start = ea.pages_reserve(*dev.state(), _i32(seqs), _i32(counts))
        assert start.cpu().tolist() == m.reserve(seqs, counts)
        ea.kv4_append(pool, dev.t[0], start, k.cuda(), v.cuda(), counts=_i32(counts), seqs=_i32(seqs))
        for i, (s, c) in enumerate(zip(seqs, counts)):
            for t in range(c):
                pos = int(m.lens[s]) - c + t
                for h in range(Hkv):
                    ref.store(host, m.table[s][pos // page], h, pos % page, ref.f64(k[i, h, t]), ref.f64(v[i, h, t]))

    def look(seqs):
        q = draw(len(seqs), H, 1, d)
        o, lse = ea.kv4_attend(q.cuda(), pool, dev.t[0], dev.t[1], window=(wl, 0), sinks=ns, seqs=_i32(seqs))
        ro, rl, eo, el = ref.attend(ref.f64(q), host, m.table, m.lens, seqs, page, wl, 0, ns)
        assert np.all(np.abs(ref.f64(o) - ro) <= eo) and np.all(np.abs(ref.f64(lse) - rl) <= el)

    grow([0, 1, 2], [100, 17, 33])
    look([0, 1, 2])
    frm, to = ea.pages_fork(*dev.state(), _i32([0, 0]), _i32([3, 4]))
    assert (frm.cpu().tolist(), to.cpu().tolist()) == m.fork([0, 0], [3, 4])
    ea.pages_copy(pool, frm, to)
    for a, b in zip(frm.cpu().tolist(), to.cpu().tolist()):
        host[b] = host[a]
    beams = [0, 3, 4, 1]
    for step in range(20):
        grow(beams, [1] * 4)
        look(beams)
        ea.pages_free(*dev.state(), _i32(beams), window=(wl, 0), sinks=ns)
        m.free(beams, wl, ns)
        if step == 9:
            ea.pages_free(*dev.state(), _i32([2]))
            m.free([2])
            ea.pages_copy(pool, *ea.pages_compact(dev.t[0], dev.t[2]))
            a, b = m.compact()
            host[b] = host[a]
        dev.same(m)
    assert np.count_nonzero(m.refs) < 25 and ea.device_status() == ea.ATTN_OK
    live = np.nonzero(m.refs)[0]
    assert np.array_equal(pool.cpu().numpy()[live], host[live])


@pytest.mark.gpu
def test_a_captured_step_on_another_stream(cuda_device):
    m = Model(200, 10, 10, 16)
    m.reserve([0, 1], [50, 30])
    d = Device(m)
    pool = torch.randint(0, 256, (200, 1, 640), dtype=torch.uint8, generator=torch.Generator().manual_seed(3)).cuda()
    src, dst, ones = _i32([0, 1, 0]), _i32([5, 6, 7]), _i32([1, 1, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ea.pages_free(*d.state(), dst)
        frm, to = ea.pages_fork(*d.state(), src, dst)
        ea.pages_copy(pool, frm, to)
        start = ea.pages_reserve(*d.state(), dst, ones)
        moves = ea.pages_compact(d.t[0], d.t[2])
        ea.pages_copy(pool, *moves)
    d.same(m)                                         # capturing ran nothing
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        m.free([5, 6, 7])
        assert (frm.cpu().tolist(), to.cpu().tolist()) == m.fork([0, 1, 0], [5, 6, 7])
        assert start.cpu().tolist() == m.reserve([5, 6, 7], [1, 1, 1])
        m.compact()
        d.same(m)
    assert ea.device_status() == ea.ATTN_OK


FAKE = 1 << 20
P = ctypes.c_void_p


@pytest.mark.parametrize("kw", [
    dict(table=0), dict(lens=0), dict(refs=0), dict(refs=FAKE + 4), dict(table=FAKE + 2), dict(x=0), dict(y=0),
    dict(pages=0), dict(slots=0), dict(slots=(1 << 18) + 1), dict(width=0), dict(page=0), dict(n=0),
    dict(width=1 << 28), dict(x=FAKE + 1)])
def test_refusals_before_launch(kw):
    a = dict(table=FAKE, lens=FAKE, refs=FAKE, x=FAKE, y=FAKE, pages=9, slots=4, width=3, page=16, n=2)
    a.update(kw)
    st = [P(a["table"]), P(a["lens"]), P(a["refs"])]
    sizes = (a["pages"], a["slots"], a["width"], a["page"], a["n"])
    assert ea.attn_pages_reserve(*st, P(a["x"]), P(a["y"]), P(FAKE), *sizes, None) == ea.ATTN_ERR_INVALID
    assert ea.attn_pages_fork(*st, P(a["x"]), P(a["y"]), P(FAKE), P(FAKE), *sizes, None) == ea.ATTN_ERR_INVALID
    if "y" not in kw:
        assert ea.attn_pages_free(*st, P(a["x"]), *sizes, -1, 0, None) == ea.ATTN_ERR_INVALID
    if not {"lens", "page", "n"} & set(kw) and kw != dict(width=1 << 28):
        assert ea.attn_pages_compact(st[0], st[2], P(a["x"]), P(a["y"]), P(FAKE), *sizes[:3], P(FAKE), 1 << 30,
                                     None) == ea.ATTN_ERR_INVALID


def test_more_refusals():
    f = P(FAKE)
    assert ea.attn_pages_reserve(f, f, f, f, f, f, 9, 4, 3, 16, 8193, None) == ea.ATTN_ERR_INVALID
    assert ea.attn_pages_free(f, f, f, f, 9, 4, 3, 16, 2, 5, -1, None) == ea.ATTN_ERR_INVALID
    assert ea.attn_pages_compact(f, f, f, f, f, 9, 4, 3, f, 51, None) == ea.ATTN_ERR_WORKSPACE
    assert ea.attn_pages_compact(f, f, f, f, f, 9, 4, 3, P(FAKE + 4), 52, None) == ea.ATTN_ERR_INVALID
    assert ea.attn_pages_workspace_bytes(9) == 52 and ea.attn_pages_workspace_bytes(0) == 0
    for kw in (dict(layers=0), dict(pages=0), dict(each=0), dict(each=24), dict(n=0), dict(pool=FAKE + 8), dict(to=0)):
        a = dict(pool=FAKE, to=FAKE, layers=1, pages=4, each=32, n=2)
        a.update(kw)
        assert ea.attn_pages_copy(P(a["pool"]), f, P(a["to"]), None, a["layers"], a["pages"], a["each"], a["n"],
                                  None) == ea.ATTN_ERR_INVALID
    assert ea.attn_error_string(ea.ATTN_ERR_PAGES) != "unknown error"


def test_binding_refuses_host_tensors_and_wrong_types():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)                      # noqa: E731
    st = (i(4, 3), i(4), i(9), 16)
    pool = torch.zeros((9, 64), dtype=torch.uint8)
    for f in (lambda: ea.pages_reserve(*st, i(2), i(2)), lambda: ea.pages_reserve(*st, i(2), i(3)),
              lambda: ea.pages_fork(*st, i(2), i(2).long()), lambda: ea.pages_free(i(4, 3), i(5), i(9), 16, i(2)),
              lambda: ea.pages_free(*st, i(2)), lambda: ea.pages_compact(i(4, 3), i(9).float()),
              lambda: ea.pages_compact(i(4, 3), i(9)), lambda: ea.pages_copy(pool, i(2), i(2)),
              lambda: ea.pages_copy(pool, i(2), i(3)), lambda: ea.pages_copy(pool[0, 0], i(2), i(2))):
        with pytest.raises(ValueError):
            f()
