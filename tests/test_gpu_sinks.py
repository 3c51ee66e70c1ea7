"""GPU parity of windows with sinks against the fp64 reference: forward (bf16, fp32) and backward
(bf16, both dQ modes), whole tensors, element by element, with the bounds that bf16 rounding of P, dS,
O and the results gives (stream_ref). Sinks inside, at and behind tile borders, pairs of query tiles
whose windows join the sinks or not, grids with and without a key split, empty rows."""
import ctypes

import numpy as np
import pytest
import torch

import stream_ref as ref
from parity_util import TOL_LSE

import exact_attention_138_b200 as ea

# (B, H, Hkv, nq, nk, d, window_left, window_right, sinks)
CASES = [
    (1, 2, 2, 300, 300, 64, 64, 0, 4),
    (1, 2, 2, 1000, 1000, 128, 100, 0, 1),
    (1, 2, 2, 1000, 1000, 32, 0, 0, 3),            # a window of one key
    (1, 2, 1, 900, 900, 128, 127, 0, 128),         # sinks end with a tile
    (1, 2, 1, 900, 900, 64, 255, 0, 129),          # and one key later
    (2, 4, 2, 777, 1031, 64, 200, 0, 130),
    (1, 4, 1, 640, 1500, 128, 60, 40, 300),        # keys right of the query too
    (1, 2, 2, 900, 300, 128, 50, 0, 20),           # first 600 rows see nothing
    (1, 2, 2, 400, 1300, 32, 30, -1, 9),           # no right bound
    (1, 2, 2, 1, 1, 128, 0, 0, 1),
    (1, 2, 2, 1, 900, 64, 10, 0, 4),               # one query
    (1, 2, 2, 500, 500, 64, 20, 0, 5000),          # more sinks than keys: causal
    (1, 2, 2, 300, 300, 64, -1, 0, 7),             # open window: sinks change nothing
    (1, 40, 8, 2000, 2000, 128, 300, 0, 4),        # fills the GPU: no key split
    (1, 40, 40, 1300, 1300, 64, 129, 0, 70),
    (1, 2, 1, 700, 3000, 128, 30, 0, 2900),        # so many sink tiles that none is shared
    (2, 20, 20, 640, 1100, 64, 64, 0, 1099),       # one part per sink tile
]


def _ids(c):
    return "B{}H{}kv{}_q{}k{}_d{}_w{}_{}_s{}".format(*c)


def _draw(shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def _inputs(c, dtype=torch.bfloat16):
    B, H, Hkv, nq, nk, d = c[:6]
    return (_draw((B, H, nq, d), 1, dtype), _draw((B, Hkv, nk, d), 2, dtype),
            _draw((B, Hkv, nk, d), 3, dtype), _draw((B, H, nq, d), 4, dtype))


def _close(got, want, bound, what):
    off = np.abs(ref.f64(got) - want) - bound
    assert off.max() <= 0, (what, float(off.max()), np.unravel_index(off.argmax(), off.shape))


def _close_lse(lse, want, tol):
    got = ref.f64(lse)
    none = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), none)
    assert np.abs(got[~none] - want[~none]).max(initial=0.0) <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_forward(cuda_device, case):
    q, k, v, _ = _inputs(case)
    vis = ref.visible(*case[3:5], *case[6:])
    o, lse = ea.forward(q.cuda(), k.cuda(), v.cuda(), window=case[6:8], sinks=case[8])
    ro, rlse, bound = ref.attention(*(ref.f64(x) for x in (q, k, v)), vis, ref.default_scale(case[5]))
    assert ea.device_status() == ea.ATTN_OK
    _close(o, ro, bound, "o")
    _close_lse(lse, rlse, TOL_LSE["bf16"])


@pytest.mark.gpu
@pytest.mark.parametrize("case", [c for c in CASES if c[1] < 40], ids=_ids)
def test_forward_fp32(cuda_device, case):
    q, k, v, _ = _inputs(case, torch.float32)
    vis = ref.visible(*case[3:5], *case[6:])
    o, lse = ea.forward(q.cuda(), k.cuda(), v.cuda(), window=case[6:8], sinks=case[8])
    ro, rlse, _ = ref.attention(*(ref.f64(x) for x in (q, k, v)), vis, ref.default_scale(case[5]))
    assert ea.device_status() == ea.ATTN_OK
    _close(o, ro, 1e-5, "o")
    _close_lse(lse, rlse, TOL_LSE["fp32"])


@pytest.mark.gpu
@pytest.mark.parametrize("case", [c for c in CASES if c[5] > 32], ids=_ids)
def test_forward_fp8(cuda_device, case):
    # each weight is rounded to E4M3: by 2^-4 of itself at most, or by 2^-10 where it is below 2^-6 of a
    # reference that is at most the row's largest (so by 2^-10 max(p) of the normalised weights); scores
    # are exact in fp32, so LSE keeps the bf16 path's bound
    q, k, v, _ = (x.to(torch.float8_e4m3fn) for x in _inputs(case, torch.float32))
    vis = ref.visible(*case[3:5], *case[6:])
    o, lse = ea.forward_fp8(q.cuda(), k.cuda(), v.cuda(), v_descale=0.5, window=case[6:8], sinks=case[8])
    assert ea.device_status() == ea.ATTN_OK
    q, k, v = (ref.f64(x.float()) for x in (q, k, v))
    v = v * 0.5
    p, rlse = ref.probabilities(q, k, vis, ref.default_scale(case[5]))
    ve = ref._expand(v, case[1])
    ro = p @ ve
    bound = 2.0 ** -4 * (p @ np.abs(ve)) + 2.0 ** -10 * p.max(-1, keepdims=True) * (vis.astype(float) @ np.abs(ve))
    _close(o, ro, (bound + ref.BF16 * np.abs(ro)) * 1.02 + 1e-6, "o")
    _close_lse(lse, rlse, TOL_LSE["bf16"])


@pytest.mark.gpu
@pytest.mark.parametrize("det", [False, True])
@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_backward(cuda_device, case, det):
    q, k, v, do = _inputs(case)
    nq, nk = case[3:5]
    vis = ref.visible(nq, nk, *case[6:])
    dev = [x.cuda() for x in (q, k, v)]
    kw = dict(window=case[6:8], sinks=case[8])
    o, lse = ea.forward(*dev, **kw)
    need = ea.attn_bwd_sink_workspace_bytes(*case[:6], *case[6:], int(det))
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")     # NaNs everywhere
    got = ea.backward(*dev, o, do.cuda(), lse, deterministic=det, workspace=ws[:need], **kw)
    assert ea.device_status() == ea.ATTN_OK
    assert bool((ws[need:] == 255).all())
    want, bounds = ref.gradients(*(ref.f64(x) for x in (q, k, v, do)), vis, ref.default_scale(case[5]))
    for name, g, w, b in zip(("dq", "dk", "dv"), got, want, bounds):
        _close(g, w, b, name)
    for g, dead in ((got[0], ~vis.any(1)), (got[1], ~vis.any(0)), (got[2], ~vis.any(0))):
        assert not torch.any(g[:, :, torch.from_numpy(dead).cuda()])
    if det:
        again = ea.backward(*dev, o, do.cuda(), lse, deterministic=True, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
def test_gradient_against_differences(cuda_device):
    # directional differences of the fp32 forward: f(x + h u) - f(x - h u) over 2 h. fp32 sums of
    # ~2e5 terms are off by ~1e-3 at most, /2h = 1e-2 -> 0.1; bf16 gradients add 2^-8 of |g||u|
    case = (1, 2, 1, 400, 400, 64, 50, 0, 3)
    q, k, v, do = (x.cuda() for x in _inputs(case))
    kw = dict(window=(50, 0), sinks=3)
    o, lse = ea.forward(q, k, v, **kw)
    grads = ea.backward(q, k, v, o, do, lse, **kw)
    x = [q.float(), k.float(), v.float()]
    f = lambda a: (ea.forward(*a, **kw)[0].double() * do.double()).sum()     # noqa: E731
    h = 5e-2
    for n, g in enumerate(grads):
        u = _draw(x[n].shape, 11 + n, torch.float32).cuda()
        hi, lo = list(x), list(x)
        hi[n], lo[n] = x[n] + h * u, x[n] - h * u
        slope = float((f(hi) - f(lo)) / (2 * h))
        want = float((g.double() * u.double()).sum())
        size = float((g.double() * u.double()).square().sum().sqrt())
        # the second-order term of the differences is h^2 f'''/6, small against size
        assert abs(slope - want) <= 0.05 * size + 0.1, (n, slope, want, size)


@pytest.mark.gpu
def test_no_sinks_and_open_window_are_the_other_entries(cuda_device):
    q, k, v, _ = (x.cuda() for x in _inputs((1, 2, 2, 700, 700, 128)))
    for wl in (-1, 90):
        a = ea.forward(q, k, v, window=(wl, 0))
        o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        p = [ctypes.c_void_p(t.data_ptr()) for t in (q, k, v, o, lse)]
        n = 0 if wl >= 0 else 5
        rc = ea.attn_fwd_sink(*p, 1, 2, 2, 700, 700, 128, 128 ** -0.5, wl, 0, n, ea.ATTN_BF16,
                              ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert rc == ea.ATTN_OK
        assert torch.equal(a[0], o) and torch.equal(a[1], lse)


@pytest.mark.gpu
def test_graph_and_another_stream(cuda_device):
    case = (1, 4, 2, 600, 600, 128, 80, 0, 5)
    q, k, v, do = (x.cuda() for x in _inputs(case))
    kw = dict(window=(80, 0), sinks=5)
    o, lse = ea.forward(q, k, v, **kw)
    want = (o, lse) + ea.backward(q, k, v, o, do, lse, deterministic=True, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        go, gl = ea.forward(q, k, v, **kw)
        got = (go, gl) + ea.backward(q, k, v, go, do, gl, deterministic=True, **kw)
    for _ in range(2):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


FAKE = 1 << 20


@pytest.mark.parametrize("kw,code", [
    (dict(ns=-1), ea.ATTN_ERR_INVALID), (dict(nk=0), ea.ATTN_ERR_INVALID),
    (dict(H=3, Hkv=2), ea.ATTN_ERR_INVALID), (dict(d=96), ea.ATTN_ERR_UNSUPPORTED),
    (dict(q=0), ea.ATTN_ERR_INVALID), (dict(q=FAKE + 8), ea.ATTN_ERR_INVALID),
    (dict(scale=0.0), ea.ATTN_ERR_INVALID), (dict(dtype=9), ea.ATTN_ERR_UNSUPPORTED)])
def test_refusals(kw, code):
    a = dict(q=FAKE, H=2, Hkv=2, nk=100, d=64, scale=0.1, ns=4, dtype=ea.ATTN_BF16)
    a.update(kw)
    p = lambda x=FAKE: ctypes.c_void_p(x)                                # noqa: E731
    assert ea.attn_fwd_sink(p(a["q"]), p(), p(), p(), p(), 1, a["H"], a["Hkv"], 100, a["nk"], a["d"],
                            a["scale"], 10, 0, a["ns"], a["dtype"], None) == code
    if "dtype" not in kw:
        assert ea.attn_fwd_fp8_sink(p(a["q"]), p(), p(), p(), p(), 1, a["H"], a["Hkv"], 100, a["nk"], a["d"],
                                    a["scale"], 10, 0, a["ns"], 1.0, 1.0, 1.0, None) == code
    assert ea.attn_bwd_sink(p(a["q"]), *[p()] * 8, 1, a["H"], a["Hkv"], 100, a["nk"], a["d"],
                            a["scale"], 10, 0, a["ns"], a["dtype"], 0, p(), 1 << 40, None) == code


def test_workspace_of_many_sinks_stays_bounded():
    # partials: at most 8 x 148 + one per sink tile of 128 rows, K and V, fp32; none without parts
    for ns in (1, 4000, 60000, 131071, 131072):
        extra = (ea.attn_bwd_sink_workspace_bytes(1, 8, 8, 131072, 131072, 128, 1024, 0, ns, 0)
                 - ea.attn_bwd_workspace_bytes(1, 8, 131072, 128, 0))
        tiles = 8 * -(-ns // 128)
        assert 0 <= extra <= (8 * 148 + tiles) * 2 * 128 * 128 * 4
        assert (extra == 0) == (ns >= 131072 or tiles >= 8 * 148)


def test_backward_refuses_a_small_workspace_and_fp32():
    p = ctypes.c_void_p(FAKE)
    need = ea.attn_bwd_sink_workspace_bytes(1, 2, 2, 5000, 5000, 64, 10, 0, 4, 0)
    assert need > ea.attn_bwd_workspace_bytes(1, 2, 5000, 64, 0)
    call = lambda dt, n: ea.attn_bwd_sink(*[p] * 9, 1, 2, 2, 5000, 5000, 64, 0.1, 10, 0, 4, dt, 0, p,  # noqa: E731
                                          n, None)
    assert call(ea.ATTN_BF16, need - 1) == ea.ATTN_ERR_WORKSPACE
    assert call(ea.ATTN_FP32, need) == ea.ATTN_ERR_UNSUPPORTED
    assert ea.attn_bwd_sink_workspace_bytes(1, 2, 2, 5000, 5000, 64, 10, 0, -1, 0) == 0


@pytest.mark.parametrize("bad", [-1, 1.5, 1 << 31])
def test_binding_refuses_bad_sinks(bad):
    x = torch.zeros((1, 1, 8, 32), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ea.forward(x, x, x, window=(2, 0), sinks=bad)
