"""Calls on another stream than the current one: the outputs and workspaces that a call makes must not be
memory that the current stream still uses, nor be handed out on the current stream while the call runs. Shown
on the addresses that reach the C entry points, with nothing launched, and on the results."""
import ctypes

import pytest
import torch

import exact_attention_138_b200 as ea

LAUNCHES = ["attn_fwd", "attn_fwd_ex", "attn_fwd_gqa", "attn_fwd_sink", "attn_fwd_fp8_sink", "attn_bwd",
            "attn_bwd_ex", "attn_bwd_gqa", "attn_bwd_sink", "attn_bwd_prepare", "attn_bwd_accumulate",
            "attn_bwd_finish", "attn_kv4_gather", "attn_kv4_attend", "attn_pages_reserve", "attn_pages_fork",
            "attn_pages_compact"]


def _randn(*shape, seed=0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=g).bfloat16().cuda()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def data():
    d = dict(q=_randn(1, 4, 700, 128), k=_randn(1, 4, 700, 128, seed=1), v=_randn(1, 4, 700, 128, seed=2),
             k2=_randn(1, 2, 700, 128, seed=3), k9=_randn(1, 4, 900, 128), do=_randn(1, 4, 700, 128, seed=4))
    d["o"], d["lse"] = ea.forward(d["q"], d["k"], d["v"])
    d["f8"] = d["q"].to(torch.float8_e4m3fn)
    d["pool"], d["table"] = ea.kv4_pool(60, 4, 16, 128), torch.arange(60, dtype=torch.int32, device="cuda")[None]
    ea.kv4_append(d["pool"], d["table"], _i32([0]), d["k"], d["v"])
    d["lens"], d["zero"], d["lse2"] = _i32([700]), _i32([0]), d["lse"].clone()
    d["q1"] = _randn(1, 8, 1, 128)
    d["pages"] = [torch.full((4, 200), -1, dtype=torch.int32, device="cuda"), _i32([0] * 4), _i32([0] * 600)]
    d["rows"], d["counts"] = _i32([1, 2]), _i32([70, 5])
    torch.cuda.synchronize()
    return d


def _parts(x, stream):
    s = ea.BackwardSum(x["o"], x["do"], x["lse"], deterministic=True, stream=stream)
    dk, dv = x["dk32"], x["dv32"]
    s.add(x["q"], x["k"], x["v"], x["do"], dk, dv, stream=stream)
    return s.finish(stream=stream)


W = dict(window=(100, 0), sinks=4)
CALLS = {
    "forward": lambda x, s: ea.forward(x["q"], x["k"], x["v"], causal=True, stream=s),
    "forward, shared heads": lambda x, s: ea.forward(x["q"], x["k2"], x["k2"], stream=s),
    "forward, more keys": lambda x, s: ea.forward(x["q"], x["k9"], x["k9"], stream=s),
    "forward, sinks": lambda x, s: ea.forward(x["q"], x["k"], x["v"], stream=s, **W),
    "forward, lse given": lambda x, s: ea.forward(x["q"], x["k"], x["v"], lse=x["lse2"], stream=s)[0],
    "forward_fp8": lambda x, s: ea.forward_fp8(x["f8"], x["f8"], x["f8"], stream=s, **W),
    "backward": lambda x, s: ea.backward(x["q"], x["k"], x["v"], x["o"], x["do"], x["lse"], stream=s,
                                         deterministic=True),
    "backward, sinks": lambda x, s: ea.backward(x["q"], x["k"], x["v"], x["o"], x["do"], x["lse"], stream=s,
                                                deterministic=True, **W),
    "BackwardSum": _parts,
    "kv4_gather": lambda x, s: ea.kv4_gather(x["pool"], x["table"], x["zero"], 700, 128, stream=s),
    "kv4_attend": lambda x, s: ea.kv4_attend(x["q1"], x["pool"], x["table"], x["lens"], stream=s),
    "pages_reserve": lambda x, s: ea.pages_reserve(*x["pages"], 16, x["rows"], x["counts"], stream=s),
    "pages_fork": lambda x, s: ea.pages_fork(*x["pages"], 16, x["rows"], x["counts"], stream=s),
    "pages_compact": lambda x, s: ea.pages_compact(x["pages"][0], x["pages"][2], stream=s),
}


class Addresses:
    """Stands in for the C entry points: keeps the addresses that a call passes, and launches nothing."""

    def __init__(self, monkeypatch, data):
        flat = [t for v in data.values() for t in (v if isinstance(v, list) else [v])]
        self.inputs = {t.data_ptr() for t in flat}
        self.seen = set()
        for name in LAUNCHES:
            monkeypatch.setattr(ea._lib, name, self._call)

    def _call(self, *args):
        for a in args:
            p = a.value if isinstance(a, ctypes.c_void_p) else a
            if isinstance(p, int) and p > 1 << 32 and p not in self.inputs:
                self.seen.add(p)
        return 0

    def of(self, call):
        """The addresses of what call() makes; its results are dropped."""
        self.seen = set()
        call()
        return self.seen


def _fresh(data):
    data["dk32"], data["dv32"] = (torch.zeros((1, 4, 700, 128), device="cuda") for _ in range(2))
    return data


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_made_memory_is_not_shared_with_the_current_stream(cuda_device, data, monkeypatch, name):
    call = CALLS[name]
    at = Addresses(monkeypatch, _fresh(data))
    x = data
    s = torch.cuda.Stream()
    here = torch.cuda.current_stream()
    # the current stream is still at work on blocks that were dropped: not for the other stream's call
    torch.cuda._sleep(20_000_000)
    mine = at.of(lambda: call(x, None))
    theirs = at.of(lambda: call(x, s))
    assert mine and theirs and not mine & theirs - {s.cuda_stream, here.cuda_stream}
    torch.cuda.synchronize()
    # the other stream is still at work: what its call made is not handed out here
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    theirs = at.of(lambda: call(x, s))
    mine = at.of(lambda: call(x, None))
    assert not mine & theirs - {s.cuda_stream, here.cuda_stream}
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_results_on_a_busy_stream(cuda_device, data, name):
    flat = lambda r: list(r) if isinstance(r, (tuple, list)) else [r]        # noqa: E731
    state = [t.clone() for t in data["pages"]]
    if name in ("pages_fork", "pages_compact"):
        ea.pages_reserve(*state, 16, _i32([0, 3]), _i32([100, 33]))
    saved = [t.clone() for t in state]

    def fresh():
        x = dict(_fresh(data))
        for t, u in zip(state, saved):
            t.copy_(u)
        x["pages"] = state
        if name == "pages_fork":
            x["rows"], x["counts"] = _i32([0, 0]), _i32([1, 2])
        return x
    x = fresh()
    want = [t.clone() for t in flat(CALLS[name](x, None))] + [t.clone() for t in state + [x["dk32"], x["dv32"]]]
    ea.device_status()
    s = torch.cuda.Stream()
    x = fresh()
    torch.cuda._sleep(4_000_000)                     # work of the current stream on blocks of these sizes
    junk = [torch.full_like(t, -1) for t in want]
    del junk
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    got = flat(CALLS[name](x, s))
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            for n in (1 << 9, 1 << 12, 1 << 16, 1 << 20, 1 << 21, 1 << 22, 3 << 20, 1 << 24) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(s)
    got = got + state + [x["dk32"], x["dv32"]]
    torch.cuda.synchronize()
    del junk
    assert ea.device_status() in (ea.ATTN_OK, ea.ATTN_ERR_PAGES)
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["forward, sinks", "backward, sinks", "kv4_attend", "kv4_gather", "BackwardSum"])
def test_a_branch_of_a_captured_graph(cuda_device, data, name):
    # the call runs on a stream that joins the capture, while the capturing stream makes memory of its own
    flat = lambda r: list(r) if isinstance(r, (tuple, list)) else [r]        # noqa: E731
    x = _fresh(data)
    want = [t.clone() for t in flat(CALLS[name](x, None))]
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        got = flat(CALLS[name](x, side))
        other = [torch.full_like(t, 3) for t in want for _ in range(3)]
        main.wait_stream(side)
        back = [t.clone() for t in got]
        del got
    for _ in range(2):
        for t in back + other:
            t.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b, w) for b, w in zip(back, want))
        assert all(bool((t == 3).all()) for t in other)
