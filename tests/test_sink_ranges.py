"""Host-side check of the tile arithmetic of windows with sinks (MaskSpec::ns in the CUDA library's
kernels.h), compiled for the CPU and compared with brute force over the visibility rule: the query
tiles that the backward pass gives each key tile, and how many key tiles above one meet a query tile
(the order of the deterministic mode). Also the fp64 reference of the GPU tests against differences."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import stream_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HDR_DIR = os.path.join(ROOT, "exact_attention_138_b200", "csrc")

SHIM = r"""
#include "kernels.h"
using namespace attn;
static MaskSpec spec(const int* m) {
    return MaskSpec{m[0], m[1], m[2], m[3], (long long)m[1] - m[0], m[4]};
}
extern "C" void qtiles(const int* m, int j, int bk, int bq, int* out) {
    query_tiles_of_key_tile(spec(m), j, bk, bq, out[0], out[1]);
}
extern "C" int above(const int* m, long long a, int bq, int bk, int j) {
    return key_tiles_above(spec(m), a, bq, bk, j);
}
extern "C" int sinks(const int* m, int bk) { return sink_tiles(spec(m), bk); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    cuda_inc = "/usr/local/cuda/include"
    if gxx is None or not os.path.isdir(cuda_inc):
        pytest.skip("g++ or the CUDA headers are not available")
    d = tmp_path_factory.mktemp("sinkshim")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-I", HDR_DIR, "-I", cuda_inc,
                    str(src), "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    ip = ctypes.POINTER(ctypes.c_int)
    L.qtiles.argtypes = [ip, ctypes.c_int, ctypes.c_int, ctypes.c_int, ip]
    L.above.argtypes = [ip, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    L.sinks.argtypes = [ip, ctypes.c_int]
    return L


# (nq, nk, wl, wr, ns)
CASES = [(700, 700, 64, 0, 4), (700, 700, 0, 0, 1), (700, 700, 130, 0, 128), (513, 900, 100, 30, 300),
         (900, 513, 20, 0, 7), (900, 513, 0, 5, 600), (300, 2000, 200, -1, 4), (1, 900, 10, 0, 2),
         (400, 1, 3, 0, 1), (640, 640, 127, 0, 129), (2000, 300, 50, 100, 200)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("bq", [64, 128])
def test_tiles_that_meet(lib, case, bq):
    nq, nk, wl, wr, ns = case
    m = (ctypes.c_int * 5)(*case)
    vis = ref.visible(nq, nk, wl, wr, ns)
    nqt, nkt = -(-nq // bq), -(-nk // 128)
    truth = np.array([[vis[t * bq:(t + 1) * bq, j * 128:(j + 1) * 128].any() for j in range(nkt)]
                      for t in range(nqt)])
    meets = np.zeros_like(truth)
    out = (ctypes.c_int * 2)()
    for j in range(nkt):
        lib.qtiles(m, j, 128, bq, out)
        meets[out[0]:out[1], j] = True
    assert lib.sinks(m, 128) == -(-min(ns, nk) // 128)
    assert not np.any(truth & ~meets)                # nothing visible is left out
    # a pair beyond the truth is a masked tile; the counts below must follow what is visited
    for t in range(nqt):
        js = np.nonzero(meets[t])[0]
        for x, j in enumerate(js):
            assert lib.above(m, t * bq, bq, 128, int(j)) == len(js) - 1 - x
    assert np.array_equal(meets, truth)


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(3)
    q, do = rng.normal(size=(1, 4, 9, 8)), rng.normal(size=(1, 4, 9, 8))
    k, v = rng.normal(size=(1, 2, 13, 8)), rng.normal(size=(1, 2, 13, 8))
    vis = ref.visible(9, 13, 3, 0, 2)
    grads, _ = ref.gradients(q, k, v, do, vis, 0.3)
    f = lambda *a: (ref.attention(*a, vis, 0.3)[0] * do).sum()          # noqa: E731
    h = 1e-5
    for n, g in enumerate(grads):
        x = [q, k, v]
        for _ in range(6):
            at = tuple(rng.integers(0, s) for s in x[n].shape)
            e = np.zeros_like(x[n])
            e[at] = h
            hi, lo = list(x), list(x)
            hi[n], lo[n] = x[n] + e, x[n] - e
            assert abs((f(*hi) - f(*lo)) / (2 * h) - g[at]) < 1e-7
