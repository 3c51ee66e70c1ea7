"""Host-side check of the bookkeeping of a warp's ring of copies (Kv4Ring of the CUDA library's kv4.h),
compiled for the CPU: after waits that ran out, in whatever segments of a run, the stages and phases it
gives are exactly those of the copies that were never seen to land."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HDR_DIR = os.path.join(ROOT, "exact_attention_138_b200", "csrc")

SHIM = r"""
#include "kv4.h"
// One warp's run as the kernel goes through it: steps[s] steps in segment s; wait w ends with the copy landed
// if lands[w], else it runs out and ends its segment. out: number of copies started and landed, then (stage, phase)
// of those that are waited for at the end, out[2] of them. Returns how many waits there were.
template <int ST>
static int go(const int* steps, int segments, const int* lands, int* out) {
    attn::Kv4Ring<ST> r;
    int total = 0, started = 0, landed = 0, waits = 0;
    for (int s = 0; s < segments; ++s) total += steps[s];
    auto fetch = [&] {
        if (started == total) return;
        if (r.fill != started++ % ST) waits = -1000;
        r.start();
    };
    for (int s = 0; s < ST; ++s) fetch();
    for (int s = 0; s < segments; ++s)
        for (int i = 0; i < steps[s]; ++i) {
            if (r.use != landed % ST || r.phase != (unsigned)(landed / ST % 2)) return -1;
            if (!lands[waits++]) break;
            r.take();
            ++landed;
            fetch();
        }
    out[0] = started, out[1] = landed, out[2] = 0;
    for (; r.taken < r.issued; r.take()) {
        out[3 + 2 * out[2]] = r.use;
        out[4 + 2 * out[2]++] = (int)r.phase;
    }
    return waits;
}
extern "C" int run(const int* steps, int segments, int stages, const int* lands, int* out) {
    return stages == 3 ? go<3>(steps, segments, lands, out) : stages == 4 ? go<4>(steps, segments, lands, out)
                                                                          : go<8>(steps, segments, lands, out);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    cuda_inc = "/usr/local/cuda/include"
    if gxx is None or not os.path.isdir(cuda_inc):
        pytest.skip("g++ or the CUDA headers are not available")
    d = tmp_path_factory.mktemp("copies")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-I", HDR_DIR, "-I", cuda_inc,
                    str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def test_copies_in_flight_after_waits_that_ran_out(lib):
    rng = random.Random(2)
    whole = 0
    for _ in range(3000):
        steps = [rng.randrange(0, 6) for _ in range(rng.randrange(1, 9))]
        stages, total = rng.choice([3, 4, 8]), sum(steps)
        lands = [int(rng.random() > rng.choice([0, 0.02, 0.5])) for _ in range(total + 1)]
        out = (ctypes.c_int * 20)()
        ints = lambda x: (ctypes.c_int * len(x))(*x)                     # noqa: E731
        assert lib.run(ints(steps), len(steps), stages, ints(lands), out) >= 0
        started, landed, n = out[:3]
        assert started == min(total, landed + stages) and n == started - landed
        assert list(out[3:3 + 2 * n]) == [x for i in range(landed, started) for x in (i % stages, i // stages % 2)]
        whole += n == 0
    assert 300 < whole < 2700
