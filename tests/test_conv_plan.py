"""How the convolution's launches cut up sequences and channels (csrc/conv_plan.h), up to the largest sizes that a call may
have, on the CPU, by the same header."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

import test_neural_memory_gb300 as ttm

CSRC = os.path.join(os.path.dirname(os.path.abspath(ttm.__file__)), "csrc")
MOST_T, MOST = 2 ** 31 - 8193, 2 ** 31 - 1
SOURCE = """
#include "conv_plan.h"
extern "C" void fwd(int N, int T, int groups, int one, long long* out) {
    const ttm::ConvFwdPlan p = ttm::conv_fwd_plan(N, T, groups, one != 0);
    out[0] = p.strip; out[1] = p.strips; out[2] = p.blocks;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-shared", "-fPIC", f"-I{CSRC}", str(at / "plan.cpp"), "-o",
                    str(at / "plan.so")], check=True)
    lib = ctypes.CDLL(str(at / "plan.so"))

    def call(name, n, *args):
        out = (ctypes.c_longlong * n)()
        getattr(lib, name)(*[ctypes.c_int(a) for a in args], out)
        return list(out)
    return lambda *a: call("fwd", 3, *a)


def sizes():
    """(N, T, C): the borders of 31 bits, where sums of two sizes wrap, and others between."""
    rng = random.Random(1)
    spread = lambda most: int(round(2 ** rng.uniform(0, 31))) % most + 1  # noqa: E731
    edges = [1, 2, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 1, 1_431_655_765, 1_500_000_000, MOST_T - 300_000, MOST_T - 20_000, MOST_T]
    out = [(1, t, c) for t in edges for c in (1, 7, 8, 768)]
    out += [(n, 5, c) for n, c in ((MOST, 1), (2 ** 15, 2 ** 15), (3, MOST // 3))]
    out += [(77824, t, 1) for t in edges] + [(4, t, 40000) for t in edges]
    while len(out) < 3000:
        n, t, c = spread(MOST), spread(MOST_T), spread(MOST)
        if n * c <= MOST and c < MOST - 63:
            out.append((n, t, c))
    return out


def strips_cover(T, strip, strips):
    assert strip >= 1 and 1 <= strips <= MOST and (strips - 1) * strip < T <= strips * strip


def test_forward_and_step(plan):
    fwd = plan
    for N, T, C in sizes():
        for V in (1, 2, 4, 8):
            if C % V:
                continue
            for one in (0, 1):
                strip, strips, blocks = fwd(N, T, C // V, one)
                strips_cover(T, strip, strips)
                # a step's state is updated in place: no other strip may read it
                assert strips == 1 if one else 8 <= strip <= 128
                assert (blocks - 1) * 128 < N * (C // V) * strips <= blocks * 128
