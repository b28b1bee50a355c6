"""How the convolution's launches cut up sequences and channels (csrc/conv_plan.h), up to the largest sizes that a call may
have: on the CPU, by the same header; and one gradient whose last strip ends past 2^31."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest
import torch

import test_neural_memory_gb300 as ttm

CSRC = os.path.join(os.path.dirname(os.path.abspath(ttm.__file__)), "csrc")
MOST_T, MOST = 2 ** 31 - 8193, 2 ** 31 - 1
SOURCE = """
#include "conv_plan.h"
extern "C" int strip_end(int T, int t0, int strip) { return ttm::conv_strip_end(T, t0, strip); }
extern "C" void fwd(int N, int T, int groups, int one, long long* out) {
    const ttm::ConvFwdPlan p = ttm::conv_fwd_plan(N, T, groups, one != 0);
    out[0] = p.strip; out[1] = p.strips; out[2] = p.blocks;
}
extern "C" void bwd(int N, int T, int C, int groups, int per_sm, long long* out) {
    const ttm::ConvBwdPlan p = ttm::conv_bwd_plan(N, T, C, groups, per_sm);
    out[0] = p.bx; out[1] = p.by; out[2] = p.across; out[3] = p.rows; out[4] = p.strip; out[5] = p.strips;
}
extern "C" int most_rows(int C) { return ttm::conv_most_rows(C); }
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
    return lib, lambda *a: call("fwd", 3, *a), lambda *a: call("bwd", 6, *a)


def sizes():
    """(N, T, C): the borders of 31 bits, where sums of two sizes wrap, and others between."""
    rng = random.Random(1)
    spread = lambda most: int(round(2 ** rng.uniform(0, 31))) % most + 1  # noqa: E731
    edges = [1, 2, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 1, 1_431_655_765, 1_500_000_000, MOST_T - 300_000, MOST_T - 20_000, MOST_T]
    out = [(1, t, c) for t in edges for c in (1, 7, 8, 768)]
    out += [(n, 5, c) for n, c in ((1, MOST), (1, MOST - 1), (1, MOST - 31), (1, MOST - 7), (MOST, 1), (2 ** 15, 2 ** 15), (3, MOST // 3))]
    out += [(77824, t, 1) for t in edges] + [(4, t, 40000) for t in edges]
    while len(out) < 3000:
        n, t, c = spread(MOST), spread(MOST_T), spread(MOST)
        if n * c <= MOST:
            out.append((n, t, c))
    return out


def strips_cover(lib, T, strip, strips):
    assert strip >= 1 and 1 <= strips <= MOST and (strips - 1) * strip < T <= strips * strip
    last = (strips - 1) * strip
    for t0 in {0, last // strip // 2 * strip, last}:
        assert lib.strip_end(T, t0, strip) == min(T, t0 + strip)


def test_forward_and_step(plan):
    lib, fwd, _ = plan
    for N, T, C in sizes():
        for V in (1, 2, 4, 8):
            if C % V:
                continue
            for one in (0, 1):
                strip, strips, blocks = fwd(N, T, C // V, one)
                strips_cover(lib, T, strip, strips)
                # a step's state is updated in place: no other strip may read it
                assert strips == 1 if one else 8 <= strip <= 128
                assert (blocks - 1) * 128 < N * (C // V) * strips <= blocks * 128


def test_gradient(plan):
    lib, _, bwd = plan
    for N, T, C in sizes():
        for V in (1, 2, 4):
            if C % V:
                continue
            for per_sm in (3, 4):
                bx, by, across, rows, strip, strips = bwd(N, T, C, C // V, per_sm)
                strips_cover(lib, T, strip, strips)
                assert bx * by == 128 and (across - 1) * bx < C // V <= across * bx < 2 ** 32 // V
                assert 1 <= rows <= lib.most_rows(C) <= 608 and strip % 4 == 0 and strip >= 16


@pytest.mark.gpu
@pytest.mark.parametrize("K", [4, 7])
def test_a_sequence_of_nearly_2_31_tokens(K):
    """One channel; all but the last rows are zero.  The last ones' gradient is that of a call on them alone, bit for bit, as
    every row sums its own taps; sums over the tokens by their order, 2^-24 of the sum of sizes a term."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    T, tail = MOST_T, 60000
    r = torch.Generator(device="cuda").manual_seed(K)
    rand = lambda *s: torch.randn(s, generator=r, device="cuda")  # noqa: E731
    x, dy = (torch.zeros((1, T, 1), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for t in (x, dy):
        t[:, -tail - 8:] = rand(1, tail + 8, 1).to(t.dtype)
    dy[:, :-tail] = 0
    w, ds = rand(1, K), rand(1, K - 1, 1).to(x.dtype)
    g = ttm.causal_conv_bwd(dy, x, w, dstate=ds)
    last = ttm.causal_conv_bwd(dy[:, -tail:].clone(), x[:, -tail:].clone(), w, dstate=ds,
                               state0=x[:, -tail - K + 1:-tail].clone())
    assert torch.equal(g["dx"][:, -tail:], last["dx"])
    assert torch.equal(g["dx"][:, -tail - K + 1:-tail], last["dstate0"]) and not g["dx"][:, :-tail - K + 1].any()
    size = dy[:, -tail:].double().abs().sum() * x.abs().max() * 1.1     # SiLU's slope is at most 1.1
    assert float((g["dw"] - last["dw"]).abs().max()) <= float(size) * tail * 2.0 ** -24
    y, state = ttm.causal_conv_fwd(x, w)
    y2, state2 = ttm.causal_conv_fwd(x[:, -tail:].clone(), w, state0=x[:, -tail - K + 1:-tail].clone())
    assert torch.equal(y[:, -tail:], y2) and torch.equal(state, state2)
    assert ttm.device_status() == ttm.OK
