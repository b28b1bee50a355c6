"""The kept answers of the cluster query (csrc/known_clusters.h), on the CPU by the same header: one per device and width, none
of a query that failed."""
import ctypes
import os
import shutil
import subprocess

import pytest

import test_neural_memory_gb300 as ttm

CSRC = os.path.join(os.path.dirname(os.path.abspath(ttm.__file__)), "csrc")
SOURCE = """
#include "known_clusters.h"
static ttm::KnownClusters known;
// (*n, asked): the answer and how often the query was put, which gives `answer` and the code `error`
extern "C" int get(int device, int width, int answer, int error, int* n, int* asked) {
    *asked = 0;
    return known.get(device, width, *n, [&](int* out) { ++*asked; *out = answer; return error; });
}
"""


@pytest.fixture
def get(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    (tmp_path / "known.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", str(tmp_path / "known.cpp"), "-o",
                    str(tmp_path / "known.so")], check=True)
    lib = ctypes.CDLL(str(tmp_path / "known.so"))

    def call(device, width, answer, error=0):
        n, asked = ctypes.c_int(), ctypes.c_int()
        code = lib.get(device, width, answer, error, ctypes.byref(n), ctypes.byref(asked))
        return code, n.value, asked.value
    return call


def test_one_answer_per_device_and_width(get):
    assert get(0, 2, 70) == (0, 70, 1) and get(0, 2, 5) == (0, 70, 0)
    assert get(1, 2, 66) == (0, 66, 1) and get(1, 2, 70) == (0, 66, 0) and get(0, 2, 1) == (0, 70, 0)
    assert get(0, 8, 16) == (0, 16, 1) and get(0, 8, 1) == (0, 16, 0)
    assert get(0, 4, 0) == (0, 0, 1) and get(0, 4, 3) == (0, 0, 0)      # none fits: an answer too


def test_a_failure_is_passed_on_and_not_kept(get):
    assert get(3, 2, 70, error=9)[0] == 9 and get(3, 2, 70, error=9)[2] == 1
    assert get(3, 2, 70) == (0, 70, 1) and get(3, 2, 1, error=9) == (0, 70, 0)


def test_places_that_are_not_kept(get):
    for device, width in ((64, 2), (1000, 2), (0, 9)):
        assert get(device, width, 7) == (0, 7, 1) and get(device, width, 8) == (0, 8, 1)
