"""The steps that attention with a window takes, on the host: every token that a row sees is in one of them, none is read
that no row sees, and those said to be seen whole by all rows are."""

import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "affine_quantized_gemm_amd", "csrc")
SOURCE = """
#include "qmm_kv_window.hpp"
extern "C" int pieces(int pos0, int n, int64_t cap, int window, int sinks, int masked, int most, int* real, int* all) {
    const qmm::kv::Window w = qmm::kv::window_of(pos0, n, cap, window, sinks, masked != 0);
    for (int t = 0; t < w.len && t < most; ++t) real[t] = w.real(t);
    *all = w.all;
    return w.len;
}
"""


@pytest.fixture(scope="module")
def pieces(tmp_path_factory):
    d = tmp_path_factory.mktemp("window")
    (d / "w.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "w.cpp"), "-o",
                    str(d / "w.so")], check=True, timeout=60)
    f = ctypes.CDLL(str(d / "w.so")).pieces
    f.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64, *[ctypes.c_int] * 4, ctypes.c_void_p, ctypes.c_void_p]

    def call(pos0, n, cap, window, sinks, masked):
        most = max(0, pos0 + n) + 64
        real, all_seen = np.zeros(most, np.int32), ctypes.c_int(0)
        length = f(pos0, n, cap, window, sinks, int(masked), most, real.ctypes.data, ctypes.byref(all_seen))
        assert 0 <= length <= most
        return real[:length], all_seen.value

    return call


def seen_by(word, pos0, n, length, window, sinks):
    """Positions below `length` that a row sees, of all that it would see."""
    there = [t for t in range(max(0, pos0 + n)) if t < pos0 or word >> (t - pos0) & 1]
    return {t for t in there[-window:] + [t for t in there if t < sinks] if t < length}


def look_at(pieces, pos0, n, cap, window, sinks, masked):
    what = f"pos0={pos0} n={n} cap={cap} window={window} sinks={sinks} masked={masked}"
    real, all_seen = pieces(pos0, n, cap, window, sinks, masked)
    length = max(0, min(pos0 + n, cap))
    # (a mask's words may be any: none, all, each one by itself)
    words = [0, (1 << n) - 1, *(1 << i for i in range(n))] if masked else [(2 << i) - 1 for i in range(n)]
    rows = [seen_by(w, pos0, n, length, window, sinks) for w in words]
    some, every = set().union(*rows), set(real.tolist())
    assert len(every) == len(real) and all(0 <= t < length for t in every), what
    assert some <= every, what
    for t in range(0, len(real), 32):  # whole steps, in place
        step = real[t:t + 32]
        assert step[0] % 32 == 0 and (np.diff(step) == 1).all() and (len(step) == 32 or step[-1] == length - 1), what
        assert some.intersection(step.tolist()), (what, int(step[0]))  # (a page is steps)
    assert all_seen % 32 == 0 and all(set(real[:all_seen].tolist()) <= r for r in rows), what


@pytest.mark.parametrize("masked", [False, True])
def test_pieces_at_ends(pieces, masked):
    """Windows and sinks that end in, at and beside steps, meet, overlap and reach past the sequence or the table."""
    for pos0 in (-3, 0, 1, 31, 32, 33, 200, 255, 256):
        for n in (1, 5, 32, 33):
            for window in (1, 2, 31, 32, 33, 64, 65, 97, 225, 1000, 1 << 30):
                for sinks in (0, 1, 32, 70, 300, 1 << 30):
                    for cap in (1 << 30, 128):
                        look_at(pieces, pos0, n, cap, window, sinks, masked)


def test_pieces_of_any_sizes(pieces):
    g = random.Random(1)
    for _ in range(1000):
        n = g.randint(1, 64)
        look_at(pieces, g.randint(-n, 700), n, g.choice([1 << 30, 32 * g.randint(1, 20)]), int(2 ** g.uniform(0, 10)),
                g.choice([0, g.randint(0, 100)]), g.random() < 0.5)


def test_no_rows_and_no_tokens(pieces):
    for masked in (False, True):
        assert len(pieces(0, 0, 1 << 30, 5, 3, masked)[0]) == 0
        assert len(pieces(-7, 5, 1 << 30, 5, 3, masked)[0]) == 0
        assert len(pieces(40, 5, 0, 5, 3, masked)[0]) == 0
