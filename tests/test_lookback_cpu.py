"""The look-back of the gated recurrence's tiles (csrc/msr_lookback.hpp) on the
CPU: compiled by the host compiler over words that lie in an array, which the
test's pause changes as other workgroups would.  Nothing is launched."""
import ctypes
import shutil
import subprocess
from pathlib import Path

import numpy as np
import pytest

CSRC = Path(__file__).resolve().parents[1] / "retnet_scale_retention_amd" / "csrc"
SOURCE = r"""
#define __device__
#define __forceinline__ inline
#include "msr_lookback.hpp"
using namespace msr;
extern "C" {
uint64_t make_pair(float z, float h) { return pair_word(z, h); }
uint64_t make_state(float p) { return pack(kState, p); }
uint64_t unset() { return pack(kUnset, 0.f); }
float apply_factor(float z, float p) { return apply(z, p); }
// words[0] .. words[n - 1]: the tiles before tile n; poll k makes words[order[k]] the one of later[order[k]]
float look(uint64_t *words, int n, int spins, const uint64_t *later, const int *order, int changes, int *polls) {
    int k = 0;
    *polls = 0;
    return look_back<8>(
        spins, [&](int i) { const int t = n - 1 - i; return words[t > 0 ? t : 0]; },
        [&] {
            ++*polls;
            if (k < changes) words[order[k]] = later[order[k]], ++k;
        });
}
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("lookback")
    (d / "l.cpp").write_text(SOURCE)
    subprocess.run([gxx, "-O1", "-std=c++17", "-Wno-unknown-pragmas", "-shared", "-fPIC", f"-I{CSRC}", str(d / "l.cpp"), "-o",
                    str(d / "l.so")], check=True)
    lib = ctypes.CDLL(str(d / "l.so"))
    f, u, i, p = ctypes.c_float, ctypes.c_uint64, ctypes.c_int, ctypes.c_void_p
    for name, args, res in (("make_pair", [f, f], u), ("make_state", [f], u), ("unset", [], u), ("apply_factor", [f, f], f),
                            ("look", [p, i, i, p, p, i, p], f)):
        getattr(lib, name).argtypes, getattr(lib, name).restype = args, res
    return lib


def factor(f):
    return 1 - f if f >= 0.5 else -f


def look(lib, words, later=(), order=(), spins=50):
    w = np.array(words, np.uint64)
    l, o, polls = np.array(later or [0], np.uint64), np.array(order or [0], np.int32), ctypes.c_int()
    p = lib.look(w.ctypes.data, len(w), spins, l.ctypes.data, o.ctypes.data, len(order), ctypes.byref(polls))
    return np.float32(p), polls.value


def test_factors(lib):
    inf = float("inf")
    for f in (0.75, 0.5, 0.25, 2.0 ** -30):
        assert lib.apply_factor(factor(f), 8.0) == 8 * f
        assert lib.apply_factor(factor(f), inf) == inf and lib.apply_factor(factor(f), -inf) == -inf
        assert np.isnan(lib.apply_factor(factor(f), float("nan")))
    assert lib.apply_factor(-0.0, 8.0) == 0 and np.isnan(lib.apply_factor(-0.0, inf)) and np.isnan(lib.apply_factor(float("nan"), 1.0))
    # a NaN factor or end never looks like a word that is missing or a state
    bits = float(np.array([0xffffffff], np.uint32).view(np.float32)[0])
    assert lib.make_pair(bits, 1.0) >> 32 == 0x7fc00000
    assert np.isnan(look(lib, [lib.make_state(1.0), lib.make_pair(factor(0.5), bits)])[0])


@pytest.mark.parametrize("n", [1, 2, 5, 8, 9, 30])
def test_every_state_that_can_be_the_latest_gives_the_same(lib, n):
    rng = np.random.default_rng(n)
    pairs = [(float(np.float32(f)), float(np.float32(h))) for f, h in zip(rng.uniform(0, 1, n), rng.standard_normal(n))]
    zs = [(float(np.float32(factor(f))), h) for f, h in pairs]
    state, p = [], 0.0
    for z, h in zs:
        p = float(np.float32(lib.apply_factor(z, p)) + np.float32(h))
        state.append(p)
    pair, done = [lib.make_pair(z, h) for z, h in zs], [lib.make_state(p) for p in state]
    for known in range(max(0, n - 8), n):
        words = [done[t] if t <= known else pair[t] for t in range(n)]
        assert look(lib, words) == (np.float32(state[-1]), 0), known
        # the words of later tiles appear one by one, in any order
        order = list(rng.permutation(n))
        assert look(lib, [lib.unset()] * n, words, order)[0] == np.float32(state[-1]), known


def test_a_wait_without_end_gives_nan(lib):
    # no word at all, pairs without a state among them, a state behind a word that never comes
    u, q, s = lib.unset(), lib.make_pair(factor(0.5), 1.0), lib.make_state(3.0)
    for words in ([u] * 8, [q] * 8, [u] * 4 + [q] * 4, [s, u, q, q], [s] + [q] * 8):
        p, polls = look(lib, words, spins=20)
        assert np.isnan(p) and polls == 20, words
    assert look(lib, [s] + [q] * 7) == (np.float32(3.0 / 128 + 2 * (1 - 2.0 ** -7)), 0)
