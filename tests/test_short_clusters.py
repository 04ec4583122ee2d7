"""The choice of cluster size for a short cache's decode (csrc/mala_short_cluster.h), compiled
by itself and asked with GPUs of our making: whole ones, ones whose parts hold fewer clusters
than their CTAs would make, and ones that hold none of the larger sizes."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mass_gated_causal_b200", "csrc")

SHIM = """
#include "mala_short_cluster.h"
// room: clusters at once by log2 of the size, for CTAs of up to `pair_tiles` tiles and for larger ones
extern "C" int pick(long long units, long long tiles, long long ctas, const int* pair, const int* alone, int pair_tiles) {
  return mala::short_cluster(units, tiles, ctas, [&](int c, int each) {
    int lg = 0;
    while ((1 << lg) < c) ++lg;
    return (each <= pair_tiles ? pair : alone)[lg];
  });
}
"""


@pytest.fixture(scope="module")
def pick(tmp_path_factory):
    at = tmp_path_factory.mktemp("shim")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + CSRC,
                           str(at / "shim.cpp"), "-o", str(at / "shim.so")])
    fn = ctypes.CDLL(str(at / "shim.so")).pick
    fn.argtypes = [ctypes.c_longlong] * 3 + [ctypes.POINTER(ctypes.c_int)] * 2 + [ctypes.c_int]

    def call(units, tiles, pair, alone=None, ctas=296, pair_tiles=8):
        room = lambda x: (ctypes.c_int * 5)(*x)
        return fn(units, tiles, ctas, room(pair), room(alone or pair), pair_tiles)
    return call


WHOLE = (296, 148, 71, 33, 14)      # what a B200 of 148 SMs holds, two CTAs to an SM
ALONE = (148, 74, 33, 15, 7)        # one CTA to an SM


@pytest.mark.parametrize("units,tiles,want", [
    (4, 32, 16), (1, 1, 1), (1, 2, 1), (1, 3, 2), (1, 128, 16), (1, 129, 0), (14, 128, 16),
    (15, 32, 8),     # 240 CTAs would be there, but not 15 clusters of sixteen of them
    (18, 32, 8), (18, 128, 0), (33, 64, 8), (34, 32, 4), (36, 32, 4), (71, 32, 4), (72, 32, 0), (72, 16, 2),
    (148, 16, 2), (149, 8, 1), (296, 8, 1), (297, 8, 0),
])
def test_on_a_whole_gpu(pick, units, tiles, want):
    assert pick(units, tiles, WHOLE) == want


def test_one_wave_whatever_the_sizes(pick):
    for units in range(1, 300):
        for tiles in range(1, 140):
            c = pick(units, tiles, WHOLE, ALONE, pair_tiles=5)
            if c:
                each = -(-tiles // c)
                assert each <= 8 and units <= (WHOLE if each <= 5 else ALONE)[c.bit_length() - 1]


@pytest.mark.parametrize("room,units,tiles,want", [
    ((16, 8, 4, 2, 0), 1, 60, 8),     # a part of a GPU that no cluster of sixteen fits
    ((16, 8, 4, 2, 0), 1, 100, 0),    # whose eight CTAs would have too many tiles: the other path
    ((16, 8, 4, 0, 0), 1, 30, 4),
    ((0, 0, 0, 0, 0), 1, 1, 0),       # or the question failed
])
def test_on_a_part_of_a_gpu(pick, room, units, tiles, want):
    assert pick(units, tiles, room) == want
