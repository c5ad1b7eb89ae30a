"""The arithmetic that finds a new token's place in the paged cache, compiled for the host and
compared with Python's unbounded integers at the ends of 32 bits."""
import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

LO, HI = -2 ** 31, 2 ** 31 - 1
CSRC = os.path.join(ROOT, "sparse_top_landmark_gb300", "csrc")
SOURCE = """
#include "token_place.h"
extern "C" int position(int len, int begin, int end, int t) {
  return mita::token_position(len, begin, end, t);
}
extern "C" int fits(int len, int width, int page_log2) {
  return mita::fits_table(len, width, page_log2);
}
"""


@pytest.fixture(scope="module")
def place(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("place")
    (d / "place.cpp").write_text(SOURCE)
    # -fwrapv would hide an overflow, the trap shows one
    subprocess.run([cxx, "-std=c++17", "-O1", "-ftrapv", "-shared", "-fPIC", "-I", CSRC,
                    str(d / "place.cpp"), "-o", str(d / "place.so")], check=True)
    return ctypes.CDLL(str(d / "place.so"))


def want_position(n, begin, end, t):
    pos = n - (end - t)
    return pos if n > 0 and end - begin <= n and 0 <= pos < n else -1


def test_positions_at_the_ends_of_32_bits(place):
    ends = [LO, LO + 1, LO + 10, -7, -4, -1, 0, 1, 2, 5, 8, 100, HI - 1, HI]
    seen = 0
    for begin in ends:
        for end in ends:
            for t in [t for t in (0, 1, 5, 99, HI - 1) if begin <= t < end]:
                for n in ends:
                    got = place.position(n, begin, end, t)
                    assert got == want_position(n, begin, end, t), (n, begin, end, t)
                    assert got < max(n, 0)
                    seen += 1
    assert seen > 500


def test_a_negative_length_between_far_row_starts_has_no_place(place):
    # end - begin and len - (end - t) both leave 32 bits here
    assert place.position(-4, LO + 10, HI, 0) == -1


def test_lengths_that_fit_a_table(place):
    for log2 in (0, 4, 20):
        for width in (0, 1, 7, (HI - (1 << 16)) >> log2):
            room = width << log2
            for n in (1, 2, room - 1, room, room + 1, HI):
                if 0 < n <= HI:
                    assert bool(place.fits(n, width, log2)) == (n <= room), (n, width, log2)
