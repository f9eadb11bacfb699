"""Which blocks and tokens of the 16-bit cache a query sees, checked on the host:
the kernels' own header, compiled as plain C++, against a plain count.  Covers
positions below zero (a sequence of fewer tokens than queries) and windows up
to 2^31 - 1."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOP = 2**31 - 1
HARNESS = r"""
#include "kv16_span.h"
extern "C" void span(int first, int last, int window, int sink, int* out) {
  const oscar::Span s(first, last, window, sink);
  out[0] = s.sink_blocks;
  out[1] = s.w0;
  out[2] = s.blocks;
}
extern "C" int block(int first, int last, int window, int sink, int i) {
  return oscar::Span(first, last, window, sink).block(i);
}
extern "C" int visible(int j, int at, int window, int sink) {
  return oscar::kv16_visible(j, at, window, sink);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("span")
    src, so = d / "span.cpp", d / "span.so"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "int2_kv_cache_02_gb300", "csrc"), str(src), "-o", str(so)],
                   check=True)
    return ctypes.CDLL(str(so))


def seen(at, window, sink):
    return [j for j in range(at + 1) if window == 0 or j > at - window or j < sink]


@pytest.mark.parametrize("window", [0, 1, 2, 31, 32, 33, 100, 5000, TOP - 1, TOP])
@pytest.mark.parametrize("sink", [0, 1, 32, 33, 200, TOP])
def test_span_covers_what_is_seen(lib, window, sink):
    out = (ctypes.c_int * 3)()
    for first, count in [(0, 1), (5, 1), (31, 2), (0, 300), (63, 40), (200, 128), (299, 1),
                         (-1, 1), (-7, 10), (-7, 3), (-100, 130), (-300, 40), (-TOP + 500, 64)]:
        last = first + count - 1
        lib.span(first, last, window, sink, out)
        assert out[0] >= 0 and out[1] >= 0 and out[2] >= 0, (first, last, list(out))
        blocks = [lib.block(first, last, window, sink, i) for i in range(out[2])]
        assert blocks == sorted(set(blocks))
        want = {j // 32 for at in range(max(first, 0), last + 1) for j in seen(at, window, sink)}
        assert want <= set(blocks), (first, last, list(out))
        # and no block outside the queries' own range and reach
        assert all(32 * b <= max(last, -1) for b in blocks)


def test_visible(lib):
    for window in (0, 1, 30, TOP):
        for sink in (0, 4, TOP):
            for at in (-5, -1, 0, 3, 100):
                got = [j for j in range(130) if lib.visible(j, at, window, sink)]
                assert got == seen(at, window, sink)


def test_largest_positions(lib):
    """The last tokens of the longest sequence, under the widest windows."""
    out = (ctypes.c_int * 3)()
    last = TOP - 129
    for window, sink in ((0, 0), (1, 0), (TOP, TOP), (TOP, 0), (100, TOP), (100, 64)):
        lib.span(last - 127, last, window, sink, out)
        assert min(out) >= 0 and lib.block(last - 127, last, window, sink, out[2] - 1) == last // 32
