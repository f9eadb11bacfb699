"""What a group and its sequences read of a cache, on the host: the parts of a
span before and behind a shared prefix are together the span's blocks, no more."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HARNESS = r"""
#include "kv16_span.h"
using oscar::Span;
extern "C" int part(int first, int last, int window, int sink, int n, int which, int* out) {
  const Span all(first, last, window, sink), s = which == 0 ? all : which == 1 ? all.below(n) : all.from(n);
  for (int i = 0; i < s.blocks && i < 4096; ++i) out[i] = s.block(i);
  return s.blocks;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("parts")
    src, so = d / "parts.cpp", d / "parts.so"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "int2_kv_cache_02_gb300", "csrc"), str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


@pytest.mark.parametrize("window", [0, 1, 32, 100, 128, 1000, 2**31 - 1])
@pytest.mark.parametrize("sink", [0, 1, 4, 33, 64, 100, 200, 2000, 2**31 - 1])
def test_no_block_is_read_that_the_span_lacks(lib, window, sink):
    out = (ctypes.c_int * 4096)()
    for first, count in [(0, 1), (63, 1), (500, 1), (5000, 1), (4000, 200), (90, 40), (-3, 9)]:
        blocks = lambda which, n: [out[i] for i in range(lib.part(first, first + count - 1, window, sink, n, which, out))]
        whole = blocks(0, 0)
        for n in (0, 1, 2, 3, 4, 6, 7, 20, 62, 63, 64, 130, 200):
            assert blocks(1, n) == [j for j in whole if j < n]
            assert blocks(2, n) == [j for j in whole if j >= n], (first, count, n)
