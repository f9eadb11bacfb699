"""Shared prefixes that end among the sinks of a window, on the GPU: each
sequence's own part is what is left of the sinks and its window."""
import pytest
import torch

from tests import _kv16_ref as R
from tests._shared_ref import SharedCase
from tests.test_gpu_kv16_shared import L, attend, decode  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("window,sink", [(128, 100), (40, 300), (1, 65), (1000, 1024), (700, 2000)])
@pytest.mark.parametrize("prefix", [32, 64, 256])
@pytest.mark.parametrize("Hq,Hkv,dtype,paged", [(8, 2, BF, True), (16, 1, FP, False)])
def test_decode(L, window, sink, prefix, Hq, Hkv, dtype, paged):
    lens = [prefix + 1, 2500, 3333, 4100, 90 + prefix, 1024, 2048]
    case = SharedCase([4, 3], [prefix, prefix], lens, Hkv, dtype=dtype, paged=paged, seed=sink % 100 + prefix)
    decode(L, case, case.cache(L), Hq, window, sink)


@pytest.mark.parametrize("window,sink", [(128, 100), (40, 300), (700, 2000)])
@pytest.mark.parametrize("prefix", [32, 256])
@pytest.mark.parametrize("Hq,Hkv,dtype", [(8, 2, FP), (3, 1, BF)])
def test_attention(L, window, sink, prefix, Hq, Hkv, dtype):
    lens = [prefix + 30, 2500, 3333, 1900, 90 + prefix]
    case = SharedCase([3, 2], [prefix, prefix], lens, Hkv, dtype=dtype, seed=sink % 100 + prefix)
    attend(L, case, case.cache(L), [20, 1, 300, 90, 33], Hq, window, sink)


def test_what_lies_between_is_not_read(L):
    """Between the sinks and the window: pages out of the pool's range, which
    the status word would name."""
    window, sink, prefix, n = 128, 100, 64, 4000
    case = SharedCase([3], [prefix], [n, n - 7, n + 90], 2, dtype=FP)
    cache = case.cache(L)
    q = case.normal(3, 8)
    want = [R.attend(case, b, q[b:b + 1], window, sink) for b in range(3)]
    cache.block_table[:, 4:(n - 7 - window) // 32] = 1 << 20
    for out in decode(L, case, cache, 8, window, sink, q=q, check=False):
        assert L.device_status() == 0
        for b in range(3):
            R.assert_within(out[b:b + 1], want[b][0], want[b][3], f"sequence {b}")
    out, _ = attend(L, case, cache, [1, 1, 1], 8, window, sink, q=q, extra=0, check=False)
    assert L.device_status() == 0
    for b in range(3):
        R.assert_within(out[b:b + 1], want[b][0], want[b][3], f"sequence {b}")
