"""The 16-bit cache's calls at the edges of what their documentation allows:
bad lengths under windows, values that are not finite, weights of very unequal
size, waits that run out, rows too long to hold.  Against the same plain 64-bit
forms as the other tests of these calls."""
import math

import pytest
import torch

from tests import _kv16_ref as R
from tests.test_gpu_kv16 import i32, run_attention, run_decode  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
TOP = 2**31 - 1


@pytest.fixture(scope="module")
def L():
    from int2_kv_cache_02_gb300 import _build
    _build.build()
    from int2_kv_cache_02_gb300 import oscar
    oscar.device_status()
    return oscar


# ------------------------------------------------- bad lengths under windows

@pytest.mark.parametrize("window,sink", [(TOP, 0), (TOP, TOP), (TOP - 5, 4), (5, 0), (40, 3), (1, 200)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (3, 1)])
def test_fewer_tokens_than_queries_under_a_window(L, window, sink, Hq, Hkv):
    """A sequence that holds fewer tokens than it has queries, under windows up to
    the widest: recorded, and every other sequence is right, before it and behind
    it in the order of work."""
    lens, news = [300, 100, 200, 260], [300, 60, 40, 200]
    for bad in (3, 0, -5, 10**6):
        case = R.Case(lens, Hkv, BF, seed=Hq, weights=True)
        cache, start = case.cache(L, [300, bad, 200, 260]), R.start_of(news)
        q = case.normal(start[-1], Hq)
        out = torch.zeros((start[-1], Hq, 128), dtype=BF, device="cuda")
        lse = torch.zeros((start[-1], Hq), device="cuda")
        ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, Hq, start[-1], 320, window, sink))
        L.kv16_attention(cache, q.cuda(), i32(start), R.SCALE, 320, out, ws, window, sink, lse)
        assert L.device_status() != 0 and L.device_status() == 0
        L.kv16_accumulate(cache, q.cuda(), lse, i32(start), R.SCALE, 320, window, sink)
        assert L.device_status() != 0
        for b in (0, 2, 3):
            rows = slice(start[b], start[b + 1])
            o, z, p, tol, ztol, dmax = R.attend(case, b, q[rows], window, sink)
            R.assert_within(out[rows], o, tol, f"out {b}")
            R.assert_within(lse[rows], z, ztol, f"lse {b}")
            w, t = R.weight_of(p, dmax, Hq // Hkv)
            R.assert_within(R.tokens(cache, b, lens[b], "weight"), w + case.w[b].double(),
                            t + 4 * float(ztol.max()) * w + 2 * R.U32, f"weight {b}")


@pytest.mark.parametrize("window,sink", [(TOP, 0), (TOP, TOP), (5, 3)])
def test_decode_bad_lengths_under_a_window(L, window, sink):
    for bad in (-5, -TOP, TOP, 10**6):
        case = R.Case([300, 100, 33], 2, BF, weights=True)
        cache = case.cache(L, [300, bad, 33])
        q = case.normal(3, 8)
        out = torch.zeros((3, 8, 128), dtype=BF, device="cuda")
        ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 8, 320, window, sink, True))
        L.kv16_decode_attention(cache, q.cuda(), R.SCALE, 320, out, ws, window, sink, accumulate=True)
        assert L.device_status() != 0
        assert (ws[:65536].view(torch.int32) == 0).all()
        for b in (0, 2):
            o, _, p, tol, _, dmax = R.attend(case, b, q[b:b + 1], window, sink)
            R.assert_within(out[b:b + 1], o, tol, str(b))
            w, t = R.weight_of(p, dmax, 4)
            R.assert_within(R.tokens(cache, b, case.lens[b], "weight"), w + case.w[b].double(),
                            t + 2 * R.U32, str(b))
