"""Waits of the attention over shared prefixes that run out, on the GPU: its copies
end early, every block gives up in time, says so in the status word and leaves the
GPU's memory and the next call as they should be."""
import time

import pytest
import torch

from tests import _kv16_ref as R
from tests._shared_ref import SharedCase
from tests.test_gpu_kv16_shared import L, decode  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
DEVICE_STATUS = 7

CASES = {
    # rows for one query tile and for two, tiles cleared behind a last token
    "groups": ([40, 3, 60], [700, 400, 1500], 8, 2, BF),
    "long": ([70], [9000], 16, 1, FP),
    "many short": ([2] * 100, [64] * 100, 4, 2, BF),
}


def case_of(name):
    members, prefix, Hq, Hkv, dtype = CASES[name]
    lens = [p + 1 + (37 * i) % 90 for m, p in zip(members, prefix) for i in range(m)]
    return SharedCase(members, prefix, lens, Hkv, dtype=dtype, seed=len(lens)), Hq


# A CTA's run of the line reaches into two rows in "groups" and "long" (57 and
# 51 places, of rows that take 38 and 41 for their one tile), four in "many short" (150).
@pytest.mark.parametrize("name,items", [
    ("groups", None), ("groups", 0), ("groups", 1), ("long", 0), ("long", 1),
    ("many short", None), ("many short", 0), ("many short", 1), ("many short", 2)])
def test_copies_that_end_early(L, name, items):
    """items None: by the bound that takes a CTA a row where that is quicker ("many
    short"); else the copies of so many pieces of every CTA's work."""
    case, Hq = case_of(name)
    cache = case.cache(L)
    group, prefix = case.groups()
    most = cache.capacity if items is None else 1 << 20
    q = case.normal(case.B, Hq).cuda()
    out = torch.empty_like(q)
    ws = L.alloc_workspace(L.kv16_shared_decode_workspace_bytes(cache, Hq, len(case.prefix), most))
    L.kv16_shared_decode_attention(cache, q, group, prefix, R.SCALE, most, out, ws)
    torch.cuda.synchronize()
    t = time.time()
    L.selftest_kv16_shared_timeout(cache, q, group, prefix, most, out, ws, items=items or 0)
    torch.cuda.synchronize()
    assert time.time() - t < 10
    assert L.device_status() == DEVICE_STATUS and L.device_status() == 0
    decode(L, case, cache, Hq)


def test_no_wait_runs_out_where_all_is_copied(L):
    case, Hq = case_of("groups")
    cache = case.cache(L)
    group, prefix = case.groups()
    q = case.normal(case.B, Hq).cuda()
    outs = [torch.empty_like(q) for _ in range(2)]
    ws = L.alloc_workspace(L.kv16_shared_decode_workspace_bytes(cache, Hq, len(case.prefix), 1 << 20))
    L.kv16_shared_decode_attention(cache, q, group, prefix, 1.0, 1 << 20, outs[0], ws)
    L.selftest_kv16_shared_timeout(cache, q, group, prefix, 1 << 20, outs[1], ws, items=2**31 - 1)
    assert L.device_status() == 0
    assert torch.equal(outs[0], outs[1])
