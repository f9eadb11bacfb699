"""The 16-bit cache's calls from host threads: one that has never used the GPU,
and two at once."""
import threading

import pytest
import torch

from tests import _kv16_ref as R
from tests._shared_ref import bits, i32

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    from int2_kv_cache_02_gb300 import _build
    _build.build()
    from int2_kv_cache_02_gb300 import oscar
    oscar.device_status()
    return oscar


def in_thread(*calls):
    """Runs the calls, a thread each; what they raised."""
    raised = []

    def go(f):
        try:
            f()
        except Exception as e:      # noqa: BLE001 (handed to the test)
            raised.append(e)

    threads = [threading.Thread(target=go, args=(f,)) for f in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return raised


def calls_of(L, case, cache, Hq, most):
    """name -> (call(stream), its outputs): one call of each kind on this cache."""
    B, g = case.B, Hq // case.Hkv
    q = case.normal(B, Hq).cuda()
    start, pos, zero = i32(list(range(B + 1))), cache.n_tok - 1, i32([0] * B)
    group, prefix = i32([0, B]), i32([32])
    outs = [torch.zeros_like(q) for _ in range(3)]
    lse = torch.zeros((B, Hq), device="cuda")
    ws = [L.alloc_workspace(n) for n in (
        L.kv16_attention_workspace_bytes(cache, Hq, B, most), L.kv16_decode_workspace_bytes(cache, Hq, most),
        L.kv16_shared_decode_workspace_bytes(cache, Hq, 1, most),
        L.kv16_shared_attention_workspace_bytes(cache, Hq, 1, B, most),
        L.kv16_evict_workspace_bytes(cache, most, 1, 1, 1),
        L.page_compact_workspace_bytes(cache.block_table, cache.k.shape[0]))]
    row = case.normal(B, case.Hkv).cuda()
    kept = torch.empty((B, case.Hkv, 3), dtype=torch.int32, device="cuda")
    to = L.KV16Cache.contiguous(B, case.Hkv, most, weights=True)
    few = L.KV16Cache.contiguous(B, case.Hkv, 3)
    table, moves, counts = torch.empty_like(cache.block_table), i32([[0, 0]] * (cache.k.shape[0] // 2)), i32([0, 0])
    pairs, n_pairs = i32([[0, 0]]), i32([0])
    return {
        "write": (lambda s: L.kv16_write(cache, row, row, start, pos, stream=s), [cache.n_tok]),
        "attention": (lambda s: L.kv16_attention(cache, q, start, R.SCALE, most, outs[0], ws[0], lse=lse, stream=s), [outs[0], lse]),
        "decode": (lambda s: L.kv16_decode_attention(cache, q, R.SCALE, most, outs[1], ws[1], stream=s), [outs[1]]),
        "accumulate": (lambda s: L.kv16_accumulate(cache, q, lse, start, R.SCALE, most, stream=s), []),
        "evict": (lambda s: L.kv16_evict(cache, few, most, 1, 1, 1, ws[4], kept, stream=s), [kept]),
        "shared decode": (lambda s: L.kv16_shared_decode_attention(cache, q, group, prefix, R.SCALE, most, outs[2], ws[2], stream=s), [outs[2]]),
        "shared attention": (lambda s: L.kv16_shared_attention(cache, q, start, group, prefix, R.SCALE, most, outs[2], ws[3], lse=lse, stream=s), [outs[2], lse]),
        "fork": (lambda s: L.kv16_fork(cache, to, zero, most, share=False, stream=s), [to.n_tok, to.k]),
        "compact": (lambda s: L.page_compact(cache.block_table, table, cache.k.shape[0], moves, counts, ws[5], stream=s), [table, counts]),
        "copy pages": (lambda s: L.kv16_copy_pages(cache, cache, pairs, n_pairs, stream=s), []),
    }


NAMES = ("write", "attention", "decode", "accumulate", "evict", "shared decode", "shared attention", "fork", "compact",
         "copy pages")


@pytest.mark.parametrize("name", NAMES)
def test_the_first_call_of_a_thread(L, name):
    """Everything is made by this thread; the other one makes the call and nothing else."""
    case = R.Case([70, 50], 2, BF, weights=True)
    cache = case.cache(L)
    call, outs = calls_of(L, case, cache, 8, cache.capacity)[name]
    stream = torch.cuda.current_stream().cuda_stream
    call(stream)
    torch.cuda.synchronize()
    want = [bits(x).clone() for x in outs]
    for x in outs[:1]:
        x.zero_()
    assert in_thread(lambda: call(stream)) == []
    assert L.device_status() == 0
    for x, y in zip(outs, want):
        assert torch.equal(bits(x), y)
