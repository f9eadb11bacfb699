"""The 16-bit cache's calls from host threads: one that has never used the GPU,
and several at once."""
import ctypes
import os
import subprocess
import threading
from ctypes import c_int, c_size_t, c_void_p

import pytest
import torch

from tests import _kv16_ref as R
from tests._shared_ref import bits, i32

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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
    to = L.KV16Cache.contiguous(B, case.Hkv, cache.capacity, weights=True)
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


# Host threads in calls at the same time, a large one and small ones, without the
# interpreter's lock between them.
HARNESS = r"""
#include <atomic>
#include <thread>
#include "oscar.h"
struct Call {
  int kind, large;
  const oscar_kv16_cache* c;
  const uint16_t* q;
  int Hq;
  const int32_t *group, *prefix;
  int max_tok;
  uint16_t* out;
  const int32_t* table;
  int32_t *new_table, *moves, *counts;
  int B, blocks, n_pages;
  const oscar_kv16_cache* to;
  void* ws;
  size_t ws_bytes;
  void* stream;
};
using Compact = decltype(&oscar_page_compact);
using Shared = decltype(&oscar_kv16_shared_decode_attention);
using Decode = decltype(&oscar_kv16_decode_attention);
using Evict = decltype(&oscar_kv16_evict);
static int call(const void* const* f, const Call& x) {
  switch (x.kind) {
    case 0: return ((Compact)f[0])(x.table, x.new_table, x.B, x.blocks, x.n_pages, x.moves, x.counts, x.ws,
                                   x.ws_bytes, x.stream);
    case 1: return ((Shared)f[1])(x.c, x.q, (long long)x.Hq * 128, x.Hq, x.group, x.prefix, 1, 0.1f, x.max_tok, 0, 0,
                                  x.out, x.ws, x.ws_bytes, x.stream);
    case 2: return ((Evict)f[3])(x.c, x.to, x.max_tok, 1, 1, 1, nullptr, x.ws, x.ws_bytes, x.stream);
    default: return ((Decode)f[2])(x.c, x.q, (long long)x.Hq * 128, x.Hq, 0.1f, x.max_tok, 0, 0, x.kind == 4, x.out,
                                   x.ws, x.ws_bytes, x.stream);
  }
}
extern "C" int hammer(const void* const* f, const Call* calls, int n, int times) {
  std::atomic<int> failed{0}, ready{0};
  auto run = [&](const Call& x) {
    for (++ready; ready < n;) {}
    for (int i = 0; i < times; ++i) failed += call(f, x) != 0;
  };
  std::thread t[8];
  for (int i = 0; i < n; ++i) t[i] = std::thread(run, std::cref(calls[i]));
  for (int i = 0; i < n; ++i) t[i].join();
  return failed;
}
"""
FIELDS = [("kind", c_int), ("large", c_int), ("c", c_void_p), ("q", c_void_p), ("Hq", c_int), ("group", c_void_p),
          ("prefix", c_void_p), ("max_tok", c_int), ("out", c_void_p), ("table", c_void_p), ("new_table", c_void_p),
          ("moves", c_void_p), ("counts", c_void_p), ("B", c_int), ("blocks", c_int), ("n_pages", c_int),
          ("to", c_void_p), ("ws", c_void_p), ("ws_bytes", c_size_t), ("stream", c_void_p)]


class Call(ctypes.Structure):
    _fields_ = FIELDS


@pytest.fixture(scope="module")
def hammer(tmp_path_factory):
    d = tmp_path_factory.mktemp("hammer")
    src, so = d / "hammer.cpp", d / "hammer.so"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so)).hammer


KINDS = {"compact": 0, "line": 1, "short": 1, "evict": 2, "decode": 3, "weights": 4}


def sized(L, what, large, keep):
    """A call whose blocks ask for much or for little shared memory, and its outputs."""
    x = Call(kind=KINDS[what], large=large)
    if what == "compact":
        x.B, x.blocks, x.n_pages = 1, 4, 8000000 if large else 16
        table, moves, counts = i32([[5, 1, -1, 7]]), torch.empty(x.n_pages, dtype=torch.int32, device="cuda"), i32([0, 0])
        new = torch.empty_like(table)
        ws = L.alloc_workspace(L.page_compact_workspace_bytes(table, x.n_pages))
        x.table, x.new_table, x.moves, x.counts = (t.data_ptr() for t in (table, new, moves, counts))
        outs = [new, counts]
        keep += [table, moves]
    else:
        B = 1500 if large and what in ("line", "decode", "weights") else 2
        x.Hq = 16 if large and what == "short" else 1
        case = R.Case([40] * B, 1, weights=True, slack=700 if large and what == "evict" else 1)
        cache = case.cache(L)
        x.max_tok = 1 << 20 if what == "line" else cache.capacity
        q, group, prefix = case.normal(B, x.Hq).cuda(), i32([0, B]), i32([32])
        out, to = torch.empty_like(q), L.KV16Cache.contiguous(B, 1, 3)
        if what == "evict":
            n = L.kv16_evict_workspace_bytes(cache, x.max_tok, 1, 1, 1)
        elif what in ("line", "short"):
            n = L.kv16_shared_decode_workspace_bytes(cache, x.Hq, 1, x.max_tok)
        else:
            n = L.kv16_decode_workspace_bytes(cache, x.Hq, x.max_tok, accumulate=what == "weights")
        ws = L.alloc_workspace(n)
        x.c, x.to = ctypes.addressof(cache.struct), ctypes.addressof(to.struct)
        x.q, x.group, x.prefix, x.out = (t.data_ptr() for t in (q, group, prefix, out))
        outs = [to.k, to.n_tok] if what == "evict" else [out]
        keep += [cache, q, group, prefix, to]
    stream = torch.cuda.Stream()
    x.ws, x.ws_bytes, x.stream = ws.data_ptr(), ws.nbytes, stream.cuda_stream
    keep += [ws, stream]
    return x, outs


@pytest.mark.parametrize("what", KINDS)
def test_calls_of_unequal_size_at_once(L, hammer, what):
    """A small call between a large one's preparation and its launch does not fail it."""
    lib, keep = L.library(), []
    f = (c_void_p * 4)(*(ctypes.cast(getattr(lib, "oscar_" + n), c_void_p) for n in (
        "page_compact", "kv16_shared_decode_attention", "kv16_decode_attention", "kv16_evict")))
    calls = [sized(L, what, large, keep) for large in (True, False, False)]
    torch.cuda.synchronize()
    want = []
    for x, outs in calls:
        assert hammer(f, (Call * 1)(x), 1, 1) == 0
        torch.cuda.synchronize()
        want.append([bits(t).clone() for t in outs])
    assert hammer(f, (Call * 3)(*(x for x, _ in calls)), 3, 2000) == 0
    torch.cuda.synchronize()
    assert L.device_status() == 0
    for (_, outs), w in zip(calls, want):
        for t, y in zip(outs, w):
            assert torch.equal(bits(t), y)
