"""Host-side checks of the calls over sequences with tokens in common: bad
arguments are refused before anything is launched (made-up device addresses,
skipped where a GPU is present), the parts of a span, the page allocator."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

from tests._shared_ref import compacted
from tests.test_kv16_host import (ALIGNMENT, BAD_CACHES, FAKE, INVALID, L, OK, P, UNSUPPORTED,  # noqa: F401
                                  WORKSPACE, cache, no_gpu_only)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOP = 2**31 - 1


def decode(L, c, q=P(FAKE), qs=512, Hq=4, group=P(FAKE), prefix=P(FAKE), n=2, scale=1.0, most=64, win=0, sink=0,
           out=P(FAKE), ws=P(FAKE), wb=1 << 34):
    return L.oscar_kv16_shared_decode_attention(ctypes.byref(c), q, qs, Hq, group, prefix, n, scale, most, win, sink,
                                                out, ws, wb, None)


def attention(L, c, q=P(FAKE), qs=512, st=P(FAKE), total=4, Hq=4, group=P(FAKE), prefix=P(FAKE), n=2, scale=1.0,
              most=64, win=0, sink=0, out=P(FAKE), lse=None, ws=P(FAKE), wb=1 << 34):
    return L.oscar_kv16_shared_attention(ctypes.byref(c), q, qs, st, total, Hq, group, prefix, n, scale, most, win,
                                         sink, out, lse, ws, wb, None)


def fork(L, src, dst, parent=P(FAKE), share=0, most=64):
    return L.oscar_kv16_fork(ctypes.byref(src), ctypes.byref(dst), parent, share, most, None)


def copy(L, src, dst, pairs=P(FAKE), n=P(FAKE), most=4):
    return L.oscar_kv16_copy_pages(ctypes.byref(src), ctypes.byref(dst), pairs, n, most, None)


def compact(L, table=P(FAKE), new=P(FAKE + 0x1000), B=2, blocks=8, pages=16, moves=P(FAKE + 0x2000),
            counts=P(FAKE + 0x3000), ws=P(FAKE + 0x100000), wb=1 << 34):
    return L.oscar_page_compact(table, new, B, blocks, pages, moves, counts, ws, wb, None)


@no_gpu_only
@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_every_call_checks_its_cache(L, bad, status):
    c, good = cache(**bad), cache(at=0x100000000)
    assert decode(L, c) == attention(L, c) == status
    assert fork(L, c, good) == fork(L, good, c) == copy(L, c, good) == copy(L, good, c) == status
    assert L.oscar_kv16_shared_decode_workspace_bytes(ctypes.byref(c), 4, 2, 64, 0, 0) == 0
    assert L.oscar_kv16_shared_attention_workspace_bytes(ctypes.byref(c), 4, 2, 4, 64, 0, 0) == 0


@no_gpu_only
def test_shared_refusals(L):
    c = cache()
    apart = P(FAKE + 0x10000000)
    for f in (lambda **k: decode(L, k.pop("c", c), **k), lambda **k: attention(L, k.pop("c", c), **k)):
        assert f(q=None) == f(out=None) == f(group=None) == f(prefix=None) == f(n=0) == f(n=-1) == INVALID
        assert f(qs=511) == f(qs=516) == f(qs=500) == INVALID
        assert f(scale=float("nan")) == f(scale=float("inf")) == f(most=-1) == f(win=-1) == f(sink=-1) == INVALID
        assert f(Hq=0) == f(Hq=3) == f(Hq=34) == UNSUPPORTED
        assert f(n=4097) == f(c=cache(B=4097)) == UNSUPPORTED
        assert f(q=P(FAKE + 8)) == f(out=P(FAKE + 8)) == f(group=P(FAKE + 2)) == f(prefix=P(FAKE + 1)) == ALIGNMENT
        # the output in the queries' memory
        assert f(out=P(FAKE + 1024)) == INVALID
    need = L.oscar_kv16_shared_decode_workspace_bytes(ctypes.byref(c), 4, 2, 64, 0, 0)
    assert need > 0
    assert decode(L, c, out=apart, wb=need - 1) == decode(L, c, out=apart, ws=None) == WORKSPACE
    assert decode(L, c, out=apart, ws=P(FAKE + 8)) == ALIGNMENT
    assert attention(L, c, st=None) == attention(L, c, total=-1) == INVALID
    assert attention(L, c, st=P(FAKE + 2)) == attention(L, c, lse=P(FAKE + 2)) == ALIGNMENT
    assert attention(L, c, out=apart, lse=P(FAKE)) == INVALID
    assert attention(L, c, total=0, q=None, out=None) == OK           # nothing to do
    assert attention(L, c, total=2**30) == UNSUPPORTED
    # records that 32 bits do not number
    assert attention(L, c, total=15750001, out=P(1 << 50), ws=None) == UNSUPPORTED
    assert attention(L, c, total=15750000, out=P(1 << 50), ws=None) == WORKSPACE
    need = L.oscar_kv16_shared_attention_workspace_bytes(ctypes.byref(c), 4, 2, 4, 64, 0, 0)
    assert need > 0
    assert attention(L, c, out=apart, wb=need - 1) == attention(L, c, out=apart, ws=None) == WORKSPACE
    assert decode(L, cache(B=4096, Hkv=17), qs=34 * 128, Hq=34) == UNSUPPORTED


@no_gpu_only
def test_fork_refusals(L):
    far = 0x100000000
    a, b = cache(), cache(at=far)
    assert fork(L, a, b, parent=None) == fork(L, a, b, share=2) == fork(L, a, b, most=-1) == INVALID
    assert fork(L, a, b, parent=P(FAKE + 2)) == ALIGNMENT
    assert fork(L, a, cache(at=far, Hkv=1)) == fork(L, a, cache(at=far, dtype=1)) == INVALID
    assert fork(L, cache(weight=None), b) == INVALID                   # weights from nowhere
    # pages are shared within a pool only
    assert fork(L, a, b, share=1) == fork(L, a, cache(n_pages=15, n_tok=FAKE + far), share=1) == INVALID
    assert fork(L, a, cache(at=far, block_table=None), share=1) == INVALID
    # memory in common that is not one pool's
    assert fork(L, a, cache(at=far, v=FAKE)) == fork(L, a, cache(at=far, k=FAKE + 4096)) == INVALID
    assert fork(L, cache(block_table=None), cache(block_table=None)) == INVALID
    # one pool: lengths and tables apart, or one cache
    pool = dict(n_tok=FAKE + 2 * far, block_table=FAKE + 3 * far)
    for clash in (dict(n_tok=a.n_tok + 4), dict(block_table=a.block_table + 8), dict(n_tok=a.block_table),
                  dict(block_table=a.n_tok - 4)):
        assert fork(L, a, cache(**{**pool, **clash}), parent=P(FAKE + 9 * far)) == INVALID
    # the parents in what the call writes
    assert fork(L, a, cache(**pool), parent=P(pool["n_tok"])) == INVALID
    assert fork(L, a, cache(**pool), parent=P(pool["block_table"]), share=1) == INVALID


@no_gpu_only
def test_copy_refusals(L):
    far = 0x100000000
    a, b = cache(), cache(at=far)
    assert copy(L, a, b, pairs=None) == copy(L, a, b, n=None) == copy(L, a, b, most=-1) == INVALID
    assert copy(L, a, b, pairs=P(FAKE + 4)) == copy(L, a, b, n=P(FAKE + 2)) == ALIGNMENT
    assert copy(L, a, cache(at=far, block_table=None)) == copy(L, cache(block_table=None), b) == INVALID
    assert copy(L, a, cache(at=far, Hkv=1)) == copy(L, a, cache(at=far, dtype=1)) == INVALID
    assert copy(L, cache(weight=None), b) == copy(L, a, cache(at=far, k=FAKE)) == INVALID
    assert copy(L, a, b, most=2**31 - 1) == UNSUPPORTED
    assert copy(L, a, b, most=0, pairs=None) == OK


def packed(**kw):
    from int2_kv_cache_02_gb300.oscar import OscarPagedCacheStruct
    s = OscarPagedCacheStruct()
    s.B, s.Hkv, s.max_blocks, s.n_pages = 2, 2, 8, 16
    for i, name in enumerate(("pages", "block_table", "n_packed", "n_res", "k_res", "v_res", "k_res_norm")):
        setattr(s, name, FAKE + i * 0x1000000)
    for name, x in kw.items():
        setattr(s, name, x)
    return s


@no_gpu_only
def test_packed_copy_refusals(L):
    f = lambda c=packed(), pairs=P(FAKE), n=P(FAKE), most=4: L.oscar_paged_copy_pages(
        ctypes.byref(c) if c is not None else None, pairs, n, most, None)
    assert f(c=None) == f(pairs=None) == f(n=None) == f(most=-1) == f(c=packed(pages=None)) == INVALID
    assert f(c=packed(Hkv=0)) == f(c=packed(n_pages=0)) == f(c=packed(bits=3)) == INVALID
    assert f(pairs=P(FAKE + 4)) == f(n=P(FAKE + 2)) == f(c=packed(pages=FAKE + 8)) == ALIGNMENT
    assert f(c=packed(Hkv=1 << 20)) == f(c=packed(Hkv=1 << 12), most=2**20) == UNSUPPORTED
    assert f(most=0, pairs=None) == OK


@no_gpu_only
def test_compact_refusals(L):
    assert compact(L, table=None) == compact(L, new=None) == compact(L, moves=None) == compact(L, counts=None) == INVALID
    assert compact(L, B=0) == compact(L, blocks=0) == compact(L, pages=0) == INVALID
    assert compact(L, table=P(FAKE + 2)) == compact(L, new=P(FAKE + 1)) == compact(L, moves=P(FAKE + 4)) == \
        compact(L, counts=P(FAKE + 2)) == compact(L, ws=P(FAKE + 8)) == ALIGNMENT
    assert compact(L, B=2**16, blocks=2**15) == compact(L, pages=12582913) == UNSUPPORTED
    assert L.oscar_page_compact_workspace_bytes(2, 8, 12582913) == 0
    # outputs in the table or in one another (but for the table in place)
    assert compact(L, new=P(FAKE + 4)) == compact(L, moves=P(FAKE + 8)) == compact(L, counts=P(FAKE + 60)) == INVALID
    assert compact(L, moves=P(FAKE + 0x1008)) == compact(L, counts=P(FAKE + 0x1000)) == compact(L, counts=P(FAKE + 0x2008)) == INVALID
    need = L.oscar_page_compact_workspace_bytes(2, 8, 16)
    assert need > 0 and L.oscar_page_compact_workspace_bytes(0, 8, 16) == 0
    assert compact(L, wb=need - 1) == compact(L, ws=None) == compact(L, new=P(FAKE), wb=need - 1) == WORKSPACE


# ------------------------------------------------------------ parts of a span

HARNESS = r"""
#include "kv16_span.h"
extern "C" int part(int first, int last, int window, int sink, int n, int own, int* out) {
  const oscar::Span all(first, last, window, sink), s = own ? all.from(n) : all.below(n);
  for (int i = 0; i < s.blocks && i < 4096; ++i) out[i] = s.block(i);
  return s.blocks;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("part")
    src, so = d / "part.cpp", d / "part.so"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "int2_kv_cache_02_gb300", "csrc"), str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


@pytest.mark.parametrize("window", [0, 1, 2, 32, 33, 100, 1000, TOP])
@pytest.mark.parametrize("sink", [0, 1, 32, 33, 200, TOP])
def test_the_parts_of_a_span_cover_what_is_seen_once(lib, window, sink):
    out = (ctypes.c_int * 4096)()
    for first, count in [(0, 1), (31, 2), (0, 300), (299, 1), (700, 64), (-1, 1), (-7, 10), (-100, 3)]:
        last = first + count - 1
        want = {j // 32 for at in range(max(first, 0), last + 1) for j in range(at + 1)
                if window == 0 or j > at - window or j < sink}
        for n in (0, 1, 2, 5, 8, 9, 22, 23, 24, 40):
            parts = []
            for own in (0, 1):
                k = lib.part(first, last, window, sink, n, own, out)
                assert 0 <= k <= 4096
                parts.append([out[i] for i in range(k)])
            assert all(j < n for j in parts[0]) and all(j >= n for j in parts[1])
            both = parts[0] + parts[1]
            assert both == sorted(set(both)) and want <= set(both)
            assert all(0 <= 32 * j <= max(last, -1) for j in both)


# ---------------------------------------------------------- the page allocator

def make_pool(B=3, blocks=6, pages=16):
    from int2_kv_cache_02_gb300.oscar import _PagePool

    class Pool(_PagePool):
        pass

    p = Pool()
    p.block_table = torch.full((B, blocks), -1, dtype=torch.int32)
    p._init_pool(B, blocks, pages)
    return p


def test_shared_pages_are_free_when_no_sequence_has_them(L):
    p = make_pool()
    p.map_blocks(0, 4)
    p.share_blocks(1, 0, 3)
    p.map_blocks(1, 5)
    p.share_blocks(2, 1, 2)
    assert p.block_table.tolist() == [[0, 1, 2, 3, -1, -1], [0, 1, 2, 4, 5, -1], [0, 1, -1, -1, -1, -1]]
    assert p._free == list(range(6, 16))
    p.release_blocks(0)
    assert p._free == list(range(6, 16)) + [3]
    p.release_blocks(1, 1)
    assert p._free == list(range(6, 16)) + [3, 2, 4, 5]
    p.release_blocks(2)
    p.release_blocks(1)
    assert sorted(p._free) == list(range(16)) and p._named == [0] * 16
    # pages that a sequence had there are given back, its parent's own stay
    p.map_blocks(0, 2)
    p.map_blocks(1, 3)
    had = p._table_host[1][:2]
    p.share_blocks(1, 0, 2)
    p.share_blocks(1, 0, 2)
    p.share_blocks(0, 0, 2)
    assert p._table_host[1][:2] == p._table_host[0][:2] and set(had) <= set(p._free)
    assert [p._named[x] for x in p._table_host[0][:2]] == [2, 2]


def test_share_blocks_refusals(L):
    from int2_kv_cache_02_gb300.oscar import OscarError
    p = make_pool()
    p.map_blocks(0, 2)
    for n in (3, 7, -1):
        with pytest.raises(OscarError):
            p.share_blocks(1, 0, n)
    assert p.block_table.tolist()[1] == [-1] * 6


def test_compact_keeps_the_allocator_in_step(L, monkeypatch):
    """The host's copy goes by the kernel's rule (here: by the plain form in its place)."""
    from int2_kv_cache_02_gb300 import oscar
    rng = random.Random(3)

    def plan(table, new, n_pages, moves, counts, workspace, stream=None):
        rows, m, live = compacted(table.tolist(), n_pages)
        new.copy_(torch.tensor(rows, dtype=torch.int32))
        moves.fill_(-1)
        moves[:len(m)] = torch.tensor(m, dtype=torch.int32).view(-1, 2)
        counts.copy_(torch.tensor([len(m), live], dtype=torch.int32))

    monkeypatch.setattr(oscar, "page_compact", plan)
    for _ in range(50):
        p = make_pool(5, 6, 40)
        for b in range(5):
            if b and rng.random() < 0.5:
                parent = rng.randrange(b)
                p.share_blocks(b, parent, rng.randint(0, sum(x >= 0 for x in p._table_host[parent])))
            p.map_blocks(b, rng.randint(0, 6), order=rng.sample(range(40), 40))
        for b in rng.sample(range(5), rng.randint(0, 4)):
            p.release_blocks(b, rng.randint(0, 3))
        moves, counts = p.compact()
        live = int(counts[1])
        assert p.block_table.tolist() == p._table_host
        named = [x for row in p._table_host for x in row if x >= 0]
        assert set(named) == set(range(live)) and p._free == list(range(live, 40))
        assert p._named == [named.count(x) for x in range(40)]


def test_page_compact_takes_device_tensors(L):
    from int2_kv_cache_02_gb300 import oscar
    t = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        oscar.page_compact(t, t, 8, torch.zeros((4, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(64))
