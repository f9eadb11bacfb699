"""Host-side checks of the 16-bit cache's calls: bad arguments are refused
before anything is launched, workspace sizes, the page allocator.  No kernel
runs here; the cases pass made-up device addresses and are skipped where a GPU
is present, so that a hole in the checks can never become a launch."""
import ctypes

import pytest
import torch

from int2_kv_cache_02_gb300 import _build

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake-pointer validation runs only without a GPU")
FAKE = 0x7F0000000000
P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, ALIGNMENT, CAPACITY, WORKSPACE, CUDA = range(7)


@pytest.fixture(scope="module")
def L():
    _build.build()
    from int2_kv_cache_02_gb300 import oscar
    return oscar.library()


def cache(at=0, **kw):
    from int2_kv_cache_02_gb300.oscar import OscarKV16CacheStruct
    s = OscarKV16CacheStruct()
    s.B, s.Hkv, s.max_blocks, s.n_pages, s.T_cap, s.dtype = 2, 2, 8, 16, 256, 0
    base = FAKE + at
    s.k, s.v, s.weight = base, base + 0x1000000, base + 0x2000000
    s.block_table, s.n_tok = base + 0x3000000, base + 0x4000000
    for name, x in kw.items():
        setattr(s, name, x)
    return s


BAD_CACHES = [(dict(B=0), INVALID), (dict(Hkv=-1), INVALID), (dict(k=None), INVALID),
              (dict(v=None), INVALID), (dict(n_tok=None), INVALID), (dict(dtype=2), INVALID),
              (dict(dtype=-1), INVALID), (dict(max_blocks=0), INVALID), (dict(n_pages=0), INVALID),
              (dict(block_table=None, T_cap=0), INVALID), (dict(k=FAKE + 8), ALIGNMENT),
              (dict(v=FAKE + 2), ALIGNMENT), (dict(weight=FAKE + 4), ALIGNMENT),
              (dict(block_table=FAKE + 2), ALIGNMENT), (dict(n_tok=FAKE + 1), ALIGNMENT),
              (dict(n_pages=2**26), UNSUPPORTED), (dict(max_blocks=2**30), UNSUPPORTED),
              (dict(B=2**16, max_blocks=2**15), UNSUPPORTED),
              (dict(block_table=None, T_cap=2**30), UNSUPPORTED)]


@no_gpu_only
@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_every_call_checks_its_cache(L, bad, status):
    c, good = cache(**bad), cache(at=0x100000000)
    r = ctypes.byref(c)
    x = P(FAKE)
    assert L.oscar_kv16_write(r, x, 256, x, 256, x, x, 4, None) == status
    assert L.oscar_kv16_attention(r, x, 512, x, 4, 4, 1.0, 64, 0, 0, x, None, x, 1 << 30,
                                  None) == status
    assert L.oscar_kv16_decode_attention(r, x, 512, 4, 1.0, 64, 0, 0, 0, x, x, 1 << 30,
                                         None) == status
    assert L.oscar_kv16_accumulate(r, x, 512, x, x, 4, 4, 1.0, 64, 0, 0, 0, None) == status
    assert L.oscar_kv16_evict(r, ctypes.byref(good), 64, 1, 1, 1, None, x, 1 << 30,
                              None) == status
    assert L.oscar_kv16_evict(ctypes.byref(good), r, 64, 1, 1, 1, None, x, 1 << 30,
                              None) == status
    assert L.oscar_kv16_decode_workspace_bytes(r, 4, 64, 0, 0, 0) == 0
    assert L.oscar_kv16_attention_workspace_bytes(r, 4, 4, 64, 0, 0) == 0
    assert L.oscar_kv16_evict_workspace_bytes(r, 64, 1, 1, 1) == 0


@no_gpu_only
def test_write_refusals(L):
    c = cache()
    r, x = ctypes.byref(c), P(FAKE)
    f = lambda k=x, ks=256, v=x, vs=256, st=x, pos=x, n=4: L.oscar_kv16_write(r, k, ks, v, vs, st, pos, n, None)
    assert f(k=None) == f(v=None) == f(st=None) == f(pos=None) == f(n=-1) == INVALID
    assert f(ks=255) == f(vs=128) == f(ks=260) == f(ks=-256) == f(vs=1 << 41) == INVALID
    assert f(k=P(FAKE + 8)) == f(v=P(FAKE + 2)) == f(st=P(FAKE + 2)) == f(pos=P(FAKE + 1)) == ALIGNMENT
    # the lengths are written while the positions and ranges are read
    assert f(pos=P(c.n_tok)) == f(pos=P(c.n_tok + 4)) == f(pos=P(c.n_tok - 4)) == INVALID
    assert f(st=P(c.n_tok - 8)) == INVALID
    assert L.oscar_kv16_write(None, x, 256, x, 256, x, x, 4, None) == INVALID


@no_gpu_only
def test_attention_refusals(L):
    c = cache()
    r, x = ctypes.byref(c), P(FAKE)

    def f(q=x, qs=512, st=x, n=4, Hq=4, scale=1.0, most=64, win=0, sink=0, out=x, lse=None, ws=x, wb=1 << 34):
        return L.oscar_kv16_attention(r, q, qs, st, n, Hq, scale, most, win, sink, out, lse, ws, wb, None)

    assert f(q=None) == f(out=None) == f(st=None) == f(n=-1) == f(qs=511) == f(qs=516) == INVALID
    assert f(scale=float("nan")) == f(scale=float("inf")) == f(most=-1) == f(win=-1) == f(sink=-1) == INVALID
    assert f(Hq=0) == f(Hq=3) == f(Hq=34) == f(Hq=-4) == UNSUPPORTED
    assert f(q=P(FAKE + 8)) == f(out=P(FAKE + 4)) == f(lse=P(FAKE + 2)) == f(st=P(FAKE + 2)) == ALIGNMENT
    assert f(n=2**30) == UNSUPPORTED
    assert f(n=0, q=None, out=None) == OK                 # nothing to do
    need = L.oscar_kv16_attention_workspace_bytes(r, 4, 4, 64, 0, 0)
    if need:
        assert f(ws=None) == f(wb=need - 1) == WORKSPACE


@no_gpu_only
def test_decode_refusals(L):
    c = cache()
    r, x = ctypes.byref(c), P(FAKE)

    def f(ref=r, q=x, qs=512, Hq=4, scale=1.0, most=64, win=0, sink=0, acc=0, out=x, ws=x, wb=1 << 34):
        return L.oscar_kv16_decode_attention(ref, q, qs, Hq, scale, most, win, sink, acc, out, ws, wb, None)

    assert f(q=None) == f(out=None) == f(qs=500) == f(acc=2) == INVALID
    assert f(scale=float("nan")) == f(most=-1) == f(win=-1) == f(sink=-1) == INVALID
    assert f(ref=ctypes.byref(cache(weight=None)), acc=1) == INVALID
    assert f(Hq=3) == f(Hq=0) == f(Hq=64) == UNSUPPORTED
    assert f(ref=ctypes.byref(cache(B=4097))) == UNSUPPORTED
    assert f(ref=ctypes.byref(cache(B=4096, Hkv=17)), qs=34 * 128, Hq=34) == UNSUPPORTED
    assert f(ref=ctypes.byref(cache(B=4000, Hkv=16, max_blocks=2**18)), qs=2048, Hq=16, most=2**23) == UNSUPPORTED
    for acc in (0, 1):
        need = L.oscar_kv16_decode_workspace_bytes(r, 4, 64, 0, 0, acc)
        assert need >= 65536 * 4
        assert f(acc=acc, wb=need - 1) == f(acc=acc, ws=None) == WORKSPACE
        assert f(acc=acc, ws=P(FAKE + 8), wb=need) == ALIGNMENT
    assert f(out=P(FAKE + 8)) == f(q=P(FAKE + 2)) == ALIGNMENT


@no_gpu_only
def test_accumulate_refusals(L):
    c = cache()
    x = P(FAKE)

    def f(c=c, q=x, qs=512, lse=x, st=x, n=4, Hq=4, scale=1.0, most=64, win=0, sink=0, obs=0):
        return L.oscar_kv16_accumulate(ctypes.byref(c), q, qs, lse, st, n, Hq, scale, most, win, sink, obs, None)

    assert f(q=None) == f(lse=None) == f(st=None) == f(n=-1) == f(obs=-1) == f(qs=8) == INVALID
    assert f(c=cache(weight=None)) == f(scale=float("inf")) == f(most=-1) == f(win=-2) == f(sink=-2) == INVALID
    assert f(Hq=5) == UNSUPPORTED
    assert f(q=P(FAKE + 8)) == f(lse=P(FAKE + 2)) == f(st=P(FAKE + 3)) == ALIGNMENT
    assert f(n=0, q=None, lse=None) == f(most=0) == OK


@no_gpu_only
def test_evict_refusals(L):
    src, dst = cache(), cache(at=0x100000000)
    x = P(FAKE + 0x200000000)

    def f(src=src, dst=dst, most=64, first=1, recent=2, top=3, kept=None, ws=x, wb=1 << 34):
        return L.oscar_kv16_evict(ctypes.byref(src), ctypes.byref(dst), most, first, recent, top, kept, ws, wb, None)

    assert f(most=-1) == f(first=-1) == f(recent=-1) == f(top=-1) == INVALID
    assert f(first=0, recent=0, top=0) == f(first=2**30, recent=2**30, top=2**30) == INVALID
    assert f(src=cache(weight=None)) == f(dst=cache(at=1 << 32, B=3)) == INVALID
    assert f(dst=cache(at=1 << 32, Hkv=4)) == f(dst=cache(at=1 << 32, dtype=1)) == INVALID
    assert f(top=300) == CAPACITY
    assert f(dst=src) == INVALID
    for name in ("k", "v", "weight", "n_tok"):            # one shared buffer is enough
        assert f(dst=cache(at=1 << 32, **{name: getattr(src, name)})) == INVALID
    assert f(dst=cache(at=1 << 32, v=src.k + 256)) == INVALID
    assert f(kept=P(FAKE + 2)) == ALIGNMENT
    need = L.oscar_kv16_evict_workspace_bytes(ctypes.byref(src), 64, 1, 2, 3)
    assert need > 0 and f(wb=need - 1) == f(ws=None) == WORKSPACE
    assert f(ws=P(FAKE + 8)) == ALIGNMENT


def test_page_allocator_takes_pages_back():
    """release_blocks frees the pages behind the kept ones, for any sequence."""
    from int2_kv_cache_02_gb300 import oscar as O

    class Pool(O._PagePool):
        def __init__(self):
            self.block_table = torch.full((2, 4), -1, dtype=torch.int32)
            self._init_pool(2, 4, 6)

    p = Pool()
    p.map_blocks(0, 4)
    p.map_blocks(1, 2, order=[5, 4, 3, 2, 1, 0])
    assert p.block_table.tolist() == [[0, 1, 2, 3], [5, 4, -1, -1]] and p._free == []
    with pytest.raises(O.OscarError):
        p.map_blocks(1, 3)
    p.release_blocks(0, 1)
    assert p.block_table[0].tolist() == [0, -1, -1, -1] and sorted(p._free) == [1, 2, 3]
    p.map_blocks(1, 4)
    assert set(p.block_table[1].tolist()[2:]) <= {1, 2, 3} and p.page_of(0, 1) == -1
    p.release_blocks(1)
    assert len(p._free) == 5


def test_cache_takes_fitting_tensors_only():
    from int2_kv_cache_02_gb300 import oscar as O
    k = torch.zeros((4, 2, 32, 128), dtype=torch.bfloat16)
    n, t = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32)
    for bad in (dict(k=k.float(), v=k.float()), dict(v=k[:3]), dict(v=k.half()),
                dict(k=k[:, :, :16], v=k[:, :, :16]), dict(block_table=t[0]),
                dict(k=k[..., :64], v=k[..., :64]), dict(weight=torch.zeros(4, 2, 31))):
        with pytest.raises(ValueError):
            O.KV16Cache(**{**dict(k=k, v=k, n_tok=n, block_table=t), **bad})


@no_gpu_only
def test_output_apart_from_the_queries(L):
    """A row whose result is not finite reads its query again after results
    are written, so an output in the queries' memory is refused."""
    r, x, ws = ctypes.byref(cache()), P(FAKE), P(FAKE + 0x8000000)
    n = 4 * 4 * 128 * 2
    far = P(FAKE + 0x6000000)
    prompt = lambda out, lse=None: L.oscar_kv16_attention(
        r, x, 512, x, 4, 4, 1.0, 64, 0, 0, out, lse, ws, 1 << 30, None)
    assert prompt(x) == prompt(P(FAKE + n - 16)) == prompt(P(FAKE - n + 16)) == INVALID
    assert prompt(far, x) == prompt(far, P(FAKE + n - 4)) == INVALID
    assert prompt(P(FAKE + n)) == prompt(P(FAKE - n)) == prompt(far, P(FAKE + n)) == CUDA
    n = 2 * 4 * 128 * 2
    step = lambda out: L.oscar_kv16_decode_attention(
        r, x, 512, 4, 1.0, 64, 0, 0, 0, out, ws, 1 << 30, None)
    assert step(x) == step(P(FAKE + n - 16)) == step(P(FAKE - n + 16)) == INVALID
    assert step(P(FAKE + n)) == step(P(FAKE - n)) == CUDA


@no_gpu_only
def test_decode_timeout_selftest_refusals(L):
    """The self-test of the decode's waits takes what the decode takes."""
    r, x, out, ws = ctypes.byref(cache()), P(FAKE), P(FAKE + 0x6000000), P(FAKE + 0x8000000)
    f = lambda q=x, Hq=4, most=64, o=out, w=ws, n=1 << 30: L.oscar_selftest_kv16_decode_timeout(
        r, q, Hq, most, o, w, n, None)
    assert f(q=None) == f(o=None) == f(most=-1) == f(o=x) == INVALID
    assert f(Hq=3) == UNSUPPORTED and f(o=P(FAKE + 0x6000008)) == ALIGNMENT
    assert f(w=None) == f(n=100) == WORKSPACE
    assert L.oscar_selftest_kv16_decode_timeout(None, x, 4, 64, out, ws, 1 << 30, None) == INVALID


def test_tc_wait_selftest_refusals(L):
    # rejected on the host before any device call: safe with or without a GPU
    f = L.oscar_selftest_tc_wait_timeout
    assert f(0, P(FAKE), None) == f((1 << 16) + 1, P(FAKE), None) == f(16, None, None) == INVALID
    assert f(16, P(FAKE + 2), None) == ALIGNMENT


def pool_of(kind, B=2, blocks=4, pages=6):
    from int2_kv_cache_02_gb300 import oscar as O
    p = object.__new__(getattr(O, kind))
    p.block_table = torch.full((B, blocks), -1, dtype=torch.int32)
    p._init_pool(B, blocks, pages)
    return p


@pytest.mark.parametrize("kind", ["PagedKVCache", "PagedKV16Cache"])
def test_an_empty_pool_names_its_cache(kind):
    from int2_kv_cache_02_gb300 import oscar as O
    p = pool_of(kind, pages=1)
    with pytest.raises(O.OscarError, match=f"^{kind}.map_blocks: page pool exhausted"):
        p.map_blocks(0, 2)


@pytest.mark.parametrize("kind", ["PagedKVCache", "PagedKV16Cache"])
def test_a_pool_with_too_few_pages_gives_none(kind):
    """The pages stay free and the host's table stays the device's."""
    from int2_kv_cache_02_gb300 import oscar as O
    p = pool_of(kind)
    p.map_blocks(0, 3)
    for n in (4, 5):                            # more than are free, more than a row has
        with pytest.raises((O.OscarError, IndexError)):
            p.map_blocks(1, n)
        assert p._free == [3, 4, 5] and p.block_table[1].tolist() == [-1] * 4
        assert [p.page_of(1, j) for j in range(4)] == [-1] * 4
    p.map_blocks(1, 3)
    assert p.block_table.tolist() == [[0, 1, 2, -1], [3, 4, 5, -1]]


def test_calls_and_sizes_use_the_cache_device(monkeypatch):
    """Every call, those that plan a workspace too, runs with the cache's device
    current and leaves the caller's as it was."""
    import types
    from int2_kv_cache_02_gb300 import oscar as O
    now, seen = [0], []

    class Device:
        def __init__(self, d):
            self.to = torch.device(d).index

        def __enter__(self):
            self.was, now[0] = now[0], self.to

        def __exit__(self, *_):
            now[0] = self.was

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, now[0])) or 0

    monkeypatch.setattr(O, "_lib", Lib())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    for index in (0, 1):
        cache = types.SimpleNamespace(_ref=None, _index=index, device=torch.device("cuda", index))
        O.kv16_attention_workspace_bytes(cache, 4, 4, 64)
        O.kv16_decode_workspace_bytes(cache, 4, 64)
        O.kv16_evict_workspace_bytes(cache, 64, 1, 1, 1)
        O._kv16_call(cache, "call", O._lib.call, (), None)
        assert len(seen) == 4 and all(d == index for _, d in seen) and now == [0]
        seen.clear()
