"""Host-side refusals of the self-test of the shared attention's waits."""
import ctypes

from tests.test_kv16_host import ALIGNMENT, FAKE, INVALID, L, P, UNSUPPORTED, WORKSPACE, cache, no_gpu_only  # noqa: F401


@no_gpu_only
def test_shared_timeout_selftest_refusals(L):
    c, out, ws, x = cache(), P(FAKE + 0x10000000), P(FAKE + 0x20000000), P(FAKE)
    f = lambda q=x, Hq=4, group=x, prefix=x, n=2, most=64, items=0, out=out, w=ws, wb=1 << 30: \
        L.oscar_selftest_kv16_shared_timeout(ctypes.byref(c), q, Hq, group, prefix, n, most, items, out, w, wb, None)
    assert f(q=None) == f(out=None) == f(group=None) == f(prefix=None) == f(n=0) == f(most=-1) == f(items=-1) == INVALID
    assert f(Hq=3) == f(n=4097) == UNSUPPORTED
    assert f(q=P(FAKE + 8)) == f(group=P(FAKE + 2)) == f(w=P(FAKE + 8)) == ALIGNMENT
    assert f(w=None) == f(wb=16) == WORKSPACE
    assert f(out=P(FAKE + 1024)) == INVALID              # in the queries' memory
    assert L.oscar_selftest_kv16_shared_timeout(None, x, 4, x, x, 2, 64, 0, out, ws, 1 << 30, None) == INVALID
