"""The page allocator beside forks by reference on the GPU: tokens stay where
their sequences read them, whatever is mapped, released and compacted next."""
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


def filled(L, lens, B, blocks=8, n_pages=48):
    """A pool whose first sequences hold tokens, and the tokens."""
    case = R.Case(lens, 2, BF, seed=len(lens))
    pool = L.PagedKV16Cache(B, 2, blocks, n_pages, dtype=BF)
    for b, n in enumerate(lens):
        pool.map_blocks(b, -(-n // 32))
    k, v = (torch.cat([x[b].transpose(0, 1) for b in range(len(lens))]).cuda() for x in (case.k, case.v))
    start = R.start_of(lens)
    L.kv16_write(pool, k, v, i32(start + [start[-1]] * (B - len(lens))), i32([0] * B))
    return case, pool


def assert_tokens(pool, case, b, of, n):
    for x in ("k", "v"):
        assert torch.equal(bits(R.tokens(pool, b, n, x).cpu()), bits(getattr(case, x)[of][:, :n]))


def agrees(pool):
    rows = pool.block_table.tolist()
    named = [p for row in rows for p in row if p >= 0]
    assert rows == pool._table_host and sorted(pool._free) == sorted(set(range(len(pool._named))) - set(named))
    assert pool._named == [named.count(p) for p in range(len(pool._named))]


def grow(L, pool, b, n):
    """n more tokens for sequence b, of which nothing else may see a trace."""
    k, v = torch.full((2, n, 2, 128), 9.0, dtype=BF, device="cuda")
    pool.map_blocks(b, -(-(int(pool.n_tok[b]) + n) // 32))
    L.kv16_write(pool, k, v, i32([0] * (b + 1) + [n] * (pool.B - b)), pool.n_tok.clone())


@pytest.mark.parametrize("stream", [False, True])
def test_fork_then_map_release_and_compact(L, stream):
    case, pool = filled(L, [150, 100], 4)
    pool.map_blocks(2, 5)
    pool.map_blocks(3, 5)
    s = None
    if stream:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
    L.kv16_fork(pool, pool, i32([-1, -1, 0, 1]), 256, stream=s)
    grow(L, pool, 2, 70)
    agrees(pool)
    for b, of, n in ((0, 0, 150), (1, 1, 100), (2, 0, 150), (3, 1, 100)):
        assert_tokens(pool, case, b, of, n)
    pool.release_blocks(0)
    pool.n_tok[0] = 0
    grow(L, pool, 0, 230)                    # wherever there is room: not where 2 reads
    agrees(pool)
    for b, of, n in ((1, 1, 100), (2, 0, 150), (3, 1, 100)):
        assert_tokens(pool, case, b, of, n)
    pool.map_blocks(3, 7)                    # a place for the last page of 2's 220 tokens
    L.kv16_fork(pool, pool, i32([-1, -1, -1, 2]), 256)
    pool.release_blocks(1)
    pool.n_tok[1] = 0
    moves, counts = pool.compact()
    L.kv16_copy_pages(pool, pool, moves, counts)
    agrees(pool)
    assert int(counts[1]) == len({p for row in pool._table_host for p in row if p >= 0})
    assert L.device_status() == 0
    for b in (2, 3):
        assert_tokens(pool, case, b, 0, 150)


def test_a_captured_fork(L):
    """Replays write the table again: the allocator looks every time."""
    case, pool = filled(L, [150, 100], 3)
    pool.map_blocks(2, 5)
    parent = i32([-1, -1, -1])
    L.kv16_fork(pool, pool, parent, 256)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.kv16_fork(pool, pool, parent, 256)
    pool.map_blocks(2, 5)
    for of, n in ((0, 150), (1, 100), (0, 150)):
        parent[2] = of
        pool.release_blocks(2)               # (pages of its own again, for the last tokens)
        pool.map_blocks(2, 6)
        g.replay()
        pool.map_blocks(2, 6)
        agrees(pool)
        assert_tokens(pool, case, 0, 0, 150)
        assert_tokens(pool, case, 1, 1, 100)
        assert_tokens(pool, case, 2, of, n)
        assert pool._table_host[2][:n // 32] == pool._table_host[of][:n // 32]
    assert L.device_status() == 0


@pytest.mark.parametrize("call", [lambda p: p.compact(), lambda p: p.map_blocks(0, 6), lambda p: p.release_blocks(0, 2),
                                  lambda p: p.share_blocks(1, 0, 2)])
def test_not_in_a_captured_graph(L, call):
    """What a graph would replay on the device alone is refused, and changes nothing."""
    _, pool = filled(L, [150, 100], 2)
    before = ([list(r) for r in pool._table_host], list(pool._free), list(pool._named))
    with pytest.raises(RuntimeError, match="captured graph"), torch.cuda.graph(torch.cuda.CUDAGraph()):
        call(pool)
    torch.cuda.synchronize()
    assert before == (pool._table_host, pool._free, pool._named)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        assert pool.page_of(0, 0) == before[0][0][0]
    agrees(pool)


def test_steps_of_a_beam_search(L):
    """Beams that continue one another, through the allocator: whole pages by reference,
    the last one copied to a page that was free, one more token each, and again."""
    lens, B, rng = [100, 70, 64, 33], 4, torch.Generator().manual_seed(3)
    case, pool = filled(L, lens, B, blocks=8, n_pages=24)
    history = [[x[b].clone() for x in (case.k, case.v)] for b in range(B)]
    for parents in ([1, 0, 0, 2], [3, 3, 1, 0], [0, 1, 2, 3], [2, 2, 2, 2], [1, 0, 3, 2]):
        n = [history[p][0].shape[1] for p in parents]
        before = L.KV16Cache(pool.k, pool.v, pool.n_tok.clone(), block_table=pool.block_table.clone())
        for b in range(B):
            pool.release_blocks(b, min(n[b], int(before.n_tok[b])) // 32)
        for b in range(B):
            pool.map_blocks(b, n[b] // 32 + 1)
        L.kv16_fork(before, pool, i32(parents), 256)
        k, v = (torch.randn((B, 2, 128), generator=rng).to(BF) for _ in range(2))
        L.kv16_write(pool, k.cuda(), v.cuda(), i32([0, 1, 2, 3, 4]), pool.n_tok.clone())
        history = [[torch.cat((x, y[b][:, None]), 1) for x, y in zip(history[p], (k, v))] for b, p in enumerate(parents)]
        pool.page_of(0, 0)
        agrees(pool)
        assert L.device_status() == 0
        for b in range(B):
            for x, want in zip(("k", "v"), history[b]):
                assert torch.equal(bits(R.tokens(pool, b, n[b] + 1, x).cpu()), bits(want))
