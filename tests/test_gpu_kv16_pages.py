"""Forks of sequences, compaction of a page pool and copies of pages, on the GPU:
whole numbers and copies, so everything is compared bit for bit with a plain
form; and a run of all calls together, as a server makes them."""
import math
import random

import pytest
import torch

from tests import _kv16_ref as R
from tests._shared_ref import SharedCase, bits, compacted, i32

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def L():
    from int2_kv_cache_02_gb300 import _build
    _build.build()
    from int2_kv_cache_02_gb300 import oscar
    oscar.device_status()
    return oscar


def place(cache, b, t):
    if cache.block_table is None:
        return b, slice(None), t
    return int(cache.block_table[b, t // 32]), slice(None), t % 32


def forked(src, dst, parent, share):
    """What a fork leaves: (k, v, weight, n_tok, table) of dst, by loops."""
    k, v = dst.k.clone(), dst.v.clone()
    w = dst.weight.clone() if dst.weight is not None else None
    n_tok = dst.n_tok.clone()
    table = dst.block_table.clone() if dst.block_table is not None else None
    for b, p in enumerate(parent):
        if p < 0:
            continue
        n = int(src.n_tok[p])
        n_tok[b] = n
        whole = n // 32 if share else 0
        if whole:
            table[b, :whole] = src.block_table[p, :whole]
        for t in range(whole * 32, n):
            s, d = place(src, p, t), place(dst, b, t)
            k[d], v[d] = src.k[s], src.v[s]
            if w is not None:
                w[d] = src.weight[s]
    return k, v, w, n_tok, table


def assert_cache(cache, want):
    for name, x, y in zip(("k", "v", "weight", "n_tok", "block_table"),
                          (cache.k, cache.v, cache.weight, cache.n_tok, cache.block_table), want):
        assert (x is None) == (y is None), name
        assert x is None or torch.equal(bits(x), bits(y)), name


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("Hkv,lens,parent", [
    (1, [1], [0]), (2, [31, 32, 33], [2, 1, 0, 0, 1, 2]), (8, [0, 70, 64], [1, 0, -1, 2, 1]),
    (3, [300, 5], [0] * 9 + [-1, 1]), (5, [95], [-1, -1])])
def test_fork_shares_pages(L, Hkv, lens, parent, weights, dtype):
    """Whole pages by reference, the last page's tokens copied to the page that the
    table names; sequences without a parent, other entries and pages stay."""
    case = R.Case(lens, Hkv, dtype, weights=weights)
    src = case.cache(L)
    B, wide = len(parent), src.block_table.shape[1] + 1
    spare = src.k.shape[0]
    grow = lambda x: torch.cat((x, torch.full((B + 2,) + x.shape[1:], math.nan, dtype=x.dtype, device="cuda"))) if x is not None else None
    k, v, w = grow(src.k), grow(src.v), grow(src.weight)
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    table[:, wide - 1] = 12345
    for b, p in enumerate(parent):
        if p >= 0:
            table[b, lens[p] // 32] = spare + b
    src = L.KV16Cache(k, v, src.n_tok, block_table=src.block_table, weight=w)
    dst = L.KV16Cache(k, v, i32([77] * B), block_table=table, weight=w)
    want = forked(src, dst, parent, True)
    L.kv16_fork(src, dst, i32(parent), 320)
    assert L.device_status() == 0
    assert_cache(dst, want)
    L.kv16_fork(src, dst, i32(parent), max(lens))
    assert L.device_status() == 0
    assert_cache(dst, want)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("from_paged", [True, False])
@pytest.mark.parametrize("to_paged", [True, False])
@pytest.mark.parametrize("weights,to_weights", [(True, True), (True, False), (False, False)])
def test_fork_copies(L, from_paged, to_paged, weights, to_weights, dtype):
    """Every token copied, between the layouts; what lies behind a length stays."""
    lens, parent = [0, 1, 33, 200, 64], [3, 3, -1, 2, 0, 4, 1]
    src = R.Case(lens, 3, dtype, from_paged, weights=weights).cache(L)
    dst = R.Case([200] * len(parent), 3, dtype, to_paged, seed=1, weights=to_weights).cache(L)
    want = forked(src, dst, parent, False)
    L.kv16_fork(src, dst, i32(parent), 200, share=False)
    assert L.device_status() == 0
    assert_cache(dst, want)


def test_fork_within_a_cache(L):
    """One cache on both sides: free slots filled from a running sequence; a block whose
    page is the parent's own stays; a sequence forked from and to is refused."""
    case = R.Case([100, 70, 40, 9], 2)
    cache = case.cache(L)
    cache.block_table[3, 3] = cache.block_table[0, 3]      # the parent's own last page
    parent = [-1, -1, 0, 0]
    want = forked(cache, cache, parent, True)
    L.kv16_fork(cache, cache, i32(parent), 128)
    assert L.device_status() == 0
    assert_cache(cache, want)
    assert torch.equal(bits(R.tokens(cache, 2, 100)), bits(case.k[0]))
    want = forked(cache, cache, [1, -1, -1, -1], True)
    L.kv16_fork(cache, cache, i32([1, -1, -1, 3]), 128)     # 3 from itself: nothing
    assert L.device_status() == 0
    assert_cache(cache, want)
    cache = case.cache(L)
    before = forked(cache, cache, [-1] * 4, True)
    L.kv16_fork(cache, cache, i32([1, 0, -1, -1]), 128)     # each of the other
    assert L.device_status() != 0 and L.device_status() == 0
    assert_cache(cache, before)


def test_fork_bad_parents_lengths_and_pages(L):
    """Each is recorded and leaves its sequence as it was; the others are made."""
    case = R.Case([40, 70, 40], 2)
    for spoil in ("parent", "length", "most", "capacity", "page"):
        src = case.cache(L)
        dst = R.Case([32] * 3 if spoil == "capacity" else [96] * 3, 2, seed=2, slack=0).cache(L)
        parent, most = [0, 2, 1], 96
        if spoil == "parent":
            parent[2] = 3
        elif spoil == "length":
            src.n_tok[1] = -5
        elif spoil == "most":
            most = 69
        elif spoil == "page":
            dst.block_table[2, 1] = 99999
        want = forked(src, dst, [0 if spoil != "capacity" else -1, 2 if spoil != "capacity" else -1, -1], False)
        L.kv16_fork(src, dst, i32(parent), most, share=False)
        assert L.device_status() != 0 and L.device_status() == 0
        if spoil != "page":
            assert_cache(dst, want)
        else:
            for b in (0, 1):
                assert torch.equal(bits(R.tokens(dst, b, 40)), bits(case.k[parent[b]]))


def test_fork_does_not_take_over_unmapped_pages(L):
    """A whole page that the parent's table does not name is recorded, and the entry stays."""
    case = R.Case([70, 40], 2)
    cache = case.cache(L)
    cache.block_table[0, 1] = -1
    before = cache.block_table.clone()
    dst = L.KV16Cache(cache.k, cache.v, i32([0, 0]), block_table=before.flip(0).contiguous())
    other = dst.block_table.clone()
    L.kv16_fork(cache, dst, i32([0, -1]), 128)
    assert L.device_status() != 0 and L.device_status() == 0
    other[0, 0] = before[0, 0]
    assert torch.equal(dst.block_table, other) and dst.n_tok.tolist() == [70, 0]


# -------------------------------------------------------------- compaction

def random_table(rng, B, blocks, n_pages, mapped, shared=0.2):
    free = rng.sample(range(n_pages), n_pages)
    table = [[-1] * blocks for _ in range(B)]
    for b in range(B):
        for j in range(blocks):
            if rng.random() < mapped:
                if b and rng.random() < shared and table[b - 1][j] >= 0:
                    table[b][j] = table[b - 1][j]
                elif free:
                    table[b][j] = free.pop()
    return table


def run_compact(L, table, n_pages, in_place=False):
    t = table.cuda() if torch.is_tensor(table) else i32(table)
    new = t if in_place else torch.full_like(t, 7)
    moves = torch.full((n_pages // 2, 2), 7, dtype=torch.int32, device="cuda")
    counts = i32([7, 7])
    ws = L.alloc_workspace(L.page_compact_workspace_bytes(t, n_pages))
    ws.fill_(math.nan)
    L.page_compact(t, new, n_pages, moves, counts, ws)
    return t, new, moves, counts


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,blocks,n_pages,mapped", [
    (1, 1, 1, 1.0), (1, 1, 1, 0.0), (1, 1, 2, 1.0), (2, 3, 7, 0.5), (3, 40, 150, 0.9), (3, 40, 150, 0.1),
    (1, 33, 33, 1.0), (7, 31, 1023, 0.8), (7, 300, 1025, 0.5), (64, 257, 9000, 0.4), (64, 257, 70000, 0.9),
    (5, 1000, 300001, 0.9)])
def test_compact(L, B, blocks, n_pages, mapped, in_place):
    rng = random.Random(B * 1000 + n_pages)
    table = random_table(rng, B, blocks, n_pages, mapped)
    old, new, moves, counts = run_compact(L, table, n_pages, in_place)
    assert L.device_status() == 0
    want, want_moves, live = compacted(table, n_pages)
    assert counts.tolist() == [len(want_moves), live]
    assert new.tolist() == want
    assert moves.tolist() == want_moves + [[-1, -1]] * (n_pages // 2 - len(want_moves))
    if not in_place:
        assert old.tolist() == table


def test_compact_large_pool(L):
    """More pages than one block of threads holds at a time, sparse and dense."""
    gen = torch.Generator().manual_seed(5)
    for n_pages, live in ((3_000_001, 1000), (3_000_001, 2_500_000), (12_582_912, 70_000)):
        ids = torch.randperm(n_pages, generator=gen)[:live].int()
        table = torch.full((2, (live + 1) // 2 + 3), -1, dtype=torch.int32)
        table.view(-1)[:live] = ids
        old, new, moves, counts = run_compact(L, table, n_pages)
        assert L.device_status() == 0
        n = int(counts[0])
        named = torch.zeros(n_pages, dtype=torch.bool)
        named[ids.long()] = True
        src, dst = torch.nonzero(named[live:])[:, 0] + live, torch.nonzero(~named[:live])[:, 0]
        assert counts.tolist() == [len(src), live]
        assert torch.equal(moves[:n].cpu().long(), torch.stack((src, dst), 1))
        assert (moves[n:] == -1).all()
        to = torch.arange(n_pages)
        to[src] = dst
        want = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table)
        assert torch.equal(new.cpu(), want)


def test_compact_bad_entries(L):
    """Entries past the pool are recorded and stay; negative ones name no page."""
    table = [[5, 9, -7], [-1, 100, 3]]
    _, new, moves, counts = run_compact(L, table, 9)
    assert L.device_status() != 0 and L.device_status() == 0
    assert new.tolist() == [[1, 9, -7], [-1, 100, 0]]
    assert counts.tolist() == [2, 2] and moves.tolist() == [[3, 0], [5, 1], [-1, -1], [-1, -1]]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("weights", [True, False])
def test_copy_pages(L, Hkv, dtype, weights):
    """Within a pool and into another; pairs behind the count are not looked at, bad ones skipped."""
    a = R.Case([32 * 40], Hkv, dtype, weights=weights).cache(L)
    b = R.Case([32 * 50], Hkv, dtype, weights=weights, seed=1).cache(L)
    pairs = [[3, 11], [39, 0], [5, 10], [1 << 30, 2], [2, 1 << 30], [7, 9], [7, 8]]
    names = ("k", "v") + (("weight",) if weights else ())
    for dst in (a, b):
        for n in (0, 3, 6):
            want = [getattr(dst, x).clone() for x in names]
            for s, d in pairs[:n]:
                if max(s, d) < 1 << 30:
                    for x, w in zip(names, want):
                        w[d] = getattr(a, x)[s]
            L.kv16_copy_pages(a, dst, i32(pairs), i32([n, 99]))
            assert (L.device_status() != 0) == (n > 3)
            for x, w in zip(names, want):
                assert torch.equal(bits(getattr(dst, x)), bits(w))
    want = a.k.clone()
    for n in (-1, 8):
        L.kv16_copy_pages(a, a, i32(pairs), i32([n]))
        assert L.device_status() != 0
        assert torch.equal(bits(a.k), bits(want))


@pytest.mark.parametrize("bits_", [2, 4])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_packed_pages_are_compacted(L, Hkv, bits_):
    """A packed cache's pool after a sequence has ended: the others' records are where
    the table says, bit for bit, and nothing else has moved."""
    cache = L.PagedKVCache(4, Hkv, 6, 40, bits=bits_)
    cache.pages.copy_(torch.randint(0, 256, cache.pages.shape, dtype=torch.uint8))
    for b, n in enumerate((5, 2, 6, 3)):
        cache.map_blocks(b, n, order=random.Random(b).sample(range(40), 40))
    cache.share_blocks(3, 0, 2)
    cache.release_blocks(1)
    cache.release_blocks(2, 4)
    blocks = {0: 5, 2: 4, 3: 3}
    want = {(b, j): cache.pages[cache.page_of(b, j)].clone() for b, n in blocks.items() for j in range(n)}
    before = cache.pages.clone()
    moves, counts = cache.compact()
    L.paged_copy_pages(cache, moves, counts)
    assert L.device_status() == 0
    live = len({x for row in cache._table_host for x in row if x >= 0})
    assert counts[1] == live and cache.block_table.tolist() == cache._table_host
    for (b, j), page in want.items():
        assert cache.page_of(b, j) < live
        assert torch.equal(cache.pages[cache.page_of(b, j)], page)
    assert torch.equal(cache.pages[live:], before[live:])
    L.paged_copy_pages(cache, i32([[1, 100], [2, 39]]), i32([2]))
    assert L.device_status() != 0 and L.device_status() == 0
    assert torch.equal(cache.pages[39], cache.pages[2])
    with pytest.raises(ValueError):
        L.paged_copy_pages(cache, moves.long(), counts)


# ------------------------------------------------- all calls, as a server's

def test_a_run_of_them(L):
    """A prompt is written, forked to samples, which grow by decode steps that read
    the prompt once; some end, the pool is compacted into the lowest pages, and the
    remaining samples go on with the same results; then they are drafted for."""
    Hkv, Hq, P, S = 2, 8, 150, 6
    case = R.Case([P + 60] * S, Hkv, seed=4)
    for b in range(1, S):      # one prompt
        case.k[b][:, :P], case.v[b][:, :P] = case.k[0][:, :P], case.v[0][:, :P]
    pool = L.PagedKV16Cache(S, Hkv, 8, 64, dtype=BF)
    pool.map_blocks(0, 8, order=list(range(40, 64)) + list(range(40)))
    put = lambda b, t0, t1: [x[b][:, t0:t1].transpose(0, 1).contiguous().cuda() for x in (case.k, case.v)]
    k, v = put(0, 0, P)
    L.kv16_write(pool, k, v, i32([0] + [P] * S), i32([0] * S))
    # samples 1.. share the prompt's whole pages; their own begin with its last
    for b in range(1, S):
        pool.share_blocks(b, 0, P // 32)
        pool.map_blocks(b, 8)
    L.kv16_fork(pool, pool, i32([-1] + [0] * (S - 1)), P)
    group, prefix = i32([0, S]), i32([P])
    ws = L.alloc_workspace(max(L.kv16_shared_decode_workspace_bytes(pool, Hq, 1, 256),
                               L.kv16_shared_attention_workspace_bytes(pool, Hq, 1, 3 * S, 256)))
    out = torch.empty((S, Hq, 128), dtype=BF, device="cuda")

    def step(t, live):
        k, v = (torch.stack([x[b][:, t] for b in live]).cuda() for x in (case.k, case.v))
        start = [0]
        for b in range(S):
            start.append(start[-1] + (b in live))
        L.kv16_write(pool, k, v, i32(start), i32([t if b in live else 0 for b in range(S)]))
        q = case.normal(S, Hq)
        L.kv16_shared_decode_attention(pool, q.cuda(), group, prefix, R.SCALE, 256, out, ws)
        assert L.device_status() == 0
        for b in live:
            o, _, _, tol, _, _ = R.attend(case, b, q[b:b + 1], lens=[t + 1] * S)
            R.assert_within(out[b:b + 1], o, tol, f"step {t}, sequence {b}")

    for t in range(P, P + 45):
        step(t, range(S))
    live = [0, 2, 5]
    for b in (1, 3, 4):
        pool.release_blocks(b)
    held = {b: [R.tokens(pool, b, P + 45, x).clone() for x in ("k", "v")] for b in live}
    named = len({x for row in pool._table_host for x in row if x >= 0})
    moves, counts = pool.compact()
    L.kv16_copy_pages(pool, pool, moves, counts)
    assert L.device_status() == 0
    assert counts[1] == named and int(pool.block_table.max()) == named - 1
    assert pool.block_table.tolist() == pool._table_host
    assert sorted(pool._free) == list(range(named, 64))
    for b in live:
        for x, was in zip(("k", "v"), held[b]):
            assert torch.equal(bits(R.tokens(pool, b, P + 45, x)), bits(was))
    for t in range(P + 45, P + 50):
        step(t, live)
    # three drafted tokens each, verified at once
    news, t = [3 if b in live else 0 for b in range(S)], P + 50
    k, v = (torch.cat([x[b][:, t:t + 3].transpose(0, 1) for b in live]).cuda() for x in (case.k, case.v))
    start = R.start_of(news)
    L.kv16_write(pool, k, v, i32(start), i32([t if b in live else 0 for b in range(S)]))
    q = case.normal(start[-1], Hq)
    got = torch.empty((start[-1], Hq, 128), dtype=BF, device="cuda")
    L.kv16_shared_attention(pool, q.cuda(), i32(start), group, prefix, R.SCALE, 256, got, ws)
    assert L.device_status() == 0
    for b in live:
        rows = slice(start[b], start[b + 1])
        o, _, _, tol, _, _ = R.attend(case, b, q[rows], lens=[t + 3] * S)
        R.assert_within(got[rows], o, tol, f"drafts of {b}")


def test_fork_and_compact_in_graphs(L):
    """Captured, and replayed with other parents, lengths and tables."""
    case = R.Case([100, 70], 2)
    src = case.cache(L)
    dst = R.Case([100] * 4, 2, seed=3).cache(L)
    parent = i32([0, 1, 0, -1])
    table, n_pages = i32([[5, 3, -1], [9, 3, 1]]), 12
    new, moves, counts = torch.empty_like(table), i32([[0, 0]] * 6), i32([0, 0])
    ws = L.alloc_workspace(L.page_compact_workspace_bytes(table, n_pages))

    def calls():
        L.kv16_fork(src, dst, parent, 128, share=False)
        L.page_compact(table, new, n_pages, moves, counts, ws)

    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for par, rows in (([1, 0, -1, 0], [[11, 10, 9], [8, 7, 6]]), ([-1, -1, 1, 1], [[0, 1, 2], [0, 1, 2]])):
        parent.copy_(i32(par))
        table.copy_(i32(rows))
        want = forked(src, dst, par, False)
        g.replay()
        torch.cuda.synchronize()
        assert L.device_status() == 0
        assert_cache(dst, want)
        t, m, live = compacted(rows, n_pages)
        assert new.tolist() == t and counts.tolist() == [len(m), live]
        assert moves.tolist()[:len(m)] == m


def test_bindings_check_their_tensors(L):
    """Types, shapes and places that the binding refuses before it calls."""
    t = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    moves, counts, ws = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(64, device="cuda")
    for bad in (moves[:3], moves.long(), moves.cpu(), moves.t().contiguous().t()):
        with pytest.raises(ValueError):
            L.page_compact(t, t, 8, bad, counts, ws)
    with pytest.raises(ValueError):
        L.page_compact(t, t[:1], 8, moves, counts, ws)
    k = torch.zeros((8, 2, 32, 128), dtype=torch.bfloat16, device="cuda")
    c = L.KV16Cache(k, k.clone(), torch.zeros(2, dtype=torch.int32, device="cuda"), block_table=t)
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    group = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (dict(group=n), dict(group=group.long()), dict(prefix=n.float()), dict(out=q[:1]), dict(q=q.half())):
        kw = {**dict(q=q, group=group, prefix=n, out=q.clone()), **bad}
        with pytest.raises(ValueError):
            L.kv16_shared_decode_attention(c, kw["q"], kw["group"], kw["prefix"], 1.0, 64, kw["out"], ws)
        with pytest.raises(ValueError):
            L.kv16_shared_attention(c, kw["q"], torch.zeros(3, dtype=torch.int32, device="cuda"), kw["group"], kw["prefix"], 1.0, 64, kw["out"], ws)
    with pytest.raises(ValueError):
        L.kv16_fork(c, c, n, 64)
    with pytest.raises(ValueError):
        L.kv16_copy_pages(c, c, n, n)
    with pytest.raises(ValueError):
        L.kv16_copy_pages(c, c, moves.long(), n)
