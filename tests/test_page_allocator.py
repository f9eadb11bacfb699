"""The page allocator beside forks by reference, which write the block table on
the device: the host's copy, the counts and the free pages go by what the table
says from then on.  On the CPU: the fork's kernel is replaced by its rule."""
import random

import pytest
import torch

from tests._shared_ref import compacted
from tests.test_kv16_shared_host import L  # noqa: F401


@pytest.fixture
def O(L, monkeypatch):
    from int2_kv_cache_02_gb300 import oscar

    def call(cache, where, fn, args, stream):
        assert where == "oscar_kv16_fork"
        src, dst, parents = call.of
        for b, p in enumerate(parents):
            if p >= 0 and p != b:
                whole = int(src.n_tok[p]) // 32
                dst.block_table[b, :whole] = src.block_table[p, :whole]
                dst.n_tok[b] = src.n_tok[p]

    def plan(table, new, n_pages, moves, counts, workspace, stream=None):
        rows, m, live = compacted(table.tolist(), n_pages)
        new.copy_(torch.tensor(rows, dtype=torch.int32))
        moves.fill_(-1)
        moves[:len(m)] = torch.tensor(m, dtype=torch.int32).view(-1, 2)
        counts.copy_(torch.tensor([len(m), live], dtype=torch.int32))

    def fork(src, dst, parents):
        call.of = (src, dst, parents)
        oscar.kv16_fork(src, dst, torch.tensor(parents, dtype=torch.int32), 1000)

    monkeypatch.setattr(oscar, "_ptr", lambda t: t.data_ptr())      # (takes host tensors too)
    monkeypatch.setattr(oscar, "_kv16_call", call)
    monkeypatch.setattr(oscar, "page_compact", plan)
    oscar.fork_here = fork
    yield oscar
    del oscar.fork_here


def pool_of(O, B, blocks, pages, lens):
    pool = O.PagedKV16Cache(B, 1, blocks, pages, device="cpu")
    for b, n in enumerate(lens):
        pool.map_blocks(b, -(-n // 32))
        pool.n_tok[b] = n
    return pool


def check(pool):
    """The table, its copy, the counts and the free pages agree."""
    rows = pool.block_table.tolist()
    assert rows == pool._table_host
    named = [p for row in rows for p in row if p >= 0]
    assert pool._named == [named.count(p) for p in range(len(pool._named))]
    assert sorted(pool._free) == [p for p in range(len(pool._named)) if p not in named]


def test_more_blocks_for_a_forked_sequence(O):
    pool = pool_of(O, 2, 6, 16, [100, 100])
    O.fork_here(pool, pool, [-1, 0])
    assert pool.block_table[1].tolist() == [0, 1, 2, 7, -1, -1]
    pool.map_blocks(1, 5)
    assert pool.block_table[1].tolist() == [0, 1, 2, 7, 8, -1]
    check(pool)
    assert {4, 5, 6} <= set(pool._free)          # what the fork took the place of


def test_the_parents_pages_stay_while_a_fork_names_them(O):
    pool = pool_of(O, 3, 6, 16, [100, 100])
    O.fork_here(pool, pool, [-1, 0, -1])
    pool.release_blocks(0)
    pool.map_blocks(2, 6)
    check(pool)
    assert not {0, 1, 2} & set(pool.block_table[2].tolist()) and not {0, 1, 2} & set(pool._free)
    pool.release_blocks(1)
    check(pool)
    assert {0, 1, 2} <= set(pool._free)


def test_page_of_a_forked_sequence(O):
    pool = pool_of(O, 2, 6, 16, [100, 100])
    O.fork_here(pool, pool, [-1, 0])
    assert [pool.page_of(1, j) for j in range(5)] == [0, 1, 2, 7, -1]


def test_compaction_behind_a_fork(O):
    pool = pool_of(O, 3, 6, 16, [100, 100, 64])
    O.fork_here(pool, pool, [1, -1, -1])
    moves, counts = pool.compact()
    check(pool)
    # 0 has 1's first three pages and its own last
    assert counts.tolist() == [3, 7] and moves.tolist()[:3] == [[7, 0], [8, 1], [9, 2]]


def test_sequences_that_change_places(O):
    """Forked from a cache that has the lengths and the table as they were."""
    pool = pool_of(O, 2, 4, 16, [64, 96])
    before = O.KV16Cache(pool.k, pool.v, pool.n_tok.clone(), block_table=pool.block_table.clone())
    O.fork_here(before, pool, [1, 0])
    pool.map_blocks(0, 4)
    assert pool.block_table.tolist() == [[2, 3, 4, 5], [0, 1, 4, -1]]
    check(pool)


@pytest.mark.parametrize("seed", range(20))
def test_any_order_of_calls(O, seed):
    rng = random.Random(seed)
    pool = pool_of(O, 4, 5, 60, [])
    for _ in range(30):
        b, what = rng.randrange(4), rng.randrange(5)
        if what == 0:
            pool.map_blocks(b, rng.randint(0, 5))
        elif what == 1:
            pool.release_blocks(b, rng.randint(0, 3))
        elif what == 2:
            p = rng.randrange(4)
            pool.share_blocks(b, p, rng.randint(0, sum(x >= 0 for x in pool.block_table[p].tolist())))
        elif what == 3:
            pool.compact()
        else:
            p = rng.randrange(4)
            row = pool.block_table[p].tolist()
            pool.n_tok[p] = 32 * (row + [-1]).index(-1)
            O.fork_here(pool, pool, [p if i == b else -1 for i in range(4)])
            continue
        check(pool)


def test_calls_that_do_not_share_leave_the_copy_alone(O, monkeypatch):
    """What no sharing fork has written is not read back."""
    pool = pool_of(O, 2, 6, 16, [100, 100])
    monkeypatch.setattr(O, "_kv16_call", lambda *a: None)
    O.kv16_fork(pool, pool, torch.tensor([-1, 0], dtype=torch.int32), 1000, share=False)
    rows = pool._table_host
    pool.page_of(0, 0)
    assert pool._table_host is rows
