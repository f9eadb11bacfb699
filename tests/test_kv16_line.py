"""The line of work of the attention over shared prefixes, on the host: the
kernels' own arithmetic, compiled as plain C++.  Every tile of every row is one
CTA's, each CTA has at most one run for each of its two places for records, and
who joins a row's records finds the runs that have written them."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HARNESS = r"""
#include "kv16_line.h"
using namespace oscar;
extern "C" {
int row_cost_(int kind) { return row_cost(kind); }
int tile_cost_(int kind) { return tile_cost(kind); }
int share(int places, int ctas) { return line_share(places, ctas); }
int count(int tiles, int chunks, int kind, int per) { return Blocks(tiles, chunks, kind, per).count; }
int first(int tiles, int chunks, int kind, int per, int i) { return Blocks(tiles, chunks, kind, per).first(i); }
int place(int t, int kind) { return tile_place(t, kind); }
int before(int x, int kind) { return tiles_before(x, kind); }
int places(int tiles, int kind) { return row_places(tiles, kind); }
int runs(unsigned at, unsigned more, unsigned per, int ctas) {
  const Runs r = runs_of(at, more, per, ctas);
  return r.c0 | r.n << 16;
}
int block_runs() { return kBlockRuns; }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("line")
    src, so = d / "line.cpp", d / "line.so"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "int2_kv_cache_02_gb300", "csrc"), str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def draw_entries(rng):
    """Groups (chunks, tiles, kind) and sequences [(tiles, kind) of each chunk]."""
    groups, seqs = [], []
    for _ in range(rng.randint(1, 4)):
        chunks = rng.choice([1, 1, 2, 3, 7])
        groups.append((chunks, rng.choice([0, 1, 2, 5, 17, 60, 200, 2000]),
                       (chunks > 1 or rng.random() < 0.5) + 2 * (rng.random() < 0.3)))
    for _ in range(rng.randint(1, 9)):
        n = rng.choice([1, 1, 2, 3])
        rows = [(rng.randint(0, 6) + 3 * i, True) for i in range(n)]
        if rng.random() < 0.7:
            rows[-1] = (rows[-1][0], False)
        seqs.append(rows)
    return groups, seqs


def pieces(lib, groups, seqs, heads, ctas):
    """What the kernel's CTAs work: (entry, head, chunk) -> {tile: (CTA, record place)}."""
    first = [0]
    for chunks, tiles, kind in groups:
        first.append(first[-1] + heads * chunks * lib.places(tiles, kind))
    for rows in seqs:
        first.append(first[-1] + heads * sum(lib.places(t, p) for t, p in rows))
    total = first[-1]
    per = lib.share(total, ctas)
    done, taken = {}, set()
    for cta in range(ctas):
        x, x1 = min(cta * per, total), min(cta * per + per, total)
        while x < x1:
            e = next(i for i in range(len(first) - 1) if first[i] <= x < first[i + 1])
            at = x - first[e]
            if e < len(groups):
                chunks, tiles, kind = groups[e]
                to, p0, chunk = lib.places(tiles, kind), 0, 0
                if chunks == 1:
                    head, start = divmod(at, to)
                else:
                    head, y = divmod(at, chunks * to)
                    t = max(y // chunks - lib.row_cost_(kind), 0) // lib.tile_cost_(kind)
                    n = lib.count(tiles, chunks, kind, per)
                    least = lib.first(tiles, chunks, kind, per, 1)
                    i = min(t // least, n - 1)
                    p0 = lib.place(lib.first(tiles, chunks, kind, per, i), kind)
                    if i + 1 < n:
                        to = lib.place(lib.first(tiles, chunks, kind, per, i + 1), kind)
                    y -= chunks * p0
                    chunk = min(y // (to - p0), chunks - 1)
                    start = p0 + y - chunk * (to - p0)
                where = "row" if start <= lib.row_cost_(kind) else 1 if start > p0 else 2
            else:
                rows = seqs[e - len(groups)]
                head, start = divmod(at, (first[e + 1] - first[e]) // heads)
                chunk = 0
                while start >= lib.places(*rows[chunk]):
                    start -= lib.places(*rows[chunk])
                    chunk += 1
                tiles, kind = rows[chunk]
                to = lib.places(tiles, kind)
                where = "row" if start <= lib.row_cost_(kind) else 1
            end = min(start + x1 - x, to, start + first[e + 1] - x)
            k0, k1 = lib.before(start, kind), lib.before(end, kind)
            row = (e, head, chunk)
            if k1 > k0:
                place = ("row", row) if where == "row" else (cta, where)
                assert place not in taken
                taken.add(place)
                for k in range(k0, k1):
                    assert (row, k) not in done
                    done[row, k] = (cta, where)
            x += max(end - start, 1)
    return first, per, done


@pytest.mark.parametrize("ctas", [1, 3, 8, 40, 152])
@pytest.mark.parametrize("heads", [1, 2, 4])
def test_every_tile_is_worked_and_joined_once(lib, heads, ctas):
    rng = random.Random(heads * 1000 + ctas)
    for _ in range(60):
        groups, seqs = draw_entries(rng)
        first, per, done = pieces(lib, groups, seqs, heads, ctas)
        n = 0
        for e in range(len(groups) + len(seqs)):
            rows = [groups[e][1:]] * groups[e][0] if e < len(groups) else seqs[e - len(groups)]
            for head in range(heads):
                for chunk, (tiles, kind) in enumerate(rows):
                    if tiles == 0:
                        continue
                    n += tiles
                    wrote = {("row" if w == "row" else (c, w)) for c, w in
                             (done[(e, head, chunk), k] for k in range(tiles))}
                    at = first[e] + (first[e + 1] - first[e]) // heads * head
                    found = set()

                    def add(place, more, begins):
                        r = lib.runs(place, more, per, ctas)
                        assert 1 <= r >> 16
                        for j in range(r >> 16):
                            found.add(((r & 0xffff) + j, 1) if j else begins(r & 0xffff))
                        return r >> 16

                    blocks = lib.count(tiles, len(rows), kind, per) if e < len(groups) else 1
                    if blocks == 1:
                        at += sum(lib.places(t, p) for t, p in rows[:chunk])
                        add(at + lib.row_cost_(kind), (tiles - 1) * lib.tile_cost_(kind), lambda c: "row")
                    else:
                        assert 2 * blocks <= ctas + 1
                        for i in range(blocks):
                            t0, t1 = (lib.first(tiles, len(rows), kind, per, i + z) for z in (0, 1))
                            p0 = lib.place(t0, kind)
                            span = lib.places(t1, kind) - p0
                            runs = add(at + len(rows) * p0 + chunk * span + (0 if i else lib.row_cost_(kind)),
                                       (t1 - t0 - 1) * lib.tile_cost_(kind), lambda c: (c, 2) if i else "row")
                            assert runs <= lib.block_runs()
                    assert found == wrote
        assert n == len(done)
