"""Attention of sequences that share prefixes, on the GPU, against the plain
64-bit form of every sequence by itself with the bounds derived in
tests/_kv16_ref.py (a part's factor 2^(m - M) is one more base-2 exponential of
a difference of scores: within the factor 2 of those bounds).  Every place of a
cache that holds no token, and every copy of a shared page that the calls have
no business with, is NaN or unmapped."""
import math

import pytest
import torch

from tests import _kv16_ref as R
from tests._shared_ref import SharedCase, bits, i32

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def L():
    from int2_kv_cache_02_gb300 import _build
    _build.build()
    from int2_kv_cache_02_gb300 import oscar
    oscar.device_status()
    return oscar


def strided(q):
    """The same queries as a slice of a wider projection."""
    wide = torch.full((q.shape[0], q.shape[1] + 3, 128), math.nan, dtype=q.dtype, device="cuda")
    wide[:, 1:1 + q.shape[1]] = q.cuda()
    return wide[:, 1:1 + q.shape[1]]


def decode(L, case, cache, Hq, window=0, sink=0, scale=R.SCALE, q=None, check=True):
    """By both ways, which the bound on the lengths chooses between."""
    q = case.normal(case.B, Hq) if q is None else q
    group, prefix = case.groups()
    want = [R.attend(case, b, q[b:b + 1], window, sink, scale) if check and case.lens[b] else None for b in range(case.B)]
    for max_tok in (cache.capacity, 1 << 20):
        out = torch.full((case.B, Hq, 128), 7.0, dtype=case.dtype, device="cuda")
        n = L.kv16_shared_decode_workspace_bytes(cache, Hq, len(case.prefix), max_tok, window, sink)
        ws = L.alloc_workspace(n)
        ws.fill_(math.nan)
        L.kv16_shared_decode_attention(cache, strided(q), group, prefix, scale, max_tok, out, ws,
                                       window=window, n_sink=sink)
        if not check:
            if max_tok == cache.capacity:
                first = out
            continue
        assert L.device_status() == 0
        for b in range(case.B):
            if case.lens[b] == 0:
                assert (out[b] == 0).all()
                continue
            R.assert_within(out[b:b + 1], want[b][0], want[b][3], f"out of sequence {b}, bound {max_tok}")
    return out if check else (first, out)


def attend(L, case, cache, news, Hq, window=0, sink=0, scale=R.SCALE, extra=2, check=True, lse=True, q=None):
    start = R.start_of(news)
    total = start[-1] + extra
    q = case.normal(total, Hq) if q is None else q
    group, prefix = case.groups()
    out = torch.full((total, Hq, 128), 7.0, dtype=case.dtype, device="cuda")
    z = torch.full((total, Hq), 7.0, device="cuda") if lse else None
    max_tok = cache.capacity
    n = L.kv16_shared_attention_workspace_bytes(cache, Hq, len(case.prefix), total, max_tok, window, sink)
    ws = L.alloc_workspace(n)
    ws.fill_(math.nan)
    L.kv16_shared_attention(cache, strided(q), i32(start), group, prefix, scale, max_tok, out, ws,
                            window=window, n_sink=sink, lse=z)
    if not check:
        return out, z
    assert L.device_status() == 0
    for b in range(case.B):
        rows = slice(start[b], start[b + 1])
        o, ref, _, tol, ztol, _ = R.attend(case, b, q[rows], window, sink, scale)
        R.assert_within(out[rows], o, tol, f"out of sequence {b}")
        if lse:
            R.assert_within(z[rows], ref, ztol, f"lse of sequence {b}")
    assert (out[start[-1]:] == 7).all() and (z is None or (z[start[-1]:] == 7).all())
    return out, z


HEADS = [(1, 1), (2, 1), (6, 2), (8, 2), (5, 1), (16, 2), (9, 1), (12, 1), (16, 1)]


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_decode_groups_of_heads(L, Hq, Hkv, dtype):
    case = SharedCase([3, 2], [300, 70], [310, 333, 301, 70, 200], Hkv, dtype=dtype, seed=Hq)
    decode(L, case, case.cache(L), Hq)


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("prefix", [0, 1, 31, 32, 33, 63, 64, 96, 127, 128, 129, 160, 255, 256, 257, 640, 1000])
@pytest.mark.parametrize("mine", [0, 1, 32, 33])
def test_decode_lengths(L, prefix, mine, paged):
    """A prefix and a sequence's own tokens at the sizes of pages and tiles; the
    first sequence has nothing behind its last shared page."""
    if prefix + mine == 0:
        return
    lens = [max(1, prefix // 32 * 32), prefix + mine, prefix + mine + 45, prefix + 1]
    case = SharedCase([4], [prefix if prefix // 32 * 32 <= lens[0] else 0], lens, 2, seed=prefix + mine, paged=paged)
    decode(L, case, case.cache(L), 8)


@pytest.mark.parametrize("members,Hq,Hkv", [(1, 8, 2), (17, 8, 2), (32, 8, 2), (33, 8, 2), (64, 4, 1), (65, 4, 1),
                                            (130, 4, 1), (25, 5, 1), (26, 5, 1), (51, 10, 2), (17, 16, 1), (300, 2, 2)])
def test_decode_members(L, members, Hq, Hkv):
    """Rows that fill one query tile, two, and more, whole and in part."""
    lens = [230 + (7 * b) % 61 for b in range(members)]
    lens[0] = 300
    case = SharedCase([members], [224], lens, Hkv, seed=members)
    decode(L, case, case.cache(L), Hq)


@pytest.mark.parametrize("window,sink", [(1, 0), (2, 1), (32, 4), (33, 33), (100, 1), (100, 64), (128, 200),
                                         (129, 5), (400, 4), (400, 300), (5000, 4), (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("Hq,Hkv,dtype,paged", [(8, 2, BF, True), (3, 1, FP, True), (16, 1, BF, False)])
def test_decode_windows(L, window, sink, Hq, Hkv, dtype, paged):
    case = SharedCase([3, 4], [290, 500], [290, 600, 431, 500, 505, 900, 501], Hkv, dtype=dtype, paged=paged,
                      seed=window % 1000 + sink % 1000)
    decode(L, case, case.cache(L), Hq, window, sink)


def test_decode_short_empty_and_ungrouped(L):
    """Sequences shorter than their group's prefix, without tokens, before and
    behind the groups; groups of one, of none, and with an empty prefix."""
    lens = [40, 300, 0, 100, 33, 1, 0, 70, 70, 65, 0]
    case = SharedCase([4, 0, 2, 2], [256, 90, 0, 64], lens[:1] + lens[1:], 2, first=1)
    decode(L, case, case.cache(L), 8)
    case = SharedCase([1, 1], [64, 0], [64, 0], 1)
    decode(L, case, case.cache(L), 4)


def test_decode_scales(L):
    for scale in (0.0, -0.3, 3.0):
        case = SharedCase([3], [200], [210, 300, 233], 1, dtype=FP)
        decode(L, case, case.cache(L), 4, scale=scale)


def test_decode_long_prefix(L):
    """Many tiles for every block of the grid; lengths and groups of unequal size."""
    members, prefix = [20, 3, 40], [9000, 20000, 4100]
    lens = []
    for m, p in zip(members, prefix):
        lens += [p + 1 + (37 * i) % 300 for i in range(m)]
    case = SharedCase(members, prefix, lens, 4, seed=3)
    decode(L, case, case.cache(L), 16)


@pytest.mark.parametrize("members,prefix,Hq,Hkv,dtype", [
    (130, 5000, 4, 1, BF), (200, 2100, 8, 2, FP), (37, 3333, 16, 1, BF), (90, 7000, 5, 1, FP)])
def test_decode_blocks(L, members, prefix, Hq, Hkv, dtype):
    """More queries than two tiles hold, over a prefix that is worked in blocks."""
    lens = [prefix + 1 + (11 * b) % 70 for b in range(members)]
    case = SharedCase([members, 3], [prefix, 600], lens + [640, 601, 700], Hkv, dtype=dtype, seed=members)
    decode(L, case, case.cache(L), Hq)


@pytest.mark.parametrize("window,sink", [(2600, 4), (700, 130), (4999, 0), (40, 1)])
@pytest.mark.parametrize("members,Hq,Hkv,dtype", [(130, 4, 1, BF), (20, 4, 2, FP), (90, 12, 2, FP)])
def test_decode_windows_in_blocks(L, members, Hq, Hkv, dtype, window, sink):
    """A prefix in blocks (or one row) under windows that begin in it, at unequal
    places, and behind it."""
    prefix = 5000
    lens = [prefix + 1 + (613 * b) % 3000 for b in range(members)]
    case = SharedCase([members, 3], [prefix, 600], lens + [640, 601, 2900], Hkv, dtype=dtype, seed=members + sink)
    decode(L, case, case.cache(L), Hq, window, sink)


def test_decode_many_sequences_and_groups(L):
    """The most sequences, each a group of its own, and all in pairs."""
    lens = [33 + b % 40 for b in range(4096)]
    case = SharedCase([1] * 4096, [32] * 4096, lens, 1)
    cache = case.cache(L)
    q = case.normal(4096, 1)
    out = decode(L, case, cache, 1, q=q, check=False)[1]
    assert L.device_status() == 0
    for b in range(0, 4096, 97):
        o, _, _, tol, _, _ = R.attend(case, b, q[b:b + 1])
        R.assert_within(out[b:b + 1], o, tol, f"out of sequence {b}")


def test_decode_agrees_with_the_plain_decode(L):
    """The same cache through kv16_decode_attention, whose table names the shared pages."""
    case = SharedCase([16], [700], [705 + 9 * b for b in range(16)], 2, dtype=FP)
    cache = case.cache(L)
    q = case.normal(16, 8)
    out = decode(L, case, cache, 8, q=q)
    cache.block_table[1:, :700 // 32] = cache.block_table[:1, :700 // 32]
    ref = torch.empty_like(out)
    ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 8, cache.capacity))
    L.kv16_decode_attention(cache, q.cuda(), R.SCALE, cache.capacity, ref, ws)
    assert L.device_status() == 0
    for b in range(16):
        _, _, _, tol, _, _ = R.attend(case, b, q[b:b + 1])
        R.assert_within(out[b:b + 1], ref[b:b + 1].double().cpu(), 2 * tol, f"sequence {b}")


def test_hidden_values_do_not_leak(L):
    """NaN and infinity that a query does not see: behind its length in a shared
    page (a member shorter than the prefix), before its window."""
    for dtype in (BF, FP):
        case = SharedCase([3], [256], [300, 100, 280], 1, dtype=dtype)
        for x in (case.k, case.v):
            x[0][:, 100:180] = math.nan
            x[2][:, 100:180] = math.nan
        cache = case.cache(L)
        q = case.normal(3, 4)
        outs = decode(L, case, cache, 4, window=90, sink=7, q=q, check=False)
        assert L.device_status() == 0
        o, _, _, tol, _, _ = R.attend(case, 1, q[1:2], 90, 7)
        for out in outs:
            R.assert_within(out[1:2], o, tol, "sequence 1")
        # the 90 tokens before position 299 and 279 start behind 180
        clean = SharedCase([3], [256], [300, 100, 280], 1, dtype=dtype)
        for b in (0, 2):
            clean.k[b], clean.v[b] = case.k[b].nan_to_num(0.0), case.v[b].nan_to_num(0.0)
            o, _, _, tol, _, _ = R.attend(clean, b, q[b:b + 1], 90, 7)
            for out in outs:
                R.assert_within(out[b:b + 1], o, tol, f"sequence {b}")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("where", [5, 130, 255, 270])
def test_what_a_query_sees_reaches_it(L, where, dtype):
    """A visible infinity in a value gives that infinity in its channel, both give
    NaN, a NaN its channel, a NaN key the whole row: in the prefix and behind it."""
    case = SharedCase([2], [256], [290, 280], 1, dtype=dtype, seed=where)
    for b in range(2):
        case.v[b][:, where, 3] = math.inf
        case.v[b][:, where, 9] = -math.inf
        case.v[b][:, where, 40] = math.nan
        case.v[b][:, where, 77] = math.inf
        case.v[b][:, 11, 77] = -math.inf
    cache = case.cache(L)
    q = case.normal(2, 4)
    for out in (*decode(L, case, cache, 4, q=q, check=False),
                attend(L, case, cache, [1, 1], 4, q=q, extra=0, check=False)[0]):
        assert L.device_status() == 0
        assert (out[:, :, 3] == math.inf).all() and (out[:, :, 9] == -math.inf).all()
        assert out[:, :, 40].isnan().all() and out[:, :, 77].isnan().all()
        keep = [c for c in range(128) if c not in (3, 9, 40, 77)]
        assert out[:, :, keep].isfinite().all()
    for b in range(2):
        case.k[b][:, where] = math.nan
    cache = case.cache(L)
    assert all(out.isnan().all() for out in decode(L, case, cache, 4, q=q, check=False))
    assert attend(L, case, cache, [1, 1], 4, q=q, extra=0, check=False)[0].isnan().all()
    assert L.device_status() == 0


@pytest.mark.parametrize("members,new,prefix", [(40, 1, 600), (3, 40, 600), (3, 9, 130), (9, 230, 4000)])
def test_infinities_in_every_kind_of_row(L, members, new, prefix):
    """The same for rows that fill both query tiles, for several queries, for many
    rows: an infinity and a NaN in the prefix's values, others in one sequence's own."""
    lens = [prefix + new + 3 * b for b in range(members)]
    case = SharedCase([members], [prefix], lens, 1, seed=members)
    for b in range(members):
        case.v[b][:, 77, 3] = math.inf
        case.v[b][:, 78, 40] = math.nan
    case.v[1][:, prefix, 9] = -math.inf          # every new query of the sequence sees it
    cache = case.cache(L)
    start = R.start_of([new] * members)
    q = case.normal(start[-1], 4)
    outs = [attend(L, case, cache, [new] * members, 4, q=q, extra=0, check=False)[0]]
    if new == 1:
        outs += decode(L, case, cache, 4, q=q, check=False)
    assert L.device_status() == 0
    for out in outs:
        assert (out[:, :, 3] == math.inf).all() and out[:, :, 40].isnan().all()
        rows = slice(start[1], start[2])
        assert (out[rows, :, 9] == -math.inf).all()
        keep = [c for c in range(128) if c not in (3, 9, 40)]
        assert out[:, :, keep].isfinite().all()
    for b in (0, 1, members - 1):
        for c in (3, 9, 40):
            case.v[b][:, :, c] = 0.0
        rows = slice(start[b], start[b + 1])
        o, _, _, tol, _, _ = R.attend(case, b, q[rows])
        for out in outs:
            R.assert_within(out[rows][:, :, keep], o[:, :, keep], tol[:, :, keep], f"sequence {b}")


def test_workspace_at_any_16_bytes(L):
    """A workspace that begins 16 bytes behind an allocation's start: the same bits."""
    case = SharedCase([5], [300], [330, 310, 420, 301, 390], 2)
    cache = case.cache(L)
    q = case.normal(5, 8).cuda()
    group, prefix = case.groups()
    n = L.kv16_shared_decode_workspace_bytes(cache, 8, 1, 1 << 20)
    big = torch.full((n + 32,), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    for at, out in zip((0, 16), outs):
        L.kv16_shared_decode_attention(cache, q, group, prefix, R.SCALE, 1 << 20, out, big[at:at + n])
    assert L.device_status() == 0
    assert torch.equal(bits(outs[0]), bits(outs[1]))
    assert (big[n + 16:] == 255).all()


def test_far_apart_scores(L):
    """One part of the keys outweighs the other by far: its output alone is left."""
    for lead in (True, False):
        case = SharedCase([2], [128], [200, 190], 1, dtype=BF)
        for b in range(2):
            part = slice(0, 128) if lead else slice(128, None)
            case.k[b][:, part] = (case.k[b][:, part].float().abs() * 40).to(BF)
        q = case.normal(2, 4).abs()
        decode(L, case, case.cache(L), 4, q=q)


def test_bad_groups_and_pages_are_recorded(L):
    """Groups out of range share nothing (the sequences' own pages are read); a bad
    page is skipped; neither stops the other sequences."""
    case = SharedCase([2, 2], [64, 64], [80, 81, 90, 91], 1)
    q = case.normal(4, 2)
    cache = case.cache(L)
    whole = R.Case.cache(case, L)
    for group, prefix in (([0, 2, 5], [64, 64]), ([0, 2, 4], [64, -1]), ([0, 2, 4], [64, 100000])):
        for most in (96, 1 << 20):
            out = torch.empty((4, 2, 128), dtype=BF, device="cuda")
            ws = L.alloc_workspace(L.kv16_shared_decode_workspace_bytes(whole, 2, 2, most))
            L.kv16_shared_decode_attention(whole, q.cuda(), i32(group), i32(prefix), R.SCALE, most, out, ws)
            assert L.device_status() != 0 and L.device_status() == 0
            for b in range(4):
                o, _, _, tol, _, _ = R.attend(case, b, q[b:b + 1])
                R.assert_within(out[b:b + 1], o, tol, f"sequence {b}")
    cache.block_table[0, 0] = 1 << 20
    outs = decode(L, case, cache, 2, q=q, check=False)
    assert L.device_status() != 0 and L.device_status() == 0
    for b in (2, 3):
        o, _, _, tol, _, _ = R.attend(case, b, q[b:b + 1])
        for out in outs:
            R.assert_within(out[b:b + 1], o, tol, f"sequence {b}")
    cache = case.cache(L)
    cache.n_tok[1] = 100000
    outs = decode(L, case, cache, 2, q=q, check=False)
    assert L.device_status() != 0 and L.device_status() == 0
    for b in (0, 2, 3):
        o, _, _, tol, _, _ = R.attend(case, b, q[b:b + 1])
        for out in outs:
            R.assert_within(out[b:b + 1], o, tol, f"sequence {b}")


# ------------------------------------------------------ several new tokens

@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_attention_groups_of_heads(L, Hq, Hkv, dtype):
    case = SharedCase([3, 2], [300, 70], [310, 433, 301, 90, 200], Hkv, dtype=dtype, seed=Hq)
    attend(L, case, case.cache(L), [10, 133, 1, 20, 40], Hq)


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("prefix", [0, 1, 31, 32, 33, 64, 127, 128, 129, 256, 257, 640])
def test_attention_lengths(L, prefix, paged):
    """New tokens that begin where the prefix ends, behind it, and inside it."""
    lens = [prefix + 1, prefix + 33, prefix + 100, prefix + 7]
    case = SharedCase([4], [prefix], lens, 2, seed=prefix, paged=paged)
    attend(L, case, case.cache(L), [1, 33, 50, min(prefix + 7, 40)], 8)


@pytest.mark.parametrize("window,sink", [(1, 0), (2, 1), (33, 33), (100, 64), (128, 200), (129, 5), (400, 4),
                                         (400, 300), (5000, 4), (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("Hq,Hkv,dtype,paged", [(8, 2, BF, True), (3, 1, FP, True), (16, 1, BF, False)])
def test_attention_windows(L, window, sink, Hq, Hkv, dtype, paged):
    case = SharedCase([3, 4], [290, 500], [300, 600, 431, 520, 505, 900, 501], Hkv, dtype=dtype, paged=paged,
                      seed=window % 1000 + sink % 1000)
    attend(L, case, case.cache(L), [10, 300, 3, 1, 5, 200, 1], Hq, window, sink)


def test_attention_short_empty_and_ungrouped(L):
    lens = [40, 300, 0, 100, 33, 1, 0, 70, 70, 65, 0]
    case = SharedCase([4, 0, 2, 2], [256, 90, 0, 64], lens, 2, first=1)
    attend(L, case, case.cache(L), [40, 12, 0, 100, 1, 1, 0, 0, 70, 3, 0], 8)


def test_attention_many_rows(L):
    """Many query tiles over one prefix, few over a long one."""
    case = SharedCase([6], [700], [1000, 900, 720, 800, 1100, 701], 2, seed=1)
    attend(L, case, case.cache(L), [300, 200, 20, 90, 400, 1], 8, extra=0)
    case = SharedCase([9], [9000], [9005 + b for b in range(9)], 2, seed=2)
    attend(L, case, case.cache(L), [5, 4, 3, 5, 1, 2, 5, 5, 3], 8, lse=False)


@pytest.mark.parametrize("window,sink", [(2600, 4), (300, 130)])
def test_attention_windows_in_blocks(L, window, sink):
    case = SharedCase([5, 2], [4500, 900], [4700, 5100, 4520, 6100, 4801, 1200, 901], 2, dtype=FP, seed=sink)
    attend(L, case, case.cache(L), [150, 90, 20, 70, 301, 40, 1], 8, window, sink)


# ------------------------------------------- graphs, streams, workspaces

def test_graphs_share_a_workspace(L):
    """Three captured calls on one workspace, replayed in turn, with lengths, prefixes
    and groups that change between replays: the same bits as the calls themselves."""
    case = SharedCase([3, 3], [400, 320], [430, 420, 410, 330, 350, 390], 2)
    cache = case.cache(L)
    group, prefix = case.groups()
    q = case.normal(6, 8).cuda()
    start = i32([0, 1, 2, 3, 4, 5, 6])
    outs = [torch.empty_like(q) for _ in range(3)]
    ws = L.alloc_workspace(max(L.kv16_shared_decode_workspace_bytes(cache, 8, 2, 1 << 20),
                               L.kv16_shared_attention_workspace_bytes(cache, 8, 2, 6, cache.capacity)))
    calls = [lambda: L.kv16_shared_decode_attention(cache, q, group, prefix, R.SCALE, 1 << 20, outs[0], ws),
             lambda: L.kv16_shared_decode_attention(cache, q, group, prefix, R.SCALE, cache.capacity, outs[2], ws),
             lambda: L.kv16_shared_attention(cache, q, start, group, prefix, R.SCALE, cache.capacity, outs[1], ws)]
    graphs = []
    for call in calls:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    whole = R.Case.cache(case, L)      # every sequence's own pages are there
    cache.block_table.copy_(whole.block_table)
    cache.k.copy_(whole.k)
    cache.v.copy_(whole.v)
    for p, n in (([400, 320], case.lens), ([64, 0], [420, 1, 410, 329, 350, 33]), ([0, 320], [0, 420, 64, 320, 321, 322])):
        prefix.copy_(i32(p))
        cache.n_tok.copy_(i32(n))
        got = []
        for call, out in zip(calls, (outs[0], outs[2], outs[1])):
            out.fill_(7)
            call()
            torch.cuda.synchronize()
            got.append(out.clone())
            out.fill_(7)
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for out, want in zip((outs[0], outs[2], outs[1]), got):
            assert torch.equal(bits(out), bits(want))
    L.device_status()


def test_streams(L):
    """Calls on two streams at once, each with its own workspace, give the bits of the calls alone."""
    cases = [SharedCase([8], [2000], [2040 + b for b in range(8)], 2, seed=s) for s in range(2)]
    caches = [c.cache(L) for c in cases]
    qs = [c.normal(8, 8).cuda() for c in cases]
    wss = [L.alloc_workspace(L.kv16_shared_decode_workspace_bytes(c, 8, 1, c.capacity)) for c in caches]
    group, prefix = cases[0].groups()

    def go(i, out, stream=None):
        L.kv16_shared_decode_attention(caches[i], qs[i], group, prefix, R.SCALE, caches[i].capacity, out, wss[i], stream=stream)

    want = [torch.empty_like(q) for q in qs]
    for i in range(2):
        go(i, want[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(20)] for q in qs]
    for n in range(20):
        for i in range(2):
            go(i, outs[i][n], streams[i])
    torch.cuda.synchronize()
    assert L.device_status() == 0
    for i in range(2):
        for out in outs[i]:
            assert torch.equal(bits(out), bits(want[i]))
