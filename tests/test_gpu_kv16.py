"""The 16-bit cache on the GPU: write, attention of a ragged batch, decode
attention, accumulated weight, eviction, and a run of them together, against
plain 64-bit forms with derived bounds (tests/_kv16_ref.py).  Every place of a
cache that holds no token is NaN."""
import math

import pytest
import torch

from tests import _kv16_ref as R

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def L():
    from int2_kv_cache_02_gb300 import _build
    _build.build()
    from int2_kv_cache_02_gb300 import oscar
    oscar.device_status()
    return oscar


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------- write

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("Hkv,news,pos", [
    (1, [1], [0]), (8, [1, 1, 1], [5, 31, 32]), (3, [0, 7, 0, 70], [4, 0, 9, 33]),
    (5, [200, 1, 33], [0, 64, 31]), (2, [0, 0], [3, 0])])
def test_write(L, dtype, paged, Hkv, news, pos):
    """Tokens land at their places, weights become 0, lengths follow, and
    everything else, rows behind the last sequence too, stays as it was."""
    case = R.Case([p + n + 40 for p, n in zip(pos, news)], Hkv, dtype, paged, weights=True)
    cache = case.cache(L)
    before = [(x.clone() if x is not None else None) for x in (cache.k, cache.v, cache.weight)]
    start = R.start_of(news)
    total = start[-1] + 3
    # rows of a fused projection: queries, keys and values of a token side by side
    fused = case.normal(total, 2 + 2 * Hkv).cuda()
    k_new, v_new = fused[:, 2:2 + Hkv], fused[:, 2 + Hkv:]
    L.kv16_write(cache, k_new, v_new, i32(start), i32(pos))
    assert L.device_status() == 0
    assert cache.n_tok.tolist() == [p + n for p, n in zip(pos, news)]
    for x, y, new in zip((cache.k, cache.v, cache.weight), before, (k_new, v_new, None)):
        want = y.clone()
        for b in range(case.B):
            for i in range(news[b]):
                t = pos[b] + i
                at = (int(cache.block_table[b, t // 32]), slice(None), t % 32) if paged else (b, slice(None), t)
                want[at] = new[start[b] + i] if new is not None else 0.0
        as_int = lambda z: z.view(torch.int16 if z.element_size() == 2 else torch.int32)
        assert torch.equal(as_int(x), as_int(want))


def test_write_over_capacity_and_bad_pages(L):
    """A sequence that would pass its capacity keeps its length and tokens; an
    unmapped page is skipped; both are recorded, the other sequences written."""
    case = R.Case([40, 40, 40], 2, slack=0)           # 2 blocks: 64 tokens
    cache = case.cache(L)
    old = [R.tokens(cache, b, 40).clone() for b in range(3)]
    new = case.normal(3, 2).cuda()
    L.kv16_write(cache, new, new, i32([0, 1, 2, 3]), i32([64, 40, 40]))
    assert L.device_status() != 0 and L.device_status() == 0
    assert cache.n_tok.tolist() == [40, 41, 41]
    assert torch.equal(R.tokens(cache, 0, 40), old[0])
    assert torch.equal(R.tokens(cache, 1, 41)[:, 40], new[1].cpu())
    cache.block_table[2, 1] = 99999
    L.kv16_write(cache, new, new, i32([0, 1, 2, 3]), i32([1, 1, 40]))
    assert L.device_status() != 0
    assert torch.equal(R.tokens(cache, 0, 2)[:, 1], new[0].cpu())


# --------------------------------------------------------------- attention

def run_attention(L, case, cache, news, Hq, window=0, sink=0, extra=0, lse=True, strided=False,
                  scale=R.SCALE, max_tok=None, check=True):
    start = R.start_of(news)
    total = start[-1] + extra
    q = case.normal(total, Hq)
    qd = q.cuda()
    if strided:
        wide = torch.full((total, Hq + 3, 128), math.nan, dtype=case.dtype, device="cuda")
        wide[:, 1:1 + Hq] = qd
        qd = wide[:, 1:1 + Hq]
    out = torch.full((total, Hq, 128), 7.0, dtype=case.dtype, device="cuda")
    ls = torch.full((total, Hq), 7.0, device="cuda") if lse else None
    max_tok = cache.capacity if max_tok is None else max_tok
    ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, Hq, total, max_tok, window, sink))
    ws.fill_(math.nan)
    L.kv16_attention(cache, qd, i32(start), scale, max_tok, out, ws, window=window, n_sink=sink, lse=ls)
    if not check:
        return out, ls
    assert L.device_status() == 0
    for b in range(case.B):
        rows = slice(start[b], start[b + 1])
        o, z, _, tol, ztol, _ = R.attend(case, b, q[rows], window, sink, scale)
        R.assert_within(out[rows], o, tol, f"out of sequence {b}")
        if lse:
            R.assert_within(ls[rows], z, ztol, f"lse of sequence {b}")
    assert (out[start[-1]:] == 7).all() and (ls is None or (ls[start[-1]:] == 7).all())
    return out, ls


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (6, 2), (8, 2), (5, 1), (7, 1), (16, 2), (9, 1), (12, 1), (15, 1), (16, 1)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_attention_groups(L, Hq, Hkv, dtype):
    case = R.Case([70, 129, 300], Hkv, dtype, paged=True, seed=Hq)
    run_attention(L, case, case.cache(L), [70, 30, 150], Hq, extra=2)


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500])
def test_attention_lengths(L, paged, n):
    """Whole prompts and their last tokens alone, at the sizes of pages and tiles."""
    case = R.Case([n, max(1, n - 3), n], 2, BF, paged, seed=n)
    run_attention(L, case, case.cache(L), [n, 1, min(n, 40)], 8)


@pytest.mark.parametrize("window,sink", [(1, 0), (2, 1), (31, 0), (32, 4), (33, 33), (100, 1), (100, 64),
                                         (128, 200), (129, 5), (400, 4), (5000, 4), (5000, 0), (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("Hq,Hkv,dtype,paged", [(8, 2, BF, True), (3, 1, FP, True), (16, 1, BF, False)])
def test_attention_windows(L, window, sink, Hq, Hkv, dtype, paged):
    case = R.Case([600, 333, 40], Hkv, dtype, paged, seed=window % 1000 + sink % 1000)
    run_attention(L, case, case.cache(L), [300, 333, 3], Hq, window, sink)


def test_attention_ragged_empty_sequences(L):
    """Sequences without new tokens, without any tokens, first, last and in a row."""
    case = R.Case([0, 50, 0, 33, 200, 64, 0], 2, BF)
    run_attention(L, case, case.cache(L), [0, 50, 0, 0, 7, 64, 0], 8, extra=5, strided=True)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_attention_scales(L, scale):
    """A uniform softmax, a negative scale, and one that makes it nearly one-hot."""
    case = R.Case([200, 300], 1, FP)
    run_attention(L, case, case.cache(L), [200, 100], 4, scale=scale)


def test_attention_growing_maxima(L):
    """Keys that grow along the sequence: the running maximum moves in every tile."""
    case = R.Case([900], 1, BF)
    f = torch.linspace(0.01, 6.0, 900)[None, :, None]
    case.k[0] = (case.k[0].float().abs() * f).to(BF)
    q_pos = case.normal
    case.normal = lambda *s: q_pos(*s).abs()
    run_attention(L, case, case.cache(L), [300], 8)


@pytest.mark.parametrize("hq", [1, 12])
def test_attention_hidden_values_do_not_leak(L, hq):
    """NaN and infinity in keys and values that a query does not see: later
    tokens, tokens before the window."""
    case = R.Case([300], 1, BF)
    cache = case.cache(L)
    bad = [20, 150, 299]
    for t, (kx, vx) in zip(bad, [(math.nan, math.nan), (math.inf, -math.inf), (math.nan, math.inf)]):
        page, slot = int(cache.block_table[0, t // 32]), t % 32
        cache.k[page, :, slot] = kx
        cache.v[page, :, slot] = vx
    out, lse = run_attention(L, case, cache, [300], hq, window=30, sink=2, check=False)
    assert L.device_status() == 0
    at = torch.arange(300)
    see = R.visible(at, 300, 30, 2)[:, bad].any(1)
    assert torch.isfinite(out[~see.cuda()].float()).all() and torch.isfinite(lse[~see.cuda()]).all()
    # what a query sees reaches it
    assert not torch.isfinite(out[see.cuda()].float()).all(-1).any()


@pytest.mark.parametrize("window,sink", [(0, 0), (30, 2)])
def test_attention_beside_hidden_values(L, window, sink):
    """The queries that see no NaN give what they give without it, next to ones
    that do, in the same tiles, split or not."""
    for n, new in ((300, 300), (7000, 5)):
        case = R.Case([n], 1, BF, seed=n)
        cache, gen = case.cache(L), case.gen.get_state()
        clean, clean_lse = run_attention(L, case, cache, [new], 6, window, sink)
        t = n - 3
        cache.v[int(cache.block_table[0, t // 32]), :, t % 32] = math.nan
        case.gen.set_state(gen)
        out, lse = run_attention(L, case, cache, [new], 6, window, sink, check=False)
        assert L.device_status() == 0
        assert torch.isnan(out[-3:]).all()
        off = (out[:-3].double() - clean[:-3].double()).abs()
        # both within their bounds of the same number: twice two roundings
        assert (off <= 4 * R.U[BF] * clean[:-3].double().abs() + 4 * R.U[BF]).all()
        assert torch.equal(lse[-3:], clean_lse[-3:]) or torch.isfinite(lse[-3:]).all()


def test_attention_long_cache_few_queries(L):
    """Few queries over long caches: the cache's length is split and joined."""
    case = R.Case([9000, 4001, 100], 2, BF, seed=5)
    for news, window, sink in (([3, 1, 2], 0, 0), ([40, 33, 2], 0, 0), ([3, 1, 2], 6000, 70)):
        run_attention(L, case, case.cache(L), news, 8, window, sink)
    case = R.Case([5000], 1, FP, paged=False, seed=6)
    run_attention(L, case, case.cache(L), [17], 7, extra=1)


def test_attention_bad_lengths_and_pages(L):
    """Lengths outside the cache, more queries than tokens, page ids outside the
    pool: recorded, no fault, and the other sequences are right."""
    case = R.Case([100, 100, 100, 100], 2, BF)
    for n_tok, spoil in (([100, 10**6, 100, 100], None), ([100, -5, 100, 100], None),
                         ([100, 3, 100, 100], None), ([100, 100, 100, 100], 123456)):
        cache = case.cache(L, n_tok)
        if spoil:
            cache.block_table[1, 2] = spoil
        q = case.normal(40, 8)
        out = torch.zeros((40, 8, 128), dtype=BF, device="cuda")
        ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, 8, 40, 128))
        L.kv16_attention(cache, q.cuda(), i32([0, 10, 20, 30, 40]), R.SCALE, 128, out, ws)
        assert L.device_status() != 0
        for b in (0, 2, 3):
            o, _, _, tol, _, _ = R.attend(case, b, q[10 * b:10 * b + 10])
            R.assert_within(out[10 * b:10 * b + 10], o, tol, str(b))


# ------------------------------------------------------------------ decode

def run_decode(L, case, cache, Hq, window=0, sink=0, accumulate=False, ws=None, max_tok=None):
    q = case.normal(case.B, Hq)
    out = torch.full((case.B, Hq, 128), 7.0, dtype=case.dtype, device="cuda")
    max_tok = cache.capacity if max_tok is None else max_tok
    n = L.kv16_decode_workspace_bytes(cache, Hq, max_tok, window, sink, accumulate)
    if ws is None:
        ws = L.alloc_workspace(n)
        ws[65536:] = math.nan
    assert ws.numel() * 4 >= n
    L.kv16_decode_attention(cache, q.cuda(), R.SCALE, max_tok, out, ws, window, sink, accumulate)
    assert L.device_status() == 0
    assert (ws[:65536].view(torch.int32) == 0).all()
    for b, n in enumerate(case.lens):
        if n == 0:
            assert (out[b] == 0).all()
            continue
        o, _, p, tol, _, dmax = R.attend(case, b, q[b:b + 1], window, sink)
        R.assert_within(out[b:b + 1], o, tol, f"out of sequence {b}")
        if accumulate:
            w, wtol = R.weight_of(p, dmax, Hq // case.Hkv)
            R.assert_within(R.tokens(cache, b, n, "weight"), w + case.w[b].double(),
                            wtol + 2 * R.U32 * case.w[b].double(), f"weight of sequence {b}")
    return q, out


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("Hq,Hkv,dtype,paged", [
    (1, 1, BF, True), (2, 1, FP, True), (6, 2, BF, True), (8, 2, BF, False), (5, 1, FP, False),
    (14, 2, BF, True), (16, 2, FP, True), (9, 1, BF, True), (16, 1, BF, True), (32, 8, BF, True)])
def test_decode_groups(L, Hq, Hkv, dtype, paged, accumulate):
    case = R.Case([1, 31, 32, 33, 700, 0, 250], Hkv, dtype, paged, seed=Hq, weights=True)
    run_decode(L, case, case.cache(L), Hq, accumulate=accumulate)


@pytest.mark.parametrize("window,sink", [(1, 0), (1, 1), (31, 0), (32, 4), (33, 33), (100, 64), (300, 4), (5000, 4), (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("paged", [True, False])
def test_decode_windows(L, window, sink, paged):
    case = R.Case([600, 333, 40, 1, 0, 128], 2, BF, paged, seed=window % 1000, weights=True)
    run_decode(L, case, case.cache(L), 8, window, sink, accumulate=True)


@pytest.mark.parametrize("lens", [[20000], [5000, 1, 9000, 64, 0, 3000]])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (16, 2)])
def test_decode_long(L, lens, Hq, Hkv):
    """Long caches cut into many pieces, and joined."""
    case = R.Case(lens, Hkv, BF, seed=3, weights=True)
    run_decode(L, case, case.cache(L), Hq, accumulate=True)


def test_decode_many_sequences(L):
    """More rows than blocks of the launch: pieces that span sequences."""
    g = torch.Generator().manual_seed(3)
    case = R.Case(torch.randint(0, 90, (700,), generator=g).tolist(), 1, BF, weights=True)
    run_decode(L, case, case.cache(L), 4, accumulate=True)
    case = R.Case(torch.randint(1, 9, (300,), generator=g).tolist(), 4, FP, paged=False)
    run_decode(L, case, case.cache(L), 4)


def test_decode_at_the_batch_limit(L):
    """4096 sequences with groups of 1 and 16 heads, sampled."""
    g = torch.Generator().manual_seed(4)
    for Hq in (1, 16):
        case = R.Case(torch.randint(0, 60, (4096,), generator=g).tolist(), 1, BF, weights=True)
        cache = case.cache(L)
        q = case.normal(4096, Hq)
        out = torch.empty((4096, Hq, 128), dtype=BF, device="cuda")
        ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, Hq, 96, 0, 0, True))
        L.kv16_decode_attention(cache, q.cuda(), R.SCALE, 96, out, ws, accumulate=True)
        assert L.device_status() == 0 and (ws[:65536].view(torch.int32) == 0).all()
        w_all, out = cache.weight.cpu(), out.cpu()
        for b in list(range(0, 4096, 311)) + [4095]:
            n = case.lens[b]
            o, _, p, tol, _, dmax = R.attend(case, b, q[b:b + 1])
            R.assert_within(out[b:b + 1], o, tol, str(b))
            w, t = R.weight_of(p, dmax, Hq)
            j = torch.arange(n)
            got = w_all[cache.block_table[b].cpu().long()[j // 32], :, j % 32].transpose(0, 1)
            R.assert_within(got, w + case.w[b].double(), t + 2 * R.U32, str(b))


def test_decode_hidden_values_do_not_leak(L):
    case = R.Case([300, 200], 2, BF, weights=True)
    cache = case.cache(L)
    for t in (5, 150, 267):
        cache.k[int(cache.block_table[0, t // 32]), :, t % 32] = math.nan
        cache.v[int(cache.block_table[0, t // 32]), :, t % 32] = math.inf
    run_decode(L, case, cache, 8, window=32, sink=5, accumulate=True)


def test_decode_visible_nan_stays_in_its_row(L):
    """A NaN that a sequence sees makes its own row NaN (that KV head's alone) and
    no other, though one block works on both rows."""
    case = R.Case([90, 80, 33], 2, BF, weights=True)
    cache = case.cache(L)
    cache.k[int(cache.block_table[1, 1]), 0, 3] = math.nan
    q = case.normal(3, 8)
    out = torch.empty((3, 8, 128), dtype=BF, device="cuda")
    ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 8, 96, 0, 0, True))
    L.kv16_decode_attention(cache, q.cuda(), R.SCALE, 96, out, ws, accumulate=True)
    assert torch.isnan(out[1, :4]).all()
    for b in range(3):
        o, _, p, tol, _, dmax = R.attend(case, b, q[b:b + 1])
        h = slice(4, 8) if b == 1 else slice(0, 8)
        R.assert_within(out[b:b + 1, h], o[:, h], tol[:, h], str(b))
        w, t = R.weight_of(p, dmax, 4)
        kv = slice(1, 2) if b == 1 else slice(0, 2)
        R.assert_within(R.tokens(cache, b, case.lens[b], "weight")[kv], (w + case.w[b].double())[kv],
                        (t + 2 * R.U32)[kv], str(b))


def test_decode_is_repeatable_and_leaves_its_workspace(L):
    """One workspace over different shapes; the same call twice gives the same bits."""
    small = R.Case([50] * 9, 4, FP)
    big = R.Case([4000, 100, 900], 2, BF, weights=True).cache(L)
    cs = small.cache(L)
    ws = L.alloc_workspace(max(L.kv16_decode_workspace_bytes(big, 16, big.capacity, 0, 0, True),
                               L.kv16_decode_workspace_bytes(cs, 8, cs.capacity)))
    outs, weights = [], []
    for _ in range(2):
        c = R.Case([4000, 100, 900], 2, BF, weights=True)
        cache = c.cache(L)
        outs.append(run_decode(L, c, cache, 16, accumulate=True, ws=ws)[1])
        weights.append([R.tokens(cache, b, n, "weight") for b, n in enumerate(c.lens)])
        run_decode(L, small, cs, 8, ws=ws)
    assert torch.equal(outs[0], outs[1])
    assert all(torch.equal(a, b) for a, b in zip(*weights))


def test_decode_shares_its_workspace_with_the_packed_decode(L):
    """One decode workspace, used in turn by the packed and the 16-bit decode."""
    case = R.Case([3000, 700], 2, BF)
    cache = case.cache(L)
    packed = L.KVCache(2, 2, 1024)
    kv = [torch.randn((2, 2, 1024, 128), device="cuda").bfloat16() for _ in range(2)]
    L.prefill_kv(packed, *kv, 1024)
    ws = L.alloc_workspace(max(L.kv16_decode_workspace_bytes(cache, 8, cache.capacity),
                               L.decode_workspace_bytes(2, 2, 8, 1024, 3)))
    qr = torch.randn((2, 8, 128), device="cuda")
    outs = []
    for _ in range(2):
        o = torch.empty((2, 8, 128), device="cuda")
        L.decode_attention(packed, qr, 8, R.SCALE, o, ws, num_splits=3)
        outs.append(o)
        run_decode(L, case, cache, 8, ws=ws)
    assert torch.equal(*outs)


def test_decode_bad_lengths_and_pages(L):
    case = R.Case([100, 100, 100], 2, BF)
    for n_tok, spoil in (([100, 10**6, 100], None), ([100, -5, 100], None), ([100, 100, 100], 123456), ([100, 100, 100], -1)):
        cache = case.cache(L, n_tok)
        if spoil:
            cache.block_table[1, 2] = spoil
        q = case.normal(3, 8)
        out = torch.zeros((3, 8, 128), dtype=BF, device="cuda")
        ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 8, 128))
        L.kv16_decode_attention(cache, q.cuda(), R.SCALE, 128, out, ws)
        assert L.device_status() != 0
        assert (ws[:65536].view(torch.int32) == 0).all()
        for b in (0, 2):
            o, _, _, tol, _, _ = R.attend(case, b, q[b:b + 1])
            R.assert_within(out[b:b + 1], o, tol, str(b))


# -------------------------------------------------------------- accumulate

@pytest.mark.parametrize("Hq,Hkv,dtype,paged", [(4, 1, BF, True), (16, 1, FP, True), (6, 2, BF, False), (7, 1, BF, True)])
@pytest.mark.parametrize("n_obs,window,sink", [(0, 0, 0), (1, 0, 0), (16, 0, 0), (1000, 50, 4), (0, 200, 40), (0, 1, 0)])
def test_accumulate(L, Hq, Hkv, dtype, paged, n_obs, window, sink):
    case = R.Case([400, 129, 1, 0, 77], Hkv, dtype, paged, seed=n_obs, weights=True)
    news = [300, 129, 1, 0, 0]
    cache, start = case.cache(L), R.start_of(news)
    q = case.normal(start[-1] + 2, Hq)
    lse = torch.full((start[-1] + 2, Hq), math.nan)
    parts = []
    for b, nq in enumerate(news):
        rows = slice(start[b], start[b + 1])
        _, z, p, _, ztol, dmax = R.attend(case, b, q[rows], window, sink)
        lse[rows] = z.float()
        parts.append((p, dmax))
    L.kv16_accumulate(cache, q.cuda(), lse.cuda(), i32(start), R.SCALE, cache.capacity, window, sink, n_obs)
    assert L.device_status() == 0
    for b, nq in enumerate(news):
        p, dmax = parts[b]
        skip = max(0, nq - n_obs) if n_obs else 0
        w, tol = R.weight_of(p[skip:], dmax[skip:], Hq // Hkv)
        # the lse as given is rounded to fp32
        tol = tol + 16 * R.U32 * w
        n = case.lens[b]
        R.assert_within(R.tokens(cache, b, n, "weight"), w + case.w[b].double(), tol, f"sequence {b}")
    # tokens that no sequence holds stay as they were
    held = sum(case.lens) * Hkv
    assert int(torch.isfinite(cache.weight).sum()) == held


def test_accumulate_is_repeatable_and_strided(L):
    """The same bits twice; queries that are a slice of a wider row."""
    case = R.Case([500, 300], 2, BF, weights=True)
    q = case.normal(350, 8)
    wide = torch.full((350, 11, 128), math.nan, dtype=BF, device="cuda")
    wide[:, 2:10] = q.cuda()
    got = []
    for qd in (q.cuda(), wide[:, 2:10]):
        case.gen.manual_seed(1)
        cache = case.cache(L)
        out, lse = torch.empty((350, 8, 128), dtype=BF, device="cuda"), torch.empty((350, 8), device="cuda")
        ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, 8, 350, 512))
        L.kv16_attention(cache, qd, i32([0, 200, 350]), R.SCALE, 512, out, ws, lse=lse)
        L.kv16_accumulate(cache, qd, lse, i32([0, 200, 350]), R.SCALE, 512)
        got.append((out, lse, torch.nan_to_num(cache.weight)))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert L.device_status() == 0


def test_accumulate_bad_lengths_and_pages(L):
    case = R.Case([100, 100, 100], 2, BF, weights=True)
    for n_tok, spoil in (([100, 10**6, 100], None), ([100, 3, 100], None), ([100, 100, 100], -1)):
        cache = case.cache(L, n_tok)
        if spoil:
            cache.block_table[1, 2] = spoil
        q, lse = case.normal(30, 8), torch.zeros((30, 8))
        parts = {b: R.attend(case, b, q[10 * b:10 * b + 10]) for b in (0, 2)}
        for b in parts:
            lse[10 * b:10 * b + 10] = parts[b][1].float()
        L.kv16_accumulate(cache, q.cuda(), lse.cuda(), i32([0, 10, 20, 30]), R.SCALE, 128)
        assert L.device_status() != 0
        for b, (_, _, p, _, _, dmax) in parts.items():
            w, tol = R.weight_of(p, dmax, 4)
            R.assert_within(R.tokens(cache, b, 100, "weight"), w + case.w[b].double(), tol + 16 * R.U32 * w, str(b))


# ------------------------------------------------------------------- evict

@pytest.mark.parametrize("dtype,paged,paged_dst", [(BF, True, True), (FP, False, True), (BF, True, False)])
@pytest.mark.parametrize("first,recent,top", [(4, 20, 40), (0, 0, 33), (1, 0, 0), (0, 64, 0), (5, 7, 500), (0, 0, 1), (40, 90, 1)])
def test_evict(L, dtype, paged, paged_dst, first, recent, top):
    keep = first + recent + top
    lens = [1500, keep + 1, keep, max(keep - 1, 1), 0, 700 + keep]
    case = R.Case(lens, 3, dtype, paged, seed=keep, weights=True)
    for b, n in enumerate(lens):                     # equal weights, zeros of both signs, NaN, infinity
        w = torch.round(case.w[b] * 8) / 8 - 0.25
        if n > 600:
            w[:, 100] = math.nan
            w[0, 101], w[1, 102] = math.inf, -math.inf
            w[:, 103:140:2] = -0.0
        case.w[b] = w
    src = case.cache(L)
    to = R.Case([keep] * len(lens), 3, dtype, paged_dst, seed=1, weights=True)
    dst = to.cache(L, [0] * len(lens))
    before = (dst.k.clone(), dst.v.clone(), dst.weight.clone())
    same = lambda a, b: torch.equal(torch.nan_to_num(a.float(), nan=1e30), torch.nan_to_num(b.float(), nan=1e30))
    for kept in (torch.full((len(lens), 3, keep), 9, dtype=torch.int32, device="cuda"), None):
        for x, y in zip((dst.k, dst.v, dst.weight), before):
            x.copy_(y)
        ws = L.alloc_workspace(L.kv16_evict_workspace_bytes(src, 4096, first, recent, top))
        L.kv16_evict(src, dst, 4096, first, recent, top, ws, kept=kept)
        assert L.device_status() == 0
        assert dst.n_tok.tolist() == [min(n, keep) for n in lens]
        for b, n in enumerate(lens):
            m = min(n, keep)
            for h in range(3):
                want = R.evicted(case.w[b][h].numpy(), n, first, recent, top)
                assert len(want) == m
                if kept is not None:
                    assert kept[b, h].tolist() == want + [-1] * (keep - m)
                assert same(R.tokens(dst, b, m, "k")[h], case.k[b][h][want])
                assert same(R.tokens(dst, b, m, "v")[h], case.v[b][h][want])
                assert same(R.tokens(dst, b, m, "weight")[h], case.w[b][h][want])
            if paged_dst and m < keep:               # what lies behind the kept tokens stays
                t = torch.arange(m, keep)
                at = (dst.block_table[b].cpu().long()[t // 32], slice(None), t % 32)
                assert same(dst.k.cpu()[at], before[0].cpu()[at])


def test_evict_long_rows(L):
    """Rows longer than what one block holds at once, nearly all weights equal."""
    n = 70000
    case = R.Case([n, n - 31], 1, BF, seed=2, weights=True)
    case.w[1] = torch.zeros(1, n - 31)
    case.w[1][0, 5::1000] = 1.0
    src = case.cache(L)
    to = R.Case([2000, 2000], 1, BF, seed=1, weights=False)
    dst = to.cache(L)
    ws = L.alloc_workspace(L.kv16_evict_workspace_bytes(src, n, 4, 100, 1896))
    kept = torch.empty((2, 1, 2000), dtype=torch.int32, device="cuda")
    L.kv16_evict(src, dst, n, 4, 100, 1896, ws, kept=kept)
    for b in range(2):
        want = R.evicted(case.w[b][0].numpy(), case.lens[b], 4, 100, 1896)
        assert kept[b, 0].tolist() == want
        assert torch.equal(R.tokens(dst, b, 2000, "v")[0], case.v[b][0][want])


def test_evict_bad_lengths_and_pages(L):
    case = R.Case([200, 200], 2, BF, weights=True)
    for spoil in ("length", "source", "destination"):
        src = case.cache(L, [200, 10**6] if spoil == "length" else None)
        to = R.Case([60, 60], 2, BF, weights=True)
        dst = to.cache(L, [0, 0])
        if spoil != "length":
            (src if spoil == "source" else dst).block_table[1, 1] = -1
        ws = L.alloc_workspace(L.kv16_evict_workspace_bytes(src, 256, 4, 16, 40))
        L.kv16_evict(src, dst, 256, 4, 16, 40, ws)
        assert L.device_status() != 0
        assert dst.n_tok.tolist()[0] == 60
        for h in range(2):
            want = R.evicted(case.w[0][h].numpy(), 200, 4, 16, 40)
            assert torch.equal(R.tokens(dst, 0, 60, "k")[h], case.k[0][h][want])


# ------------------------------------------------------- together, and how

def test_prompt_evict_decode_together(L):
    """Prompts written and attended in two parts, their weights gathered from
    the last queries, cut down to a budget into a second cache whose pages come
    from the allocator, then decode steps that append and gather weight; every
    output against the 64-bit form of the same steps."""
    B, Hkv, Hq, g = 2, 2, 8, 4
    prompts, parts = [310, 150], [[200, 31], [110, 119]]
    case = R.Case(prompts, Hkv, BF, seed=77)
    src = L.PagedKV16Cache(B, Hkv, 12, 30, weights=True)
    for b in range(B):
        src.map_blocks(b, -(-prompts[b] // 32), order=list(range(29, -1, -1)))
    qs = [case.normal(n, Hq) for n in prompts]
    done, weight = [0, 0], [torch.zeros((Hkv, n), dtype=torch.float64) for n in prompts]
    wtol = [torch.zeros((Hkv, n), dtype=torch.float64) for n in prompts]
    for part in parts:
        start = R.start_of(part)
        cut = lambda xs, dim: torch.cat([x.narrow(dim, d, n) for x, d, n in zip(xs, done, part)], dim)
        k_new, v_new = (cut(x, 1).transpose(0, 1).contiguous().cuda() for x in (case.k, case.v))
        q = cut(qs, 0).cuda()
        L.kv16_write(src, k_new, v_new, i32(start), i32(done))
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(src, Hq, q.shape[0], 384, 128, 4))
        L.kv16_attention(src, q, i32(start), R.SCALE, 384, out, ws, window=128, n_sink=4, lse=lse)
        L.kv16_accumulate(src, q, lse, i32(start), R.SCALE, 384, 128, 4, n_obs=32)
        for b in range(B):
            rows = slice(start[b], start[b + 1])
            lens = [d + n for d, n in zip(done, part)]
            o, z, p, tol, ztol, dmax = R.attend(case, b, qs[b][done[b]:lens[b]], 128, 4, lens=lens)
            R.assert_within(out[rows], o, tol, f"prompt {b}")
            w, t = R.weight_of(p[-32:], dmax[-32:], g)
            weight[b][:, :lens[b]] += w
            wtol[b][:, :lens[b]] += t + 4 * float(ztol.max()) * w
        done = [d + n for d, n in zip(done, part)]
    assert src.n_tok.tolist() == prompts and L.device_status() == 0
    for b in range(B):
        R.assert_within(R.tokens(src, b, prompts[b], "weight"), weight[b], wtol[b] + 8 * R.U32 * weight[b], "weights")
    keep = 4 + 30 + 62
    dst = L.PagedKV16Cache(B, Hkv, 5, 10, weights=True)
    for b in range(B):
        dst.map_blocks(b, 4)
    kept = torch.empty((B, Hkv, keep), dtype=torch.int32, device="cuda")
    ws = L.alloc_workspace(L.kv16_evict_workspace_bytes(src, 384, 4, 30, 62))
    gathered = [R.tokens(src, b, prompts[b], "weight").clone() for b in range(B)]
    L.kv16_evict(src, dst, 384, 4, 30, 62, ws, kept=kept)
    after = R.Case([0, 0], Hkv, BF, weights=True)
    for b in range(B):
        want = [R.evicted(gathered[b][h].numpy(), prompts[b], 4, 30, 62) for h in range(Hkv)]
        assert kept[b].tolist() == want
        pick = lambda x: torch.stack([x[h][want[h]] for h in range(Hkv)])
        after.k[b], after.v[b], after.w[b] = pick(case.k[b]), pick(case.v[b]), pick(gathered[b])
    src.release_blocks(0)
    src.release_blocks(1)
    assert sorted(src._free) == list(range(30)) and (src.block_table == -1).all()
    ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(dst, Hq, 160, 0, 0, True))
    for step in range(5):
        k, v, q = case.normal(B, Hkv), case.normal(B, Hkv), case.normal(B, Hq)
        pos = dst.n_tok.clone()
        L.kv16_write(dst, k.cuda(), v.cuda(), i32([0, 1, 2]), pos)
        out = torch.empty((B, Hq, 128), dtype=BF, device="cuda")
        L.kv16_decode_attention(dst, q.cuda(), R.SCALE, 160, out, ws, accumulate=True)
        for b in range(B):
            after.k[b] = torch.cat([after.k[b], k[b][:, None]], 1)
            after.v[b] = torch.cat([after.v[b], v[b][:, None]], 1)
            after.lens[b] = after.k[b].shape[1]
            o, _, p, tol, _, dmax = R.attend(after, b, q[b:b + 1])
            R.assert_within(out[b:b + 1], o, tol, f"step {step}")
            w, t = R.weight_of(p, dmax, g)
            old = torch.cat([after.w[b], torch.zeros(Hkv, 1)], 1)
            got = R.tokens(dst, b, after.lens[b], "weight")
            R.assert_within(got, w + old.double(), t + 2 * R.U32 * old.double(), f"weights {step}")
            after.w[b] = got.float()
    assert L.device_status() == 0


def test_decode_step_in_a_graph_and_on_another_stream(L):
    """write + decode captured once and replayed as the cache grows, on a stream
    of its own; two graphs that share a workspace, one after the other."""
    case = R.Case([40, 90], 2, BF, seed=4, weights=True)
    cache = case.cache(L)
    k, v, q = (torch.zeros((2, h, 128), dtype=BF, device="cuda") for h in (2, 2, 8))
    outs = [torch.zeros((2, 8, 128), dtype=BF, device="cuda") for _ in range(2)]
    start, pos = i32([0, 1, 2]), i32([40, 90])
    ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 8, 128, 0, 0, True))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        for o in outs:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=s):
                L.kv16_write(cache, k, v, start, pos)
                L.kv16_decode_attention(cache, q, R.SCALE, 128, o, ws, accumulate=True)
                pos.add_(1)
            graphs.append(gr)
        for step in range(4):
            kn, vn, qn = case.normal(2, 2), case.normal(2, 2), case.normal(2, 8)
            k.copy_(kn), v.copy_(vn), q.copy_(qn)
            graphs[step % 2].replay()
            s.synchronize()
            for b in range(2):
                case.k[b] = torch.cat([case.k[b], kn[b][:, None]], 1)
                case.v[b] = torch.cat([case.v[b], vn[b][:, None]], 1)
                case.lens[b] += 1
                o, _, p, tol, _, dmax = R.attend(case, b, qn[b:b + 1])
                R.assert_within(outs[step % 2][b:b + 1], o, tol, f"step {step}")
                w, t = R.weight_of(p, dmax, 4)
                old = torch.cat([case.w[b], torch.zeros(2, 1)], 1)
                got = R.tokens(cache, b, case.lens[b], "weight")
                R.assert_within(got, w + old.double(), t + 2 * R.U32 * old.double(), "weights")
                case.w[b] = got.float()
    assert L.device_status() == 0


def test_prompt_in_a_graph(L):
    """attention, accumulate and evict captured and replayed over new inputs."""
    case = R.Case([200, 130], 2, BF, seed=8, weights=True)
    cache = case.cache(L)
    dst = R.Case([80, 80], 2, BF, weights=True).cache(L)
    start = R.start_of([200, 50])
    q = torch.zeros((250, 8, 128), dtype=BF, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((250, 8), device="cuda")
    ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, 8, 250, 256))
    we = L.alloc_workspace(L.kv16_evict_workspace_bytes(cache, 256, 4, 36, 40))
    kept = torch.empty((2, 2, 80), dtype=torch.int32, device="cuda")
    st, w0 = i32(start), cache.weight.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        L.kv16_attention(cache, q, st, R.SCALE, 256, out, ws, lse=lse)
        L.kv16_accumulate(cache, q, lse, st, R.SCALE, 256)
        L.kv16_evict(cache, dst, 256, 4, 36, 40, we, kept=kept)
    for _ in range(2):
        qn = case.normal(250, 8)
        q.copy_(qn)
        cache.weight.copy_(w0)
        gr.replay()
        torch.cuda.synchronize()
        for b in range(2):
            o, z, p, tol, ztol, dmax = R.attend(case, b, qn[start[b]:start[b + 1]])
            R.assert_within(out[start[b]:start[b + 1]], o, tol, "out")
            got = R.tokens(cache, b, case.lens[b], "weight")
            w, t = R.weight_of(p, dmax, 4)
            R.assert_within(got, w + case.w[b].double(), t + 4 * float(ztol.max()) * w + 2 * R.U32, "weights")
            for h in range(2):
                assert kept[b, h].tolist() == R.evicted(got[h].numpy(), case.lens[b], 4, 36, 40)
    assert L.device_status() == 0


def test_offsets_past_32_bits(L):
    """A pool of more than 2^32 elements: the last pages are read and written."""
    Hkv, n_pages = 8, 140000                       # 140000 * 8 * 32 * 128 = 4.6e9 elements
    k = torch.empty((n_pages, Hkv, 32, 128), dtype=BF, device="cuda")
    v = torch.empty_like(k)
    w = torch.empty((n_pages, Hkv, 32), device="cuda")
    case = R.Case([100], Hkv, BF)
    table = i32([[n_pages - 1, 3, n_pages - 2, n_pages - 40]])
    cache = L.KV16Cache(k, v, i32([0]), block_table=table, weight=w)
    kn, vn = (x[0].transpose(0, 1).contiguous().cuda() for x in (case.k, case.v))
    L.kv16_write(cache, kn, vn, i32([0, 100]), i32([0]))
    q = case.normal(100, 32)
    out, lse = torch.empty((100, 32, 128), dtype=BF, device="cuda"), torch.empty((100, 32), device="cuda")
    ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, 32, 100, 128))
    L.kv16_attention(cache, q.cuda(), i32([0, 100]), R.SCALE, 128, out, ws, lse=lse)
    o, _, p, tol, ztol, dmax = R.attend(case, 0, q)
    R.assert_within(out, o, tol, "attention")
    L.kv16_accumulate(cache, q.cuda(), lse, i32([0, 100]), R.SCALE, 128)
    wt, t = R.weight_of(p, dmax, 4)
    t = t + 4 * float(ztol.max()) * wt
    R.assert_within(R.tokens(cache, 0, 100, "weight"), wt, t, "accumulate")
    ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 32, 128, 0, 0, True))
    one = torch.empty((1, 32, 128), dtype=BF, device="cuda")
    L.kv16_decode_attention(cache, q[-1:].cuda(), R.SCALE, 128, one, ws, accumulate=True)
    R.assert_within(one, o[-1:], tol[-1:], "decode")
    w1, t1 = R.weight_of(p[-1:], dmax[-1:], 4, n_before=100.0)
    R.assert_within(R.tokens(cache, 0, 100, "weight"), wt + w1, t + t1, "decode's weights")
    assert L.device_status() == 0


def test_binding_refuses(L):
    """Tensors that do not fit one another are refused before anything runs."""
    case = R.Case([40], 2, BF, weights=True)
    cache = case.cache(L)
    x = case.normal(1, 2).cuda()
    st, pos = i32([0, 1]), i32([0])
    out8 = torch.empty((1, 8, 128), dtype=BF, device="cuda")
    q = case.normal(1, 8).cuda()
    ws = L.alloc_workspace(1 << 20)
    n0 = L.kernel_launches()
    bad = [lambda: L.kv16_write(cache, x.float(), x, st, pos),
           lambda: L.kv16_write(cache, x[:, :1], x, st, pos),
           lambda: L.kv16_write(cache, x, x, st.long(), pos),
           lambda: L.kv16_write(cache, x, x, i32([0]), pos),
           lambda: L.kv16_write(cache, x, x, st, i32([0, 0])),
           lambda: L.kv16_write(cache, x.half(), x, st, pos),
           lambda: L.kv16_decode_attention(cache, q.half(), R.SCALE, 64, out8, ws),
           lambda: L.kv16_decode_attention(cache, q, R.SCALE, 64, out8[:, :4], ws),
           lambda: L.kv16_decode_attention(cache, torch.cat([q, q]), R.SCALE, 64, out8, ws),
           lambda: L.kv16_decode_attention(cache, q, R.SCALE, 64, out8.float(), ws),
           lambda: L.kv16_attention(cache, q, st, R.SCALE, 64, out8, ws, lse=torch.empty(3, device="cuda")),
           lambda: L.KV16Cache(cache.k, cache.v[:1], cache.n_tok, cache.block_table),
           lambda: L.KV16Cache(cache.k.float(), cache.v.float(), cache.n_tok, cache.block_table),
           lambda: L.KV16Cache(cache.k, cache.v, cache.n_tok.long(), cache.block_table)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    refused = [lambda: L.kv16_write(cache, x, x, st, cache.n_tok),
               lambda: L.kv16_attention(cache, q.transpose(0, 1), st, R.SCALE, 64, out8, ws),
               lambda: L.kv16_decode_attention(cache, q, math.nan, 64, out8, ws),
               lambda: L.kv16_decode_attention(cache, q, R.SCALE, 64, out8, ws, window=-1),
               lambda: L.kv16_decode_attention(cache, q, R.SCALE, 64, out8, ws[:100]),
               lambda: L.kv16_evict(cache, cache, 64, 1, 1, 1, ws)]
    for f in refused:
        with pytest.raises(L.OscarError):
            f()
    assert L.kernel_launches() == n0


# ------------------------------------------------- many items, odd placements

def test_attention_many_sequences(L):
    """Far more work than one round of the grid, of very unequal sizes."""
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(1, 220, (300,), generator=g).tolist()
    news = [max(1, int(n * f)) for n, f in zip(lens, torch.rand(300, generator=g).tolist())]
    for Hq, Hkv, window, sink in ((8, 2, 0, 0), (5, 1, 40, 3)):
        case = R.Case(lens, Hkv, BF, seed=Hq)
        run_attention(L, case, case.cache(L), news, Hq, window, sink, extra=1)


@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (1, 1)])
def test_smallest_cache(L, Hq, Hkv):
    """One sequence of one token in a cache with room for one, and its step."""
    case = R.Case([1], Hkv, FP, paged=False, slack=0, weights=True)
    cache = case.cache(L)
    assert cache.capacity == 1
    run_attention(L, case, cache, [1], Hq)
    run_decode(L, case, cache, Hq, accumulate=True)


def test_outputs_at_16_byte_addresses(L):
    """Outputs need 16-byte alignment, no more."""
    case = R.Case([150, 40], 2, BF, seed=12)
    cache = case.cache(L)
    q = case.normal(190, 8)
    flat = torch.zeros(190 * 8 * 128 + 8, dtype=BF, device="cuda")
    out = flat[8:].view(190, 8, 128)
    assert out.data_ptr() % 32 == 16
    ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, 8, 190, 256))
    L.kv16_attention(cache, q.cuda(), i32([0, 150, 190]), R.SCALE, 256, out, ws)
    for b, rows in enumerate((slice(0, 150), slice(150, 190))):
        o, _, _, tol, _, _ = R.attend(case, b, q[rows])
        R.assert_within(out[rows], o, tol, str(b))
    one = flat[8:8 + 2 * 8 * 128].view(2, 8, 128)
    last = q[[149, 189]]
    ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 8, 256))
    L.kv16_decode_attention(cache, last.cuda(), R.SCALE, 256, one, ws)
    for b in range(2):
        o, _, _, tol, _, _ = R.attend(case, b, last[b:b + 1])
        R.assert_within(one[b:b + 1], o, tol, str(b))
    assert L.device_status() == 0


@pytest.mark.parametrize("lens,Hq,Hkv,n_obs,window,sink", [
    ([2500], 16, 1, 0, 0, 0),            # few items: clusters of eight share them
    ([900, 700], 6, 2, 0, 0, 0),         # clusters, groups that do not divide a tile
    (None, 16, 8, 20, 0, 0),             # many items of 256 keys, whole and partial
    (None, 24, 8, 0, 100, 3)])
def test_accumulate_item_sizes(L, lens, Hq, Hkv, n_obs, window, sink):
    if lens is None:
        g = torch.Generator().manual_seed(Hq)
        lens = torch.randint(1, 420, (40,), generator=g).tolist()
    news = [max(1, n - n // 3) for n in lens]
    case = R.Case(lens, Hkv, BF, seed=Hq, weights=True)
    cache, start = case.cache(L), R.start_of(news)
    q = case.normal(start[-1], Hq)
    out, lse = torch.empty((start[-1], Hq, 128), dtype=BF, device="cuda"), torch.empty((start[-1], Hq), device="cuda")
    ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, Hq, start[-1], cache.capacity, window, sink))
    L.kv16_attention(cache, q.cuda(), i32(start), R.SCALE, cache.capacity, out, ws, window, sink, lse)
    L.kv16_accumulate(cache, q.cuda(), lse, i32(start), R.SCALE, cache.capacity, window, sink, n_obs)
    assert L.device_status() == 0
    for b, n in enumerate(lens):
        o, z, p, tol, ztol, dmax = R.attend(case, b, q[start[b]:start[b + 1]], window, sink)
        R.assert_within(out[start[b]:start[b + 1]], o, tol, f"out {b}")
        skip = max(0, news[b] - n_obs) if n_obs else 0
        w, t = R.weight_of(p[skip:], dmax[skip:], Hq // Hkv)
        R.assert_within(R.tokens(cache, b, n, "weight"), w + case.w[b].double(),
                        t + 4 * float(ztol.max()) * w, f"weight {b}")


def test_calls_on_two_streams_at_once(L):
    """The same caches read by attention and decode on two streams, each with a
    workspace of its own."""
    case = R.Case([700, 300], 2, BF, seed=21)
    cache = case.cache(L)
    q, q1 = case.normal(400, 8), case.normal(2, 8)
    qd, q1d, st = q.cuda(), q1.cuda(), i32([0, 300, 400])
    streams = [torch.cuda.Stream() for _ in range(2)]
    out, one = torch.empty_like(qd), torch.empty_like(q1d)
    wa = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, 8, 400, 800))
    wd = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 8, 800))
    torch.cuda.synchronize()
    for _ in range(20):
        L.kv16_attention(cache, qd, st, R.SCALE, 800, out, wa, stream=streams[0])
        L.kv16_decode_attention(cache, q1d, R.SCALE, 800, one, wd, stream=streams[1])
    torch.cuda.synchronize()
    assert L.device_status() == 0
    for b, rows in enumerate((slice(0, 300), slice(300, 400))):
        o, _, _, tol, _, _ = R.attend(case, b, q[rows])
        R.assert_within(out[rows], o, tol, str(b))
        o, _, _, tol, _, _ = R.attend(case, b, q1[b:b + 1])
        R.assert_within(one[b:b + 1], o, tol, str(b))
