"""The 16-bit cache's calls at the edges of what their documentation allows:
bad lengths under windows, values that are not finite, weights of very unequal
size, waits that run out, rows too long to hold.  Against the same plain 64-bit
forms as the other tests of these calls."""
import math

import pytest
import torch

from tests import _kv16_ref as R
from tests.test_gpu_kv16 import i32, run_attention, run_decode  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
TOP = 2**31 - 1


@pytest.fixture(scope="module")
def L():
    from int2_kv_cache_02_gb300 import _build
    _build.build()
    from int2_kv_cache_02_gb300 import oscar
    oscar.device_status()
    return oscar


# ------------------------------------------------- bad lengths under windows

@pytest.mark.parametrize("window,sink", [(TOP, 0), (TOP, TOP), (TOP - 5, 4), (5, 0), (40, 3), (1, 200)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (3, 1)])
def test_fewer_tokens_than_queries_under_a_window(L, window, sink, Hq, Hkv):
    """A sequence that holds fewer tokens than it has queries, under windows up to
    the widest: recorded, and every other sequence is right, before it and behind
    it in the order of work."""
    lens, news = [300, 100, 200, 260], [300, 60, 40, 200]
    for bad in (3, 0, -5, 10**6):
        case = R.Case(lens, Hkv, BF, seed=Hq, weights=True)
        cache, start = case.cache(L, [300, bad, 200, 260]), R.start_of(news)
        q = case.normal(start[-1], Hq)
        out = torch.zeros((start[-1], Hq, 128), dtype=BF, device="cuda")
        lse = torch.zeros((start[-1], Hq), device="cuda")
        ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, Hq, start[-1], 320, window, sink))
        L.kv16_attention(cache, q.cuda(), i32(start), R.SCALE, 320, out, ws, window, sink, lse)
        assert L.device_status() != 0 and L.device_status() == 0
        L.kv16_accumulate(cache, q.cuda(), lse, i32(start), R.SCALE, 320, window, sink)
        assert L.device_status() != 0
        for b in (0, 2, 3):
            rows = slice(start[b], start[b + 1])
            o, z, p, tol, ztol, dmax = R.attend(case, b, q[rows], window, sink)
            R.assert_within(out[rows], o, tol, f"out {b}")
            R.assert_within(lse[rows], z, ztol, f"lse {b}")
            w, t = R.weight_of(p, dmax, Hq // Hkv)
            R.assert_within(R.tokens(cache, b, lens[b], "weight"), w + case.w[b].double(),
                            t + 4 * float(ztol.max()) * w + 2 * R.U32, f"weight {b}")


@pytest.mark.parametrize("window,sink", [(TOP, 0), (TOP, TOP), (5, 3)])
def test_decode_bad_lengths_under_a_window(L, window, sink):
    for bad in (-5, -TOP, TOP, 10**6):
        case = R.Case([300, 100, 33], 2, BF, weights=True)
        cache = case.cache(L, [300, bad, 33])
        q = case.normal(3, 8)
        out = torch.zeros((3, 8, 128), dtype=BF, device="cuda")
        ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 8, 320, window, sink, True))
        L.kv16_decode_attention(cache, q.cuda(), R.SCALE, 320, out, ws, window, sink, accumulate=True)
        assert L.device_status() != 0
        assert (ws[:65536].view(torch.int32) == 0).all()
        for b in (0, 2):
            o, _, p, tol, _, dmax = R.attend(case, b, q[b:b + 1], window, sink)
            R.assert_within(out[b:b + 1], o, tol, str(b))
            w, t = R.weight_of(p, dmax, 4)
            R.assert_within(R.tokens(cache, b, case.lens[b], "weight"), w + case.w[b].double(),
                            t + 2 * R.U32, str(b))


# --------------------------------------------------- values that are not finite

def poke(case, cache, b, t, k=None, v=None, channel=None, head=0):
    """Puts numbers that are not finite into a token of the device's cache (the
    host's keep what they are)."""
    at = (b, head, t) if cache.block_table is None else (int(cache.block_table[b, t // 32]), head, t % 32)
    if k is not None:
        cache.k[at] = k
    if v is not None:
        cache.v[at if channel is None else at + (channel,)] = v


def attention_of(L, case, cache, news, Hq, window=0, sink=0):
    start = R.start_of(news)
    q = case.normal(start[-1], Hq)
    out = torch.full((start[-1], Hq, 128), 7.0, dtype=case.dtype, device="cuda")
    lse = torch.full((start[-1], Hq), 7.0, device="cuda")
    ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, Hq, start[-1], cache.capacity, window, sink))
    L.kv16_attention(cache, q.cuda(), i32(start), R.SCALE, cache.capacity, out, ws, window, sink, lse)
    assert L.device_status() == 0
    return start, q, out.cpu(), lse.cpu()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lens,news", [([700, 6000, 300], [700, 6000, 300]), ([9000, 4000], [5, 3])])
def test_nan_key_makes_its_own_rows_nan(L, dtype, lens, news):
    """A NaN in the first key of a sequence: all of that KV head's rows are NaN,
    output and lse, whole prompts and split caches alike; nothing else changes."""
    case = R.Case(lens, 2, dtype, seed=1)
    cache = case.cache(L)
    poke(case, cache, 1, 0, k=math.nan)
    start, q, out, lse = attention_of(L, case, cache, news, 8)
    mine = slice(start[1], start[2])
    assert torch.isnan(out[mine, :4]).all() and torch.isnan(lse[mine, :4]).all()
    for b in range(len(lens)):
        rows = slice(max(start[b], start[b + 1] - 40), start[b + 1])
        o, z, _, tol, ztol, _ = R.attend(case, b, q[rows])
        h = slice(4, 8) if b == 1 else slice(0, 8)
        R.assert_within(out[rows, h], o[:, h], tol[:, h], f"out {b}")
        R.assert_within(lse[rows, h], z[:, h], ztol[:, h], f"lse {b}")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lens,news,window,sink", [
    ([700, 900], [700, 900], 0, 0), ([900, 9000], [3, 5], 0, 0), ([300, 900], [300, 900], 70, 4)])
def test_a_value_reaches_its_channel_where_it_is_seen(L, dtype, what, lens, news, window, sink):
    """One channel of one value is NaN or infinite: the rows that see the token
    have that in this channel, and what they have without it in all others; rows
    that do not see it are as without it."""
    case = R.Case(lens, 2, dtype, seed=2)
    cache = case.cache(L)
    token, ch = {0: 2, 70: 500}[window], 37
    poke(case, cache, 1, token, v=what, channel=ch, head=1)
    start, q, out, lse = attention_of(L, case, cache, news, 6, window, sink)
    for b in range(2):
        rows = slice(start[b], start[b + 1])
        o, z, _, tol, ztol, _ = R.attend(case, b, q[rows], window, sink)
        if b == 1:
            at = torch.arange(lens[1] - news[1], lens[1])
            see = R.visible(at, lens[1], window, sink)[:, token]
            got = out[rows, 3:, ch][see]
            assert torch.isnan(got).all() if math.isnan(what) else (got == what).all()
            assert see.any()
            # that channel has been judged: the rest against the host's values
            out[rows, 3:, ch] = torch.where(see[:, None], o[:, 3:, ch].to(dtype), out[rows, 3:, ch])
        R.assert_within(out[rows], o, tol, f"out {b}")
        R.assert_within(lse[rows], z, ztol, f"lse {b}")


@pytest.mark.parametrize("n,dtype,what", [
    (100000, BF, math.nan), (100000, FP, math.inf), (1000000, BF, math.inf)])
def test_hidden_value_of_a_long_sequence(L, n, dtype, what):
    """The last value of a long sequence is not finite: the queries before it in its
    tile are as without it, however long their rows take (a million tokens: longer
    than the waits allow otherwise), and so are the short sequences whose work comes
    after them on the same multiprocessors."""
    new, short = 20000, 400
    case = R.Case([n] + [40] * short, 1, dtype, paged=False, slack=0, seed=3)
    blocks = n // 32
    table = torch.full((1 + short, blocks), -1, dtype=torch.int32)
    table[0] = torch.arange(blocks)
    table[1:, :2] = blocks + torch.arange(2 * short, dtype=torch.int32).view(short, 2)
    k = torch.zeros((blocks + 2 * short, 1, 32, 128), dtype=dtype, device="cuda")
    v = torch.zeros_like(k)
    for x, y in ((k, case.k), (v, case.v)):
        x[:blocks] = y[0].view(blocks, 1, 32, 128).cuda()
        tail = torch.zeros((short, 64, 128), dtype=dtype)
        tail[:, :40] = torch.cat(y[1:])
        x[blocks:] = tail.view(2 * short, 1, 32, 128).cuda()
    cache = L.KV16Cache(k, v, i32(case.lens), block_table=table.cuda())
    poke(case, cache, 0, n - 1, v=what)
    start, q, out, lse = attention_of(L, case, cache, [new] + [40] * short, 1)
    seen = out[new - 1].float()
    assert torch.isnan(seen).all() if math.isnan(what) else (seen == math.inf).all()
    for i in (new - 2, new - 100, new - 129, 0):
        o, z, _, tol, ztol, _ = R.attend(case, 0, q[i:i + 1], lens=[n - new + i + 1])
        R.assert_within(out[i:i + 1], o, tol, str(i))
        R.assert_within(lse[i:i + 1], z, ztol, str(i))
    assert torch.isfinite(out[:new - 1].float()).all() and torch.isfinite(lse).all()
    for b in range(1, 1 + short, 23):
        rows = slice(start[b], start[b + 1])
        o, z, _, tol, ztol, _ = R.attend(case, b, q[rows])
        R.assert_within(out[rows], o, tol, str(b))


# ------------------------------------------------------- waits that run out

@pytest.mark.parametrize("lens,Hq,Hkv", [([20000], 4, 1), ([5000, 1, 9000, 64, 0, 3000], 16, 2), ([50] * 300, 8, 4)])
def test_decode_workspace_after_waits_run_out(L, lens, Hq, Hkv):
    """When no copy lands in time the status word says so, the rows' counters come
    back to zero, and the next call on the workspace is right."""
    case = R.Case(lens, Hkv, BF, seed=9)
    cache = case.cache(L)
    q = case.normal(case.B, Hq).cuda()
    out = torch.empty_like(q)
    ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, Hq, cache.capacity))
    for _ in range(2):
        L.selftest_kv16_decode_timeout(cache, q, cache.capacity, out, ws)
        assert L.device_status() == 7 and L.device_status() == 0
        assert (ws[:65536].view(torch.int32) == 0).all()
    run_decode(L, case, cache, Hq, ws=ws)


def test_tensor_core_waits_run_out_together(L):
    """A wait that gives up takes the other warps of its block with it, none does
    while a warp is busy, and calls that use the same tensor memory are right after."""
    for iterations in (1, 64, 1000):
        report = torch.full((3,), -1, dtype=torch.int32, device="cuda")
        L.selftest_tc_wait_timeout(report, iterations)
        assert L.device_status() == 7 and L.device_status() == 0
        assert report.tolist() == [1, 1, 0]
    case = R.Case([300, 200], 2, BF, seed=10, weights=True)
    run_attention(L, case, case.cache(L), [300, 100], 8)


# ------------------------------------------------ weights of very unequal size

def far_bound(case, b, q, rel, flush, **kw):
    """As R.attend, with the probabilities' rounding taken token by token: off by
    `rel` of itself, or by `flush` of the row's largest where that is more."""
    o, z, p, _, ztol, dmax = R.attend(case, b, q, **kw)
    n, g = p.shape[2], q.shape[1] // case.Hkv
    v = case.v[b].double().repeat_interleave(g, 0)[:, :n].abs()
    each = torch.maximum(rel * p, flush * p.amax(-1, keepdim=True)) + (4 * dmax[..., None] + 2 * n * R.U32) * p
    tol = R.U[case.dtype] * o.abs() + torch.einsum("qhn,hnd->qhd", each, v) + 2.0 ** -25
    return o, z, tol, ztol


# fp16: the prompt's probabilities stand at 2^7 (or more) where the largest is 1,
# the decode's up to 2^14 and in two parts; half the smallest number is 2^-25
FAR = {BF: (2.0 ** -8, 0.0, 2.0 ** -15, 0.0), FP: (2.0 ** -11, 2.0 ** -32, 2.0 ** -21, 2.0 ** -39)}


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("heavy", [0, 1500])
@pytest.mark.parametrize("octaves", [20.0, 23.4, 24.4, 26.0])
def test_one_token_far_heavier_than_the_rest(L, dtype, heavy, octaves):
    """One token, with a value of zero as a sink has it, weighs 2^20 to 2^26 times
    what any other does: the others still make the output."""
    lens, news = [8192, 3001], [5, 1400]
    case = R.Case(lens, 1, dtype, seed=4, factor=0.05)
    e = torch.where(torch.rand(128, generator=case.gen) < 0.5, -1.0, 1.0)
    size = (octaves * math.log(2) / (128 * R.SCALE)) ** 0.5
    for b in range(2):
        case.k[b][0, heavy] = (size * e).to(dtype)
        case.v[b] = (case.v[b].float() * 0.25 + 1.0).to(dtype)
        case.v[b][0, heavy] = 0.0
    cache = case.cache(L)
    case.normal = lambda n, h: (size * e).to(dtype).expand(n, h, 128).contiguous()
    start, q, out, lse = attention_of(L, case, cache, news, 4)
    rel, flush, rel2, flush2 = FAR[dtype]
    for b in range(2):
        rows = slice(start[b], start[b + 1])
        o, z, tol, ztol = far_bound(case, b, q[rows], rel, flush)
        R.assert_within(out[rows], o, tol, f"prompt {b}")
        R.assert_within(lse[rows], z, ztol, f"lse {b}")
    q1 = q[[start[1] - 1, start[2] - 1]]
    one = torch.empty((2, 4, 128), dtype=dtype, device="cuda")
    ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 4, cache.capacity))
    L.kv16_decode_attention(cache, q1.cuda(), R.SCALE, cache.capacity, one, ws)
    assert L.device_status() == 0
    for b in range(2):
        o, _, tol, _ = far_bound(case, b, q1[b:b + 1], rel2, flush2)
        R.assert_within(one[b:b + 1], o, tol, f"decode {b}")


# ------------------------------------------------------------- the same bits

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("Hq", [3, 5, 6, 7, 12, 15])
def test_prompt_bits_do_not_depend_on_what_memory_held(L, dtype, Hq):
    """Groups that do not fill a tile's rows: the same call gives the same bits after
    calls that leave NaN or large numbers in shared memory."""
    case = R.Case([300, 90, 41], 1, dtype, seed=Hq)
    cache, q = case.cache(L), case.normal(431, Hq).cuda()
    fill = R.Case([64] * 320, 1, dtype, paged=False, slack=0, seed=1)
    full, qf = fill.cache(L), fill.normal(320 * 64, 8).cuda()
    got = []
    for x in (0.0, math.nan, 300.0, math.inf):
        other = torch.empty_like(qf)
        ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(full, 8, qf.shape[0], 64))
        L.kv16_attention(full, qf * x, i32(R.start_of([64] * 320)), R.SCALE, 64, other, ws)
        out, lse = torch.empty_like(q), torch.empty((431, Hq), device="cuda")
        ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, Hq, 431, 320))
        L.kv16_attention(cache, q, i32([0, 300, 390, 431]), 3 * R.SCALE, 320, out, ws, lse=lse)
        got.append((out, lse))
    assert L.device_status() == 0
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("Hq", [1, 4, 7])
def test_prompt_bits_do_not_depend_on_the_neighbours(L, dtype, Hq):
    """A sequence's results are the same bits whatever the queries of the others."""
    case = R.Case([300, 90, 41], 1, dtype, seed=Hq)
    cache, q = case.cache(L), case.normal(431, Hq)
    got = []
    for x in (1.0, 100.0, math.nan):
        mixed = q.clone()
        mixed[:300] *= x
        mixed[390:] *= x
        out, lse = torch.empty((431, Hq, 128), dtype=dtype, device="cuda"), torch.empty((431, Hq), device="cuda")
        ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, Hq, 431, 320))
        L.kv16_attention(cache, mixed.cuda(), i32([0, 300, 390, 431]), 3 * R.SCALE, 320, out, ws, lse=lse)
        got.append((out[300:390], lse[300:390]))
    assert L.device_status() == 0
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("scale,size", [(0.0, 1e17), (1e-33, 1e16), (-3e-34, 1e16), (1e-38, 1e18), (1e-41, 1e18)])
def test_scales_next_to_zero(L, scale, size):
    """Scales down to the smallest numbers and to zero, with keys and queries so large
    that they count (or, at zero, do not)."""
    case = R.Case([200, 700], 1, BF, seed=7, factor=size, weights=True)
    cache, start = case.cache(L), [0, 200, 400]
    q = (case.normal(400, 4).float() * size).to(BF)
    out, lse = torch.empty((400, 4, 128), dtype=BF, device="cuda"), torch.empty((400, 4), device="cuda")
    ws = L.alloc_workspace(L.kv16_attention_workspace_bytes(cache, 4, 400, 704))
    L.kv16_attention(cache, q.cuda(), i32(start), scale, 704, out, ws, lse=lse)
    one = torch.empty((2, 4, 128), dtype=BF, device="cuda")
    q1 = q[[199, 399]]
    ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 4, 704))
    L.kv16_decode_attention(cache, q1.cuda(), scale, 704, one, ws)
    L.kv16_accumulate(cache, q.cuda(), lse, i32(start), scale, 704)
    assert L.device_status() == 0
    # the scale as the calls take it: a float, times log2(e) to a float
    s32 = torch.tensor(scale, dtype=torch.float32)
    s64 = float((s32 * torch.tensor(1.4426950408889634)).double()) / 1.4426950408889634
    for b in range(2):
        rows = slice(start[b], start[b + 1])
        o, z, p, tol, ztol, dmax = R.attend(case, b, q[rows], scale=s64)
        R.assert_within(out[rows], o, tol, f"out {b}")
        R.assert_within(lse[rows], z, ztol, f"lse {b}")
        R.assert_within(one[b:b + 1], o[-1:], tol[-1:], f"decode {b}")
        w, t = R.weight_of(p, dmax, 4)
        R.assert_within(R.tokens(cache, b, case.lens[b], "weight"), w + case.w[b].double(),
                        t + 4 * float(ztol.max()) * w + 2 * R.U32, f"weight {b}")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv", [([700, 900, 40], 6, 2), ([9000, 20000, 1], 8, 2), ([700, 900, 40], 16, 1)])
def test_decode_of_values_that_are_not_finite(L, dtype, accumulate, lens, Hq, Hkv):
    """Infinite and NaN values that a query sees reach its output as they are: the
    infinity, NaN for a NaN or infinities of both signs; every other channel, row
    and weight as without them."""
    case = R.Case(lens, Hkv, dtype, seed=5, weights=True)
    cache, h = case.cache(L), Hkv - 1
    want = {3: math.inf, 4: -math.inf, 70: math.nan, 71: math.nan, 127: math.inf, 0: -math.inf}
    n = lens[1]
    for t, ch, x in ((2, 3, math.inf), (n - 1, 4, -math.inf), (n // 2, 70, math.nan), (40, 71, math.inf),
                     (n - 40, 71, -math.inf), (50, 127, math.inf), (n - 2, 127, math.inf), (n // 3, 0, -math.inf)):
        poke(case, cache, 1, t, v=x, channel=ch, head=h)
    # (each channel's token also as the one whose probability is the largest)
    q = case.normal(3, Hq)
    g = Hq // Hkv
    for i, t in enumerate((2, n - 1, n // 2, 40, 50, n // 3)[:g]):
        q[1, h * g + i] = (3 * case.k[1][h, t].float()).to(dtype)
    out = torch.empty((3, Hq, 128), dtype=dtype, device="cuda")
    ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, Hq, cache.capacity, 0, 0, accumulate))
    L.kv16_decode_attention(cache, q.cuda(), R.SCALE, cache.capacity, out, ws, accumulate=accumulate)
    assert L.device_status() == 0 and (ws[:65536].view(torch.int32) == 0).all()
    out = out.cpu()
    for b in range(3):
        o, _, p, tol, _, dmax = R.attend(case, b, q[b:b + 1])
        if b == 1:
            for ch, x in want.items():
                got = out[1, h * g:, ch].float()
                assert torch.isnan(got).all() if math.isnan(x) else (got == x).all(), ch
                out[1, h * g:, ch] = o[0, h * g:, ch].to(dtype)
        R.assert_within(out[b:b + 1], o, tol, f"out {b}")
        if accumulate:
            w, t = R.weight_of(p, dmax, g)
            R.assert_within(R.tokens(cache, b, lens[b], "weight"), w + case.w[b].double(),
                            t + 2 * R.U32 * case.w[b].double(), f"weight {b}")


def test_decode_nan_score_beside_infinite_values(L):
    """A row whose scores hold a NaN is NaN in every channel, infinite values or not."""
    case = R.Case([500, 300], 1, BF, seed=6)
    cache = case.cache(L)
    poke(case, cache, 0, 9, k=math.nan)
    poke(case, cache, 0, 70, v=math.inf, channel=5)
    out = torch.empty((2, 4, 128), dtype=BF, device="cuda")
    q = case.normal(2, 4)
    ws = L.alloc_workspace(L.kv16_decode_workspace_bytes(cache, 4, cache.capacity))
    L.kv16_decode_attention(cache, q.cuda(), R.SCALE, cache.capacity, out, ws)
    assert torch.isnan(out[0]).all() and L.device_status() == 0
    o, _, _, tol, _, _ = R.attend(case, 1, q[1:])
    R.assert_within(out[1:], o, tol, "the other row")


# ----------------------------------------------------- rows too long to hold

def test_evict_rows_too_long_to_hold(L):
    """A capacity beyond what a cluster's shared memory holds (8 times 48K tokens):
    the weights are read again in every pass.  Rows of a few thousand tokens, one
    over many pages of the table, with NaN, infinite and equal weights."""
    blocks = 13000
    lens = [5000, 4000, 300, 0, 20000]
    case = R.Case(lens, 2, BF, seed=11, weights=True)
    for b in (0, 1, 4):
        w = torch.round(case.w[b] * 4) / 4
        w[0, 700:720] = math.nan
        w[1, 30], w[1, 31] = math.inf, -math.inf
        case.w[b] = w
    case.w[1][:] = 0.25
    small = case.cache(L)
    table = torch.full((5, blocks), -1, dtype=torch.int32, device="cuda")
    table[:, :small.block_table.shape[1]] = small.block_table
    src = L.KV16Cache(small.k, small.v, small.n_tok, block_table=table, weight=small.weight)
    assert src.capacity > 8 * 48 * 1024
    for first, recent, top in ((4, 100, 400), (0, 0, 1), (40, 60, 3000)):
        keep = first + recent + top
        dst = R.Case([keep] * 5, 2, BF, seed=1, weights=True).cache(L, [0] * 5)
        ws = L.alloc_workspace(L.kv16_evict_workspace_bytes(src, src.capacity, first, recent, top))
        kept = torch.full((5, 2, keep), 9, dtype=torch.int32, device="cuda")
        L.kv16_evict(src, dst, src.capacity, first, recent, top, ws, kept=kept)
        assert L.device_status() == 0
        assert dst.n_tok.tolist() == [min(n, keep) for n in lens]
        for b, n in enumerate(lens):
            m = min(n, keep)
            for h in range(2):
                want = R.evicted(case.w[b][h].numpy(), n, first, recent, top)
                assert kept[b, h].tolist() == want + [-1] * (keep - m)
                assert torch.equal(R.tokens(dst, b, m, "k")[h], case.k[b][h][want])
                assert torch.equal(R.tokens(dst, b, m, "v")[h], case.v[b][h][want])


def test_evict_rows_over_a_cluster_keep_the_status_clean(L):
    """Rows of 70000 tokens, held by a cluster: the right tokens and no error."""
    n = 70000
    case = R.Case([n, n - 31], 1, BF, seed=2, weights=True)
    src = case.cache(L)
    dst = R.Case([2000, 2000], 1, BF, seed=1, weights=False).cache(L)
    ws = L.alloc_workspace(L.kv16_evict_workspace_bytes(src, n, 4, 100, 1896))
    kept = torch.empty((2, 1, 2000), dtype=torch.int32, device="cuda")
    L.kv16_evict(src, dst, n, 4, 100, 1896, ws, kept=kept)
    assert L.device_status() == 0
    for b in range(2):
        assert kept[b, 0].tolist() == R.evicted(case.w[b][0].numpy(), case.lens[b], 4, 100, 1896)
