"""Plain 64-bit forms of the 16-bit cache's operators and the error bounds that
the tests hold the kernels to (test infrastructure).

A Case holds a cache's contents in token order on the host; `cache()` lays them
out on the device, paged in a shuffled order or contiguous, with every place
that holds no token filled with NaN.
"""
import math

import torch

SCALE = 1.0 / math.sqrt(128)
U = {torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2, torch.float16: torch.finfo(torch.float16).eps / 2}
U32 = 2.0 ** -24


class Case:
    def __init__(self, lens, Hkv, dtype=torch.bfloat16, paged=True, seed=0, slack=1, weights=False,
                 factor=1.0):
        """Sequences of lens[b] tokens; `slack` more blocks (or 19 more tokens
        per slack, contiguous) than the longest needs."""
        self.lens, self.Hkv, self.dtype, self.paged = list(lens), Hkv, dtype, paged
        self.B = len(lens)
        self.gen = torch.Generator().manual_seed(1000 + seed)
        self.k = [self.normal(Hkv, n) * factor for n in lens]
        self.v = [self.normal(Hkv, n) for n in lens]
        self.w = [torch.rand((Hkv, n), generator=self.gen).float() if weights else None
                  for n in lens]
        most = max(max(lens), 1)
        self.blocks = -(-most // 32) + slack
        self.T_cap = self.blocks * 32 if paged else most + 19 * slack

    def normal(self, *shape):
        return torch.randn(shape + (128,), generator=self.gen).to(self.dtype)

    def cache(self, L, n_tok=None):
        B, Hkv = self.B, self.Hkv
        n_tok = torch.tensor(self.lens if n_tok is None else n_tok, dtype=torch.int32)
        if self.paged:
            order = torch.randperm(B * self.blocks + 3, generator=self.gen)
            table = order[: B * self.blocks].view(B, self.blocks).int()
            shape = (B * self.blocks + 3, Hkv, 32)
        else:
            table, shape = None, (B, Hkv, self.T_cap)
        k, v = (torch.full(shape + (128,), math.nan, dtype=self.dtype) for _ in range(2))
        w = torch.full(shape, math.nan) if self.w[0] is not None else None
        for b, n in enumerate(self.lens):
            t = torch.arange(n)
            if self.paged:
                at = (table[b].long()[t // 32], slice(None), t % 32)
            else:
                at = (b, slice(None), t)
            put = (lambda x: x.transpose(0, 1)) if self.paged else (lambda x: x)
            k[at], v[at] = put(self.k[b]), put(self.v[b])
            if w is not None:
                w[at] = put(self.w[b])
        table = table.cuda() if table is not None else None
        return L.KV16Cache(k.cuda(), v.cuda(), n_tok.cuda(), block_table=table,
                           weight=w.cuda() if w is not None else None)


def tokens(cache, b, n, name="k"):
    """[Hkv][n]... of sequence b, read back from a cache."""
    x = getattr(cache, name).cpu()
    t = torch.arange(n)
    if cache.block_table is None:
        return x[b][:, :n]
    return x[cache.block_table[b].cpu().long()[t // 32], :, t % 32].transpose(0, 1)


def start_of(news):
    s = [0]
    for n in news:
        s.append(s[-1] + n)
    return s


def visible(at, n, window, sink):
    j = torch.arange(n)
    at = torch.as_tensor(at)[:, None]
    see = j <= at
    if window:
        see = see & ((j > at - window) | (j < sink))
    return see


def attend(case, b, q, window=0, sink=0, scale=SCALE, lens=None):
    """q [nq][Hq][128], the last tokens' queries of sequence b ->
    out, lse, p [nq][Hq](..), and the elementwise bounds of out and lse.

    Bounds.  s is a sum of 128 exact products in fp32, each partial sum rounded:
    |ds| <= 129 u32 sum|q k| scale; the base-2 argument adds 2 u32 |s|; so a
    probability is off by a factor e^d - 1 <= 2 d, d = ds + 2^-21 (exponential).
    A probability is rounded to the type once (relative u; in fp16 absolutely
    2^-25 of the largest below 2^-14), sums over n tokens in fp32 are off by
    n u32 of the absolute sum, and the output is rounded once more."""
    n = (case.lens if lens is None else lens)[b]
    nq, Hq, _ = q.shape
    g = Hq // case.Hkv
    q = q.double()
    k = case.k[b].double().repeat_interleave(g, 0)
    v = case.v[b].double().repeat_interleave(g, 0)
    s = torch.einsum("qhd,hnd->qhn", q, k[:, :n]) * scale
    see = visible(torch.arange(n - nq, n), n, window, sink)[:, None]
    m = torch.where(see, s, -math.inf)
    lse = torch.logsumexp(m, -1) if n else torch.full((nq, Hq), -math.inf, dtype=torch.float64)
    p = torch.where(see, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None]), 0.0)
    out = torch.einsum("qhn,hnd->qhd", p, v[:, :n])
    absqk = torch.einsum("qhd,hnd->qhn", q.abs(), k[:, :n].abs()) * abs(scale)
    d = (129 * U32 * absqk + 2 * U32 * s.abs() + 2.0 ** -21)
    d = torch.where(see, d, 0.0)
    dmax = d.amax(-1) if n else torch.zeros((nq, Hq), dtype=torch.float64)
    u = U[case.dtype]
    a = torch.einsum("qhn,hnd->qhd", p, v[:, :n].abs())
    tol = u * out.abs() + (u + 4 * dmax + 2 * n * U32)[..., None] * a + 1e-30
    if case.dtype == torch.float16:
        tol = tol + n * 2.0 ** -25 * (v[:, :n].abs().amax() if n else 0.0) + 2.0 ** -25
    lse_tol = dmax + 2 * n * U32 + 8 * U32 * (1 + lse.abs())
    return out, lse, p, tol, torch.where(lse == -math.inf, 0.0, lse_tol), dmax


def weight_of(p, dmax, g, n_before=1.0):
    """Sum over queries and the group's heads of p [nq][Hq][n] -> ([Hkv][n], bound)."""
    nq, Hq, n = p.shape
    w = p.reshape(nq, Hq // g, g, n).sum((0, 2))
    # each term off by its factor and the lse's own error; a sum of nq * g terms
    tol = (p * (4 * dmax[..., None] + 2.0 ** -19 + 4 * n * U32)).reshape(nq, Hq // g, g, n).sum((0, 2))
    return w, tol + (nq * g + 2) * U32 * (w + n_before) + 1e-30


def assert_within(got, want, tol, what):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    off = (got - want).abs()[~inf]
    bad = ~(off <= tol.expand(want.shape)[~inf])       # NaN is bad too
    if bad.any():
        i = int(torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first: got "
                             f"{got[~inf][i]}, want {want[~inf][i]}, tol {tol.expand(want.shape)[~inf][i]}")


def evicted(w, n, first, recent, top):
    """Kept positions of one row of weights (numpy [n])."""
    keep = first + recent + top
    if n <= keep:
        return list(range(n))
    mid = range(first, n - recent)
    key = lambda j: (-math.inf if math.isnan(w[j]) else -(w[j] + 0.0), j)
    return list(range(first)) + sorted(sorted(mid, key=key)[:top]) + list(range(n - recent, n))
