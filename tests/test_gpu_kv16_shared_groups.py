"""Many groups that really share, on the GPU, against the plain 64-bit form: pairs
up to the most sequences, groups of unequal size and prefix, several chunks each,
and groups whose first sequence is over."""
import random

import pytest
import torch

from tests import _kv16_ref as R
from tests._shared_ref import SharedCase, i32
from tests.test_gpu_kv16_shared import L, attend, decode  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def some(L, case, Hq, every, window=0, sink=0):
    """The decode, both ways, looked at in some sequences."""
    cache = case.cache(L)
    q = case.normal(case.B, Hq)
    outs = decode(L, case, cache, Hq, window, sink, q=q, check=False)
    assert L.device_status() == 0
    for b in sorted({*range(0, case.B, every), case.B - 1}):
        o, _, _, tol, _, _ = R.attend(case, b, q[b:b + 1], window, sink)
        for out in outs:
            R.assert_within(out[b:b + 1], o, tol, f"out of sequence {b}")


@pytest.mark.parametrize("window,sink", [(0, 0), (40, 33)])
def test_the_most_sequences_in_pairs(L, window, sink):
    """2048 pairs, and as many groups of none between them."""
    members = [2, 0] * 2048
    prefix = [64 if i % 4 else 32 for i in range(4096)]
    lens = [65 + b % 40 for b in range(4096)]
    some(L, SharedCase(members, prefix, lens, 1), 1, 61, window, sink)


@pytest.mark.parametrize("Hq,Hkv,dtype", [(8, 2, BF), (16, 1, FP)])
@pytest.mark.parametrize("window,sink", [(0, 0), (150, 4)])
def test_groups_of_unequal_size(L, Hq, Hkv, dtype, window, sink):
    rng = random.Random(5)
    members = [rng.choice((1, 2, 3, 5, 9)) for _ in range(120)]
    prefix = [rng.choice((32, 40, 64, 130, 300, 511)) for _ in members]
    lens = []
    for m, p in zip(members, prefix):
        lens += [p + rng.randint(1, 120) for _ in range(m)]
    some(L, SharedCase(members, prefix, lens, Hkv, dtype=dtype, seed=1), Hq, 7, window, sink)


def test_groups_of_several_chunks(L):
    """Nine groups of more rows than two query tiles hold, worked in blocks of keys or not."""
    members, prefix = [70, 65, 64, 130, 90, 66, 200, 80, 71], [2100, 64, 700, 3000, 128, 1500, 96, 4000, 33]
    lens = []
    for m, p in zip(members, prefix):
        lens += [p + 1 + (13 * i) % 50 for i in range(m)]
    some(L, SharedCase(members, prefix, lens, 1, dtype=FP, seed=2), 4, 31)


@pytest.mark.parametrize("Hq,Hkv,dtype,window,sink", [(8, 2, BF, 0, 0), (6, 2, FP, 90, 40)])
def test_attention_of_many_groups(L, Hq, Hkv, dtype, window, sink):
    rng = random.Random(7)
    members = [rng.choice((0, 1, 2, 3, 6)) for _ in range(60)]
    prefix = [rng.choice((32, 64, 100, 260)) for _ in members]
    lens, news = [], []
    for m, p in zip(members, prefix):
        for _ in range(m):
            news.append(rng.choice((1, 1, 2, 7, 40)))
            lens.append(p + news[-1] + rng.randint(0, 60))
    case = SharedCase(members, prefix, lens, Hkv, dtype=dtype, seed=3)
    attend(L, case, case.cache(L), news, Hq, window, sink)


@pytest.mark.parametrize("paged", [True, False])
def test_a_first_sequence_that_is_over(L, paged):
    """Its tokens stay where they are and its length is 0: the others read them."""
    lens = [300, 310, 350, 70, 90, 100]
    case = SharedCase([3, 3], [288, 64], lens, 2, paged=paged, seed=4)
    cache = case.cache(L)
    cache.n_tok.copy_(i32([0, 310, 350, 0, 90, 100]))
    q = case.normal(6, 8)
    outs = list(decode(L, case, cache, 8, q=q, check=False))
    group, prefix = case.groups()
    got = torch.full((4, 8, 128), 7.0, dtype=BF, device="cuda")
    ws = L.alloc_workspace(L.kv16_shared_attention_workspace_bytes(cache, 8, 2, 4, cache.capacity))
    rows = [1, 2, 4, 5]
    L.kv16_shared_attention(cache, q[rows].cuda(), i32([0, 0, 1, 2, 2, 3, 4]), group, prefix, R.SCALE, cache.capacity, got, ws)
    assert L.device_status() == 0
    for b in (0, 3):
        assert all((out[b] == 0).all() for out in outs)
    for i, b in enumerate(rows):
        o, _, _, tol, _, _ = R.attend(case, b, q[b:b + 1])
        for out in (*(x[b:b + 1] for x in outs), got[i:i + 1]):
            R.assert_within(out, o, tol, f"sequence {b}")
