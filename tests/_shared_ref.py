"""Caches whose sequences share prefixes, and plain forms of the page operators
(test infrastructure beside _kv16_ref)."""
import math

import torch

from tests import _kv16_ref as R


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class SharedCase(R.Case):
    """Groups of `members[i]` sequences that have their first prefix[i] tokens in
    common; lens[b] tokens each.  On the device the whole pages of a prefix stand
    only where the group's first sequence has them: the others' table entries for
    them are -1 (contiguous: their rows are NaN)."""

    def __init__(self, members, prefix, lens, Hkv, first=0, **kw):
        super().__init__(lens, Hkv, **kw)
        self.group, self.prefix = [first], list(prefix)
        for m in members:
            self.group.append(self.group[-1] + m)
        for i, p in enumerate(prefix):
            lead, end = self.group[i], self.group[i + 1]
            if lead == end:
                continue
            most = max(lens[lead:end] + [0])
            # the group's tokens, as its first sequence holds them: all whole shared pages
            whole = p // 32 * 32
            assert lens[lead] >= min(whole, most), "the first sequence holds the prefix"
            for b in range(lead + 1, end):
                n = min(p, lens[b], lens[lead])
                self.k[b][:, :n] = self.k[lead][:, :n]
                self.v[b][:, :n] = self.v[lead][:, :n]

    def cache(self, L, n_tok=None):
        c = super().cache(L, n_tok)
        for i, p in enumerate(self.prefix):
            for b in range(self.group[i] + 1, self.group[i + 1]):
                if self.paged:
                    c.block_table[b, :p // 32] = -1
                else:
                    c.k[b, :, :p // 32 * 32] = math.nan
                    c.v[b, :, :p // 32 * 32] = math.nan
        return c

    def groups(self):
        return i32(self.group), i32(self.prefix)


def compacted(table, n_pages):
    """(new table, moves, live) by the rule, as lists."""
    named = sorted({x for row in table for x in row if x >= 0})
    live = len(named)
    taken = set(named)
    old = [x for x in named if x >= live]
    new = [x for x in range(live) if x not in taken]
    to = dict(zip(old, new))
    return [[to.get(x, x) for x in row] for row in table], [list(m) for m in zip(old, new)], live


def bits(x):
    return x.view(torch.int16 if x.element_size() == 2 else torch.int32)
