"""The shared prefix's work split where some SMs are kept free for the own pages' CTAs, replayed on the CPU."""

import random

import pytest

from test_prefix_schedule import CASES, MAX_GRID, MIN_PAGES, Split


class SpareSplit(Split):
    """PrefixSplit with `spare` CTAs of the grid that take no part."""

    def __init__(self, rows, kv_heads, tokens, own, own_cost, grid, spare):
        super().__init__(rows, kv_heads, tokens, own, own_cost, grid)
        mine, theirs = self.total * 2 // self.ways, own * own_cost * kv_heads / 8
        most = min(grid - spare, max(1, round(grid * mine / max(1, mine + theirs))))
        self.ctas = min(most, -(-self.total // MIN_PAGES))
        each = min(most // self.units, -(-self.pages // MIN_PAGES))
        if each > 0 and each * self.units * 8 >= self.ctas * 7:
            self.span, self.per = self.pages, each
            self.ctas = self.per * self.units
        else:
            self.span, self.per = self.total, self.ctas
        self.range, self.more = divmod(self.span, self.per)


def check(s, grid, spare):
    assert 1 <= s.ctas <= grid - spare
    assert s.start(0) == 0 and s.start(s.ctas) == s.total
    for g in range(s.ctas):
        lo, hi = s.start(g), s.start(g + 1)
        assert lo < hi
        assert all(s.owner(x) == g for x in {lo, (lo + hi) // 2, hi - 1})
        assert all(g + u < MAX_GRID + s.units for u in range(lo // s.pages, (hi - 1) // s.pages + 1))
    for u in range(s.units):
        g0, g1 = s.owner(u * s.pages), s.owner((u + 1) * s.pages - 1) + 1
        got = [x for g in range(g0, g1) for x in range(max(s.start(g), u * s.pages), min(s.start(g + 1), (u + 1) * s.pages))]
        assert got == list(range(u * s.pages, (u + 1) * s.pages))


@pytest.mark.parametrize("rows,kv_heads,tokens,own,grid", random.Random(5).sample([c for c in CASES if c[4] > 1], 120))
def test_every_page_has_one_owner_beside_spare_sms(rows, kv_heads, tokens, own, grid):
    for spare in {1, kv_heads, grid // 8}:  # the host keeps at most an eighth of the SMs free
        if spare <= grid // 8:
            check(SpareSplit(rows, kv_heads, tokens, own, rows % 5 * 12 or 7, grid, spare), grid, spare)


def test_without_spare_sms_it_is_the_split_of_the_other_replay():
    for rows, kv_heads, tokens, own, grid in CASES[::7]:
        a, b = Split(rows, kv_heads, tokens, own, 12, grid), SpareSplit(rows, kv_heads, tokens, own, 12, grid, 0)
        assert vars(a) == vars(b)
