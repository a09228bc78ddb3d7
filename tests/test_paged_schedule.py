"""CPU replay of the split of attention over all pages: PagedSplit, PagedWalk and the slots that the join reads.

A unit of P pages stands for `lead` slots without work and a slot a page; the slots of all units are cut into equal ranges.
Every page has to be taken once, in order, and the join has to find the parts of every cut unit where their CTAs put them.
"""

import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = open(os.path.join(ROOT, "sparse_attention_decode_gb300", "csrc", "paged.cu")).read()
LEADS = [int(x) for x in re.search(r"kPagedLead\[2\] = \{(\d+), (\d+)\}", SRC).groups()]


class Split:
    def __init__(self, slots, units, lead, grid):
        self.ctas = min(grid, max((slots - units * lead + 1) // 2, units))
        self.range, self.more = (slots // self.ctas, slots % self.ctas) if self.ctas else (0, 0)

    def start(self, g):
        return g * self.range + min(g, self.more)

    def owner(self, x):
        longer = self.more * (self.range + 1)
        return x // (self.range + 1) if x < longer else self.more + (x - longer) // self.range


def replay(request_pages, units, lead, grid):
    """What each CTA takes, [(slot of its part, unit, first page, pages)], and the parts of each unit as the join reads them."""
    P = [n for n in request_pages if n for _ in range(units)]
    slots = [(u, j - lead) for u, n in enumerate(P) for j in range(n + lead)]
    split = Split(len(slots), len(P), lead, grid)
    taken = []
    for g in range(split.ctas):
        left, (u, j), seg = split.start(g + 1) - split.start(g), slots[split.start(g)], 0
        left, j = left + min(j, 0), max(j, 0)
        while left > 0:
            run = min(left, P[u] - j)
            taken.append((g, 2 * g + (seg > 0), u, j, run))
            left, j, u, seg = left - run - lead, 0, u + 1, seg + 1
    joins, base = {}, 0
    for u, n in enumerate(P):
        first = base + lead  # the slot of its first page
        base += n + lead
        c = split.owner(first)
        parts = split.owner(first + n - 1) - c + 1
        blocks = []  # of the form with a block for each range's end: those that take this unit
        for x in range(min(grid, split.ctas) - 1):
            v, j = slots[split.start(x + 1)]
            if v == u and j > 0 and split.start(x) <= split.start(x + 1) - j:
                blocks.append(x)
        joins[u] = (c, [2 * c + (split.start(c) < first - lead) if i == 0 else 2 * (c + i) for i in range(parts)], blocks)
    return P, taken, joins


def check(request_pages, units, lead, grid):
    P, taken, joins = replay(request_pages, units, lead, grid)
    parts = {}
    for g, slot, u, j, run in taken:
        assert run > 0 and j + run <= P[u]
        parts.setdefault(u, []).append((j, run, g, slot))
    assert sorted(parts) == list(range(len(P)))
    used = {}
    for u, n in enumerate(P):
        assert [p[0] for p in parts[u]] == [sum(p[1] for p in parts[u][:i]) for i in range(len(parts[u]))]
        assert sum(p[1] for p in parts[u]) == n
        c, slots, blocks = joins[u]
        assert parts[u][0][2] == c and len(parts[u]) == len(slots)
        if len(slots) > 1:  # a whole unit goes straight to the output
            assert [p[3] for p in parts[u]] == slots and blocks == [c]
            for s in slots:
                assert used.setdefault(s, u) == u and s < 2 * grid
        else:
            assert blocks == []


@pytest.mark.parametrize("lead", LEADS)
def test_every_page_once_and_every_part_found(lead):
    r = random.Random(5)
    for _ in range(1500):
        request_pages = [r.choice([0, 1, 2, 3, r.randint(0, 60)]) for _ in range(r.choice([1, 2, 5, 40]))]
        check(request_pages, r.choice([1, 2, 4, 8]), lead, r.choice([2, 7, 152]))


@pytest.mark.parametrize("lead", LEADS)
@pytest.mark.parametrize("pages", [[1], [68], [1024], [83, 0, 1, 38, 1, 150, 482, 383], [2] * 300, [1] * 37 + [500], [0, 0]],
                         ids=lambda p: f"{len(p)}x{max(p)}")
def test_batches(pages, lead):
    check(pages, 4, lead, 152)


def test_a_unit_s_lead_keeps_short_units_together_with_fewer_pages():
    """A CTA with six short units takes fewer pages than one with one long unit."""
    lead = LEADS[0]
    P, taken, _ = replay([83, 0, 1, 38, 1, 150, 482, 383], 4, lead, 152)
    count = {}
    for g, _, _, _, run in taken:
        n, pages = count.get(g, (0, 0))
        count[g] = (n + 1, pages + run)
    longest = max(p for n, p in count.values() if n == 1)
    assert all(p + lead * (n - 1) <= longest for n, p in count.values())
