"""The shared prefix's work split and the protocol of its two MMA chains, replayed on the CPU."""

import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = open(os.path.join(ROOT, "sparse_attention_decode_gb300", "csrc", "prefix_attn.cuh")).read()
MIN_PAGES = int(re.search(r"kPrefixMinPages = (\d+)", SRC).group(1))
STAGES = int(re.search(r"kPrefixStages = (\d+)", SRC).group(1))
MAX_GRID = int(re.search(r"kPrefixMaxGrid = (\d+)", SRC).group(1))


class Split:
    """PrefixSplit, with the units that the host makes of the batch's rows."""

    def __init__(self, rows, kv_heads, tokens, own, own_cost, grid):
        self.tile = 128 if rows <= 128 else 256
        self.ways = 256 // self.tile
        self.head_tiles = -(-rows // self.tile)
        self.units = self.head_tiles * kv_heads
        self.pages = -(-tokens // 128)
        self.total = self.pages * self.units
        mine, theirs = self.total * 2 // self.ways, own * own_cost * kv_heads / 8
        most = min(grid, max(1, round(grid * mine / max(1, mine + theirs))))
        self.ctas = min(most, -(-self.total // MIN_PAGES))
        each = min(most // self.units, -(-self.pages // MIN_PAGES))
        if each > 0 and each * self.units * 8 >= self.ctas * 7:
            self.span, self.per = self.pages, each
            self.ctas = self.per * self.units
        else:
            self.span, self.per = self.total, self.ctas

        self.range, self.more = divmod(self.span, self.per)

    def start(self, g):
        k, i = divmod(g, self.per)
        return k * self.span + i * self.range + min(i, self.more)

    def owner(self, x):
        k, y = divmod(x, self.span)
        longer = self.more * (self.range + 1)
        return k * self.per + (y // (self.range + 1) if y < longer else self.more + (y - longer) // self.range)


CASES = [(r, h, n, o, g) for r in (1, 16, 128, 129, 256, 1024, 2500) for h in (1, 4, 8) for n in (1, 128, 129, 4133, 32768)
         for o in (0, 3, 5000) for g in (1, 132, 152)]


@pytest.mark.parametrize("rows,kv_heads,tokens,own,grid", random.Random(4).sample(CASES, 120))
def test_every_page_of_every_unit_has_one_owner(rows, kv_heads, tokens, own, grid):
    s = Split(rows, kv_heads, tokens, own, rows % 5 * 12 or 7, grid)
    assert 1 <= s.ctas <= grid <= MAX_GRID
    assert s.start(0) == 0 and s.start(s.ctas) == s.total
    slots = {}
    for g in range(s.ctas):
        lo, hi = s.start(g), s.start(g + 1)
        assert lo < hi  # no CTA without work
        for x in {lo, (lo + hi) // 2, hi - 1}:
            assert s.owner(x) == g
        for u in range(lo // s.pages, (hi - 1) // s.pages + 1):
            assert slots.setdefault(g + u, (g, u)) == (g, u)  # slot g + u is one CTA's part of one unit
            assert g + u < MAX_GRID + s.units  # what the workspace is sized for
    for u in range(s.units):  # the join's walk over a unit's parts meets all of its pages, in order
        g0, g1 = s.owner(u * s.pages), s.owner((u + 1) * s.pages - 1) + 1
        got = [x for g in range(g0, g1) for x in range(max(s.start(g), u * s.pages), min(s.start(g + 1), (u + 1) * s.pages))]
        assert got == list(range(u * s.pages, (u + 1) * s.pages))


# ---- the protocol: a producer, two MMA chains and two softmax warpgroups as coroutines over the kernel's barriers ----


class Bar:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self, n=1):
        assert self.left >= n, "more arrivals than the phase expects"
        self.left -= n
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, index):
        """Phase `index` complete, told by its parity alone, as the kernel tells it."""
        answer = (self.phase & 1) != (index & 1)
        assert answer == (self.phase > index) and self.phase <= index + 1, "a phase was skipped or reused"
        return answer


def run_chains(runs, ways, rng):
    """`runs`: pages of each of the CTA's units.  Checks data hazards; returns the pages each chain multiplied."""
    kv_full, kv_empty = [Bar(1) for _ in range(STAGES)], [Bar(2 // ways) for _ in range(STAGES)]
    q_full, s_full, o_done = ([Bar(1) for _ in range(2)] for _ in range(3))
    at_run = [0, 0]  # the named barrier of the two softmax warpgroups at the start of a unit
    p_half, p_full = [Bar(2) for _ in range(2)], [Bar(1) for _ in range(2)]  # softmax (as one) and the turn
    ring = [None] * STAGES
    s_tile, queue, log = [None, None], [[], []], [[], []]
    turn = []  # order in which the chains issue their products

    def flush(t, everything):
        # the tensor cores run a chain's work in the order of its issue, some time later
        while queue[t] and (everything or rng.random() < 0.5):
            queue[t].pop(0)()

    def producer():
        it = 0
        for r, n in enumerate(runs):
            for j in range(n):
                for kind in "KV":
                    s = it % STAGES
                    if it >= STAGES:
                        while not kv_empty[s].done(it // STAGES - 1):
                            yield
                    ring[s] = (kind, r, j)
                    kv_full[s].arrive()
                    it += 1
                    yield

    def chain(t):
        it = kp0 = seg = 0
        if t == 0:
            p_half[0].arrive()

        def scores(kp, r, j, to):
            s = (2 * kp) % STAGES

            def work():
                assert ring[s] == ("K", r, j), "scores read another tile"
                s_tile[t] = ("S", r, j)
            queue[t].append(work)
            if to >= 0:
                p_half[to].arrive()
            queue[t].append(s_full[t].arrive)
            queue[t].append(kv_empty[s].arrive)

        for r, n in enumerate(runs):
            j0 = t if ways == 2 else 0
            if j0 < n:  # a chain without a page of the unit takes no part
                while not q_full[t].done(seg):
                    yield
                seg += 1
                while not kv_full[(2 * (kp0 + j0)) % STAGES].done(2 * (kp0 + j0) // STAGES):
                    yield
                scores(kp0 + j0, r, j0, -1)
            for j in range(j0, n, ways):
                kp, more = kp0 + j, j + ways < n
                to = 0 if t == 0 and ways == 2 and j + 1 >= n else 1 - t
                waits = [(kv_full[(2 * kp + 1) % STAGES], (2 * kp + 1) // STAGES)]
                if more:
                    waits.append((kv_full[(2 * (kp + ways)) % STAGES], 2 * (kp + ways) // STAGES))
                for bar, index in waits + [(p_half[t], it), (p_full[t], it)]:
                    while not bar.done(index):
                        yield
                turn.append(t)
                sv = (2 * kp + 1) % STAGES

                def product(r=r, j=j, sv=sv):
                    assert ring[sv] == ("V", r, j) and s_tile[t] == ("P", r, j), "product read other operands"
                    log[t].append((r, j))
                queue[t].append(product)
                queue[t].append(o_done[t].arrive)
                queue[t].append(kv_empty[sv].arrive)
                if more:
                    scores(kp + ways, r, j + ways, to)
                else:
                    p_half[to].arrive()
                it += 1
                yield
            kp0 += n

    def softmax(t):
        it = 0
        for r, n in enumerate(runs):
            first = t if ways == 2 else 0
            at_run[t] += 1
            while at_run[1 - t] <= r:
                yield
            if first < n:
                q_full[t].arrive()
            for j in range(first, n, ways):
                while not s_full[t].done(it):
                    yield
                assert s_tile[t] == ("S", r, j)
                s_tile[t] = ("P", r, j)
                p_half[t].arrive()
                yield
                p_full[t].arrive()
                it += 1
            if first < n:
                while not o_done[t].done(it - 1):  # the unit's part is read before its tile and its sums are reused
                    yield
            yield

    tasks = [producer(), chain(0), chain(1), softmax(0), softmax(1)]
    idle = 0
    while tasks:
        task = rng.choice(tasks)
        try:
            next(task)
        except StopIteration:
            tasks.remove(task)
            idle = 0
        for t in range(2):
            flush(t, False)
        idle += 1
        assert idle < 20000, "the chains wait for each other"
    for t in range(2):
        flush(t, True)
    return log, turn


@pytest.mark.parametrize("ways", [1, 2])
@pytest.mark.parametrize("seed", range(300))
def test_the_chains_take_turns_and_meet_their_operands(ways, seed):
    rng = random.Random(seed)
    runs = [rng.choice((1, 1, 2, 3, 4, 7)) for _ in range(rng.randint(1, 5))]
    log, turn = run_chains(runs, ways, rng)
    want = [[(r, j) for r, n in enumerate(runs) for j in range(t if ways == 2 else 0, n, ways)] for t in range(2)]
    assert log == want
    if ways == 1:
        assert turn == [0, 1] * (len(turn) // 2)  # strictly in turns
    else:
        assert turn == [t for n in runs for j in range(n) for t in [j & 1]]
