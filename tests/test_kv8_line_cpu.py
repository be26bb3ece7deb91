"""The line of the tile kernel over looked-up segments, its index arithmetic in
plain Python (csrc/kv8_tiles.cuh): how the items of all segments are cut into one
range per CTA, where parts are left and which CTA joins them.  The line is
counted by slots, which bisect the segments' first rows, and walked by segments:
both name the same items only while those rows rise, so that the kernel leaves
where they fall."""

import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_kv_cache_02_gb300", "csrc")


def _constant(file, name):
    with open(os.path.join(CSRC, file)) as f:
        return int(re.search(rf"constexpr int {name} = (\d+);", f.read()).group(1))


ROWS, TILE_CTAS = _constant("kv8_internal.cuh", "kTileRows"), _constant("kv8_internal.cuh", "kMaxTileCtas")
ROWS_MAX, OVER = _constant("kv8_internal.cuh", "kRowsMax"), _constant("kv8_tiles.cuh", "kOver")
SLOTS = 2 * TILE_CTAS  # places for partial results


class Line:
    """Segments with rows start[s] .. start[s + 1] - 1 and units[s] units each, for
    `heads` KV heads of `group` rows; `least` line positions per CTA."""

    def __init__(self, start, units, group, heads, least, rows=None, sms=152):
        self.start, self.units, self.group, self.H, self.segs = start, units, group, heads, len(units)
        self.rows = start[-1] if rows is None else rows
        self.slots = self.row(self.segs) * group // ROWS + self.segs
        pairs = [self.pair_of_slot(i) for i in range(self.slots)]
        self.pairs = [p for p in pairs if self.cost(p)]
        self.total = sum(self.cost(p) for p in self.pairs) * heads
        self.ctas = min(sms, -(-self.total // least))

    def row(self, s):
        return min(max(self.start[s], 0), self.rows)

    def base(self, s):
        return self.row(s) * self.group // ROWS + s

    def pair_of_slot(self, slot):
        lo, hi = 0, self.segs - 1
        while lo < hi:
            mid = (lo + hi + 1) >> 1
            lo, hi = (mid, hi) if self.base(mid) <= slot else (lo, mid - 1)
        return lo, slot - self.base(lo)

    def cost(self, pair):
        """Line positions of an item of the (segment, row tile), 0: no such."""
        s, rt = pair
        a, b = self.start[s], self.start[s + 1]
        n = (b - a) * self.group if 0 <= a <= b <= self.rows else 0
        return self.units[s] + OVER if n > ROWS_MAX and self.units[s] > 0 and 0 <= rt and rt * ROWS < n else 0

    def owner(self, position):
        return ((position + 1) * self.ctas - 1) // self.total

    def parts(self, cta):
        """(item, first unit, behind the last, slot or -1, first slot, first CTA, cuts) of a CTA's range."""
        lo, hi = cta * self.total // self.ctas, (cta + 1) * self.total // self.ctas
        at, out = 0, []
        for pair in self.pairs:
            if lo < at + self.cost(pair) * self.H:
                break
            at += self.cost(pair) * self.H
        cost = self.cost(pair)
        h = (lo - at) // cost
        begin = at + h * cost
        while True:
            first = begin + OVER
            u0, u1 = max(lo - first, 0), min(cost - OVER, hi - first)
            if u1 <= u0:
                return out
            slot = join = c0 = cuts = -1
            if (u0, u1) != (0, cost - OVER):
                c0 = self.owner(first)
                cuts = self.owner(begin + cost - 1) - c0
                slot = 2 * cta + (lo < begin)
                join = 2 * c0 + (c0 * self.total // self.ctas < begin)
            out.append(((*pair, h), u0, u1, slot, join, c0, cuts))
            begin += cost
            if begin + OVER >= hi:
                return out
            h += 1
            if h == self.H:
                h, pair = 0, (pair[0], pair[1] + 1)
                while not self.cost(pair):
                    pair = (pair[0] + 1, 0)
                    if pair[0] >= self.segs:
                        return out
                cost = self.cost(pair)

    def faults(self):
        """What goes wrong when all CTAs run: an empty set where nothing does."""
        if self.total == 0:
            return set()
        wrong, seen, place, counters, later = set(), {}, {}, {}, set()
        for cta in range(self.ctas):
            for item, u0, u1, slot, join, c0, cuts in self.parts(cta):
                seen.setdefault(item, []).append((u0, u1))
                if slot < 0:
                    continue
                if not 0 <= slot < SLOTS or c0 + cuts >= TILE_CTAS or not 0 <= join < SLOTS:
                    wrong.add("range")
                if slot in place:
                    wrong.add("slot")
                place[slot] = item
                key = (c0, cuts)
                counters.setdefault(c0, {}).setdefault((item, key), 0)
                counters[c0][(item, key)] += 1
                if cuts >= 4 and u0 == 0:
                    later.add((cta, item))
        for c0, users in counters.items():  # one item per counter, which as many CTAs count as it has parts
            if len(users) != 1 or any(n != cuts + 1 for (_, (_, cuts)), n in users.items()):
                wrong.add("counter")
        for item, parts in seen.items():  # its units, each once
            parts.sort()
            if parts[0][0] != 0 or parts[-1][1] != self.cost(item[:2]) - OVER \
                    or any(x[1] != y[0] for x, y in zip(parts, parts[1:])):
                wrong.add("units")
        if len(seen) != len(self.pairs) * self.H:
            wrong.add("items")
        if len(later) > TILE_CTAS // 4 or len({c for c, _ in later}) != len(later):
            wrong.add("joins")
        return wrong

    def falls(self):
        return any(y < x for x, y in zip(self.start, self.start[1:]))


def _random_line(rng, sms):
    segs = int(rng.integers(1, 40))
    most = int(rng.choice([3, 80, 700]))
    n = rng.integers(0, most, segs) * (rng.random(segs) < 0.8)
    start = [int(x) for x in np.cumsum([int(rng.integers(0, 5)), *n])]
    units = [int(x) for x in rng.integers(0, int(rng.choice([3, 40, 400])), segs)]
    return Line(start, units, int(rng.choice([1, 2, 3, 4, 7, 16, 300])), int(rng.choice([1, 2, 4, 8])),
                int(rng.choice([2, 4])), rows=start[-1] + int(rng.integers(-2, 3)) * (rng.random() < 0.2), sms=sms)


@pytest.mark.parametrize("seed", range(150))
def test_rising_starts(seed):
    """Every unit of every item once, each part at a place of its own, as many
    counts as an item has parts, and no more late joins than the join kernel has CTAs for."""
    rng = np.random.default_rng(seed)
    line = _random_line(rng, int(rng.choice([1, 2, 7, 148, 152, 160])))
    assert line.faults() == set()


def test_rows_of_a_bad_range_are_no_items():
    """A start far behind the rows (its rows times the group pass 32 bits) does not
    move the other segments' slots."""
    line = Line([0, 300, 900, 2 ** 31 - 1, 2 ** 31 - 1], [9, 30, 50, 7], 512, 2, 4, rows=900)
    assert line.faults() == set() and {p[0] for p in line.pairs} == {0, 1} and line.base(3) < 2 ** 31


FALLS = [  # (starts, units, group, KV heads, least positions of a CTA, what goes wrong)
    ([0, 150, 50, 400], [4, 16, 28], 4, 8, 4, "items"),
    ([0, 383, 88, 449, 520, 110, 167, 533], [51, 48, 63, 4, 61, 6, 40], 4, 8, 4, "counter"),
    ([0, 218, 543, 80, 449, 119, 568, 121, 270], [200, 2, 2, 200, 200, 1, 200, 200], 4, 1, 2, "range"),
]


@pytest.mark.parametrize("start,units,group,heads,least,what", FALLS)
def test_falling_starts_are_no_line(start, units, group, heads, least, what):
    """Why the kernel leaves where starts fall: items under the wrong place,
    counters that stay set, places behind the last."""
    line = Line(start, units, group, heads, least, rows=max(start))
    assert line.falls() and what in line.faults()


def test_the_kernels_leave_where_starts_fall():
    """The lookup notes a fall of either array, the tile kernel leaves on it."""
    with open(os.path.join(CSRC, "kv8_shared.cu")) as f:
        lookup = f.read()
    with open(os.path.join(CSRC, "kv8_tiles.cuh")) as f:
        tiles = f.read()
    assert re.search(r"group_start\[i \+ 1\] < a\.group_start\[i\]", lookup)
    assert re.search(r"row_start\[s \+ 1\] < a\.row_start\[s\]", lookup)
    assert "a.falls" in lookup and "a.falls" in tiles
