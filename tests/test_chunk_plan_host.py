"""The chunk kernel's plan, restated and walked on the CPU: over ragged batches, windows,
row tilings and CTA counts every unit's key tiles are covered once, cut units leave at
most two pieces a CTA in the slots and the number that the merge expects, and ranges
carry equal weight."""
import random

import pytest


def ceil_div(a, b):
    return -(-a // b)


class Plan:
    def __init__(self, d, n, G, Hkv, NT, grid, causal=True, window=-1, cost=640, min_span=256, total=None):
        self.d, self.n, self.NT, self.Hkv, self.grid = d, n, NT, Hkv, grid
        self.causal, self.window, self.cost = causal, window, cost
        N = sum(d)
        self.tt = min(128 // G, max(N, 1)) if G <= 128 else 1
        self.hc = 1 if G <= 128 else ceil_div(G, 128)
        self.ride = Hkv > 1 and grid % Hkv == 0
        self.s = 1 if self.hc > 1 else NT * self.tt
        self.parts = ceil_div(self.hc, NT) if self.hc > 1 else 1
        self.reps = self.parts * (1 if self.ride else Hkv)
        self.rows = [self.row(b) for b in range(len(d))]
        self.weights = [self.reps * self.prefix(r, r[2]) if r[3] < r[2] else 0 for r in self.rows]
        self.total = sum(self.weights)
        self.nranges = grid // Hkv if self.ride else grid
        self.span = max(min_span, ceil_div(self.total, self.nranges))

    def row(self, b):
        n, d = self.n[b], self.d[b]
        steps = ceil_div(d, self.s)
        v0 = steps if n == 0 else ((d - n) // self.s if self.causal and d > n else 0)
        return n, d, steps, v0

    def weight(self, r, v):
        base = r[0] - r[1]
        hi = base + (v + 1) * self.s if self.causal else r[0]
        lo = 0 if self.window < 0 else max(0, base - self.window + v * self.s)
        return self.cost + 128 + hi - lo

    def prefix(self, r, v):
        s, base, v0 = self.s, r[0] - r[1], r[3]
        total = lambda a, e: (e - a) * (a + e - 1) // 2
        m = v - v0
        w = m * (self.cost + 128)
        w += m * (base + s) + s * total(v0, v) if self.causal else m * r[0]
        if self.window >= 0:
            z = base - self.window
            first = max(v0, 0 if z >= 0 else (-z) // s + 1)
            if first < v:
                w -= (v - first) * z + s * total(first, v)
        return w

    def tiles(self, r, v):
        n, d = r[0], r[1]
        t0, t1 = v * self.s, min(d, (v + 1) * self.s) - 1
        lo = 0 if self.window < 0 else max(0, n - d + t0 - self.window)
        hi = n - d + t1 + 1 if self.causal else n
        return lo // 128, ceil_div(hi, 128) - lo // 128

    def tile_at(self, x, tiles):
        x -= self.cost
        return 0 if x <= 0 else min(tiles, x >> 7)

    def walk(self, cta):
        """(unit, first tile, tiles, slot, pieces of the unit that this one begins)"""
        rng = cta // self.Hkv if self.ride else cta
        pos = self.span * rng
        end = min(self.total, pos + self.span)
        if pos >= end:
            return
        b, row0 = 0, 0
        while pos >= row0 + self.weights[b]:
            row0 += self.weights[b]
            b += 1
        r = self.rows[b]
        per_rep = self.prefix(r, r[2])
        rep = (pos - row0) // per_rep
        off = pos - row0 - rep * per_rep
        lo, hi = r[3], r[2] - 1
        while lo < hi:
            mid = (lo + hi + 1) // 2
            if self.prefix(r, mid) <= off:
                lo = mid
            else:
                hi = mid - 1
        v, start = lo, row0 + rep * per_rep + self.prefix(r, lo)
        while start < end:
            if v >= r[2]:
                v = r[3]
                rep += 1
                if v >= r[2] or rep >= self.reps:
                    b += 1
                    assert b < len(self.d)
                    r, rep = self.rows[b], 0
                    v = r[3]
                continue
            w = self.weight(r, v)
            tile0, tiles = self.tiles(r, v)
            assert tiles >= 1
            a = self.tile_at(pos - start, tiles)
            e = tiles if end >= start + w else self.tile_at(end - start, tiles)
            at, step = start, v
            start += w
            v += 1
            if a >= e:
                continue
            slot, pieces = -1, 0
            if a > 0:
                slot = 2 * cta
            elif e < tiles:
                slot = 2 * cta + 1
                last = min(ceil_div(at + self.cost + 128 * tiles, self.span), ceil_div(at + w, self.span))
                pieces = last - rng
            g = cta % self.Hkv if self.ride else rep // self.parts
            yield (b, g, rep % self.parts, step), tile0 + a, e - a, slot, pieces


def check(plan):
    covered, cut, slots = {}, {}, {}
    load = []
    for cta in range(plan.grid):
        mine = 0
        for unit, tile0, tiles, slot, pieces in plan.walk(cta):
            mine += tiles
            covered.setdefault(unit, []).append((tile0, tiles, slot, cta))
            if slot >= 0:
                assert slot not in slots, "a slot taken twice"
                slots[slot] = unit
            if pieces:
                cut[unit] = (cta, pieces)
        load.append(mine)
    want = set()
    for b, r in enumerate(plan.rows):
        for v in range(r[3], r[2]):
            for g in range(plan.Hkv):
                for part in range(plan.parts):
                    want.add((b, g, part, v))
        for v in range(0, r[3]):                       # what is left out sees nothing
            last = min(r[1], (v + 1) * plan.s) - 1
            assert r[0] == 0 or (plan.causal and r[0] - r[1] + last + 1 <= 0)
    assert set(covered) == want
    step = plan.Hkv if plan.ride else 1
    for unit, got in covered.items():
        got.sort()
        t0, t = plan.tiles(plan.rows[unit[0]], unit[3])
        at = t0
        for tile0, tiles, _, _ in got:
            assert tile0 == at
            at += tiles
        assert at == t0 + t
        if len(got) == 1:
            assert got[0][2] == -1 and unit not in cut
        else:
            cta, pieces = cut[unit]
            assert pieces == len(got)
            for k, (_, _, slot, c) in enumerate(got):
                assert c == cta + k * step and slot == (2 * cta + 1 if k == 0 else 2 * c)


@pytest.mark.parametrize("seed", range(60))
def test_ragged_batches(seed):
    r = random.Random(seed)
    B = r.choice([1, 1, 2, 5, 17, 40])
    long = r.choice([1, 3, 40, 300, 2500])
    d = [r.choice([0, 1, 1, r.randint(0, long)]) for _ in range(B)]
    n = [r.choice([0, x, x + r.randint(0, 5000), r.randint(0, 300), x + r.randint(0, 130)]) for x in d]
    G, Hkv = r.choice([(5, 8), (4, 8), (1, 16), (4, 2), (7, 4), (32, 1), (7, 1), (160, 1), (300, 2), (128, 1)])
    for NT in (1, 2):
        for grid in (152, r.choice([1, 2, 3, 7, 16])):
            for window in (-1, r.choice([0, 1, 100, 1023, 100000])):
                check(Plan(d, n, G, Hkv, NT, grid, r.random() < 0.7, window, r.choice([128, 640])))


@pytest.mark.parametrize("seed", range(12))
def test_ragged_batches_on_pairs(seed):
    """Half as many workers, two row tiles a unit."""
    r = random.Random(1000 + seed)
    d = [r.choice([1, 7, r.randint(0, 1200)]) for _ in range(r.choice([1, 4, 23]))]
    n = [x + r.choice([0, 5, r.randint(0, 6000)]) for x in d]
    for G, Hkv in ((1, 16), (8, 1), (2, 4)):
        for workers in (76, 1, 5):
            check(Plan(d, n, G, Hkv, 2, workers, r.random() < 0.7, r.choice([-1, 300]), 640))


def test_ranges_are_even():
    p = Plan([4096], [36864], 5, 8, 2, 152)
    load = [sum(t for _, _, t, _, _ in p.walk(c)) for c in range(152)]
    assert max(load) - min(load) <= 0.03 * max(load) + 8


@pytest.mark.parametrize("window", [-1, 1000])
def test_sizes_at_the_ends_of_the_range(window):
    check(Plan([1, 70000], [2 ** 30, 2 ** 21], 1, 2, 2, 152, window=window))
    check(Plan([1] * 4000, [1] * 4000, 5, 8, 1, 152, window=window))
    check(Plan([1], [2 ** 30], 8, 1, 1, 152, window=2 ** 31 - 1))
