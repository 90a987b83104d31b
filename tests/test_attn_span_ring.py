"""The ring of key tiles of attention with sinks (csrc/attn_span.cu) as a model: the
loading warp, a warp a query tile that issues its products and skips the key
tiles that its rows do not see, and copies that land in any order.  A barrier's wait
tells a phase from the one before it, no more; so a warp that passed a place unseen
may take an older copy still on its way for the one it waits for, unless it knows
that that one was released.  (The kernel cannot be made to show it: its copies hardly
ever land so late.)"""
import random

import pytest

BQ, BKV = 128, 64


class Barrier:
    def __init__(self, need):
        self.need, self.left, self.phase = need, need, 0

    def arrive(self, n=1):
        self.left -= n
        assert self.left >= 0, "a barrier has more arrivals than its phase takes"
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.need

    def done(self, parity):
        return self.phase & 1 != parity & 1


def key_tiles(left, right, sinks, r0, r1, n):
    lo, hi = max(0, r0 - left), min(n, r1 + right + 1)
    first = lo // BKV
    s = min((min(sinks, lo) + BKV - 1) // BKV, first)
    return s, first, (hi + BKV - 1) // BKV


class Stale(Exception):
    pass


class Model:
    def __init__(self, rng, nt, ring, items, limits, protocol):
        self.rng, self.nt, self.R, self.items, self.limits, self.protocol = rng, nt, ring, items, limits, protocol
        self.kv = [Barrier(1) for _ in range(ring)]
        self.kve = [Barrier(nt) for _ in range(ring)]
        self.q, self.qe = [Barrier(1) for _ in range(nt)], [Barrier(1) for _ in range(nt)]
        self.holds = [None] * ring
        self.flight = []                                  # copies and products under way: what they do at their end

    def tiles(self, n, q0):
        qb = self.nt * BQ
        whole = key_tiles(*self.limits, q0, min(q0 + qb, n) - 1, n)
        each = []
        for w in range(self.nt):
            r0 = q0 + w * BQ
            each.append(key_tiles(*self.limits, r0, min(r0 + BQ, n) - 1, n) if r0 < n else (0, 0, 0))
        return whole, each

    @staticmethod
    def listed(k):
        return list(range(k[0])) + list(range(k[1], k[2]))

    def land(self, place, fill):
        self.holds[place] = fill
        self.kv[place].arrive()

    def loader(self):
        fill = 0
        loads = [0] * self.nt
        for n, q0 in self.items:
            whole, each = self.tiles(n, q0)
            seen = [self.listed(k) for k in each]
            for t in self.listed(whole):
                for w in range(self.nt):
                    if seen[w] and seen[w][0] == t:
                        while not self.qe[w].done(loads[w] ^ 1):
                            yield
                        loads[w] += 1
                        self.flight.append(self.q[w].arrive)
                place, phase = fill % self.R, fill // self.R
                while not self.kve[place].done(phase ^ 1):
                    yield
                self.flight.append(lambda p=place, f=fill: self.land(p, f))
                idle = sum(t not in s for s in seen)
                assert idle < self.nt, "a tile that nothing sees is not listed"
                if idle:
                    self.kve[place].arrive(idle)
                fill += 1

    def issuer(self, w):
        base, had = 0, 0
        for n, q0 in self.items:
            whole, each = self.tiles(n, q0)
            order, mine = self.listed(whole), self.listed(each[w])
            assert all(t in order for t in mine)
            if mine:
                while not self.q[w].done(had):
                    yield
            at, places, released = 0, [], 0
            for i, t in enumerate(mine):
                nxt = order.index(t)
                # the products of the tile before come first where this one's place waits for them
                while released < i and (released < i - 1 or nxt - at + 1 >= self.R):
                    self.flight.append(self.kve[places[released]].arrive)
                    released += 1
                fill = base + nxt
                place, phase = fill % self.R, fill // self.R
                before = {"released": self.kve, "landed before": self.kv}.get(self.protocol)
                while before and not before[place].done(phase ^ 1):
                    yield
                while not self.kv[place].done(phase):
                    yield
                if self.holds[place] != fill:
                    raise Stale
                places.append(place)
                at = nxt + 1
                if i == len(mine) - 1:
                    self.flight.append(self.qe[w].arrive)
                yield
            while released < len(mine):
                self.flight.append(self.kve[places[released]].arrive)
                released += 1
            base += len(order)
            had += bool(mine)

    def run(self):
        """True: every item done.  False: nothing can go on."""
        agents = [self.loader()] + [self.issuer(w) for w in range(self.nt)]
        idle = 0
        while agents:
            # copies land late: agents run while they can
            if self.flight and (idle > 3 * len(agents) or self.rng.random() < 0.02):
                self.flight.pop(self.rng.randrange(len(self.flight)))()
                idle = 0
                continue
            if idle > 100 * len(agents):
                return False
            a = self.rng.choice(agents)
            before = (len(self.flight), [b.phase for b in self.kv + self.kve])
            try:
                next(a)
                idle = idle + 1 if before == (len(self.flight), [b.phase for b in self.kv + self.kve]) else 0
            except StopIteration:
                agents.remove(a)
                idle = 0
        return True


def cases(seed, nt, ring):
    rng = random.Random(seed)
    limits = (rng.choice([0, 5, 64, 200, 500, 10 ** 6]), rng.choice([0, 10, 100, 300, 10 ** 6]), rng.choice([0, 0, 3, 70, 400]))
    qb = nt * BQ
    items = []
    for _ in range(rng.randint(2, 5)):
        n = rng.choice([1, 64, 100, 129, 300, 500, 700, 1200])
        items.append((n, rng.randrange((n + qb - 1) // qb) * qb))
    return rng, items, limits


@pytest.mark.parametrize("nt,ring", [(3, 7), (2, 4), (2, 3)])
def test_no_place_is_read_before_its_copy_landed(nt, ring):
    for seed in range(500):
        rng, items, limits = cases(seed, nt, ring)
        assert Model(rng, nt, ring, items, limits, "released").run(), seed


@pytest.mark.parametrize("nt,ring", [(3, 7), (2, 4), (2, 3)])
def test_the_model_tells_protocols_apart(nt, ring):
    """Without the wait for the release copies are taken too early; a wait for the copy
    before instead stalls once the one behind it has landed."""
    stale = stalls = 0
    for seed in range(500):
        rng, items, limits = cases(seed, nt, ring)
        try:
            Model(rng, nt, ring, items, limits, "plain").run()
        except Stale:
            stale += 1
        rng, items, limits = cases(seed, nt, ring)
        try:
            stalls += not Model(rng, nt, ring, items, limits, "landed before").run()
        except Stale:
            pass
    assert stale > 0 and stalls > 0, (stale, stalls)
