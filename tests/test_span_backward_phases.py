"""The barriers of the span backward's persistent kernels, on the CPU: a model of their roles (who waits for and
arrives at what, in which order) under schedules that let one role lag behind. A wait tests a phase's parity only,
like the kernels', so a role that is two phases behind never wakes; the schedule then ends with nothing left to
run. How many barriers are used in turn is read from the kernels' source.
"""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "host_memory_streamed_stream_gb300",
                   "csrc")


def _turns(name, path="attention_span_bwd.cu"):
    """The source's `constexpr int name = n;` (1 where there is none: one barrier)."""
    with open(os.path.join(SRC, path)) as f:
        m = re.search(rf"constexpr int {name} = (\d+);", f.read())
    return int(m.group(1)) if m else 1


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != parity


class Turns:
    """Barriers used in turn: phase n is phase n // turns of barrier n % turns."""

    def __init__(self, turns, count):
        self.bars = [Barrier(count) for _ in range(turns)]

    def wait(self, n):
        return self.bars[n % len(self.bars)], n // len(self.bars) & 1

    def arrive(self, n):
        self.bars[n % len(self.bars)].arrive()


class Block:
    """One block: its roles are generators that yield (barrier, parity) to wait or None for a step. `walks` are the
    tiles of its items. Copies arrive in any order, products in the order of their commits."""

    ELEM = 2  # elementwise warps

    def __init__(self, walks, acc_turns):
        n = self.ELEM
        self.items = list(walks) + [-1]
        self.ring1 = [Turns(1, 1) for _ in range(3)], [Turns(1, 1) for _ in range(3)]  # Q of dK/dV, K of dQ
        self.ring2 = [Turns(1, 1) for _ in range(2)], [Turns(1, 1) for _ in range(2)]  # dO of dK/dV, V of dQ
        self.item_full, self.item_empty, self.slot = Turns(2, 1), Turns(2, n + 3), [None, None]
        self.own_full, self.own_empty = Turns(1, 1), Turns(1, 1)
        self.dp_free, self.acc_full, self.acc_empty = Turns(1, n), Turns(1, 1), Turns(acc_turns, n)
        self.copies, self.products = [], []

    def full(self, ring, g):
        bars = ring[0]
        return bars[g % len(bars)].wait(g // len(bars))

    def load(self, ring, g):
        full, empty = ring
        k = len(full)
        if g >= k:
            yield empty[g % k].wait(g // k - 1)
        self.copies.append(lambda: full[g % k].arrive(g // k))

    def free(self, ring, g):
        return lambda: ring[1][g % len(ring[1])].arrive(g // len(ring[1]))

    def put(self, m):
        if m >= 2:
            yield self.item_empty.wait(m - 2)
        self.slot[m & 1] = self.items[m]
        self.item_full.arrive(m)

    def get(self, m):
        yield self.item_full.wait(m)
        it = self.slot[m & 1]
        yield None
        self.item_empty.arrive(m)
        return it

    def items_and_ring1(self):
        yield from self.put(0)
        g = 0
        for m, tiles in enumerate(self.items[:-1]):
            if tiles == 0:
                yield from self.put(m + 1)
            for j in range(tiles):
                if j == max(tiles - 2, 0):
                    yield from self.put(m + 1)
                yield from self.load(self.ring1, g)
                g += 1

    def ring2_loads(self):
        m = g = 0
        while (tiles := (yield from self.get(m))) >= 0:
            for _ in range(tiles):
                yield from self.load(self.ring2, g)
                g += 1
            m += 1

    def own_and_stores(self):
        m = n = g = stored = 0

        def store(i, last):
            yield self.acc_empty.wait(i)
            yield None
            for ring in self.held:
                self.free(ring, last)()

        while (tiles := (yield from self.get(m))) >= 0:
            last = g - 1
            if tiles:
                if n:
                    yield self.own_empty.wait(n - 1)
                self.copies.append(lambda n=n: self.own_full.arrive(n))
            if stored < n:
                yield from store(stored, last)
                stored += 1
            if tiles:
                g, n = g + tiles, n + 1
            m += 1
        if stored < n:
            yield from store(stored, g - 1)

    def elementwise(self):
        m = n = g = 0
        tiles = yield from self.get(0)
        while tiles >= 0:
            for _ in range(tiles):
                yield from self.tile(g)
                g += 1
            m += 1
            following = yield from self.get(m)
            if tiles:
                yield self.acc_full.wait(n)
                yield None
                self.acc_empty.arrive(n)
                n += 1
            tiles = following

    def mma(self):
        m = n = g = 0
        while (tiles := (yield from self.get(m))) >= 0:
            m += 1
            if tiles:
                yield self.own_full.wait(n)
                yield from self.walk(n, g, tiles)
                g, n = g + tiles, n + 1

    def commit(self, arrive):
        self.products.append(arrive)

    def stuck(self, seed):
        """The roles that wait for ever under this schedule."""
        rng = random.Random(seed)
        roles = {"items": self.items_and_ring1(), "ring2": self.ring2_loads(), "store": self.own_and_stores(),
                 "mma": self.mma(), **{f"elem{i}": self.elementwise() for i in range(self.ELEM)}}
        lag, weight = rng.choice([*roles, "copies", "products"]), rng.choice([1.0, 0.1, 0.01])
        waits = {k: next(r) for k, r in roles.items()}
        while waits:
            ready = [k for k, w in waits.items() if w is None or w[0].passed(w[1])]
            ready += ["copies"] * bool(self.copies) + ["products"] * bool(self.products)
            if not ready:
                return sorted(waits)
            k = rng.choices(ready, [weight if r == lag else 1.0 for r in ready])[0]
            if k == "copies":
                self.copies.pop(rng.randrange(len(self.copies)))()
            elif k == "products":
                self.products.pop(0)()
            else:
                try:
                    waits[k] = next(roles[k])
                except StopIteration:
                    del waits[k]
        return []


class DkDv(Block):
    def __init__(self, walks, acc_turns):
        super().__init__(walks, acc_turns)
        self.sdp, self.half = [Turns(1, 1), Turns(1, 1)], [Turns(1, self.ELEM), Turns(1, self.ELEM)]
        self.held = (self.ring1, self.ring2)

    def walk(self, n, g0, tiles):
        if g0:
            yield self.dp_free.wait(g0 - 1)
        yield self.full(self.ring1, g0)
        yield self.full(self.ring2, g0)
        for h in (0, 1):
            self.commit(lambda h=h: self.sdp[h].arrive(g0))
        if tiles == 1:
            self.commit(lambda: self.own_empty.arrive(n))
        for g in range(g0, g0 + tiles):
            more = g + 1 < g0 + tiles
            for h in (0, 1):
                if h and more:
                    yield self.full(self.ring2, g + 1)
                    yield self.dp_free.wait(g)
                    yield self.full(self.ring1, g + 1)
                    self.commit(lambda g=g: self.sdp[0].arrive(g + 1))
                yield self.half[h].wait(g)
                if not h and g == g0 and n:
                    yield self.acc_empty.wait(n - 1)
            if not more:
                self.commit(lambda: self.acc_full.arrive(n))
                continue
            self.commit(self.free(self.ring1, g))
            self.commit(self.free(self.ring2, g))
            yield self.full(self.ring2, g + 1)
            self.commit(lambda g=g: self.sdp[1].arrive(g + 1))
            if g + 2 == g0 + tiles:
                self.commit(lambda: self.own_empty.arrive(n))

    def tile(self, g):
        yield self.full(self.ring2, g)
        for h in (0, 1):
            yield self.sdp[h].wait(g)
            if h:
                self.dp_free.arrive(g)
            yield None
            self.half[h].arrive(g)


class Dq(Block):
    def __init__(self, walks, acc_turns, last_half_turns):
        super().__init__(walks, acc_turns)
        self.sdp, self.half = Turns(1, 1), [Turns(1, self.ELEM), Turns(last_half_turns, self.ELEM)]
        self.held = (self.ring1,)

    def walk(self, n, g0, tiles):
        def dp(g):
            yield self.full(self.ring2, g)
            self.commit(self.free(self.ring2, g))
            self.commit(lambda: self.sdp.arrive(g))
            if g + 1 == g0 + tiles:
                self.commit(lambda: self.own_empty.arrive(n))

        yield self.full(self.ring1, g0)
        if g0:
            yield self.dp_free.wait(g0 - 1)
        yield from dp(g0)
        for g in range(g0, g0 + tiles):
            more = g + 1 < g0 + tiles
            if more:
                yield self.full(self.ring1, g + 1)
            for h in (0, 1):
                if h and more:
                    yield self.dp_free.wait(g)
                    yield from dp(g + 1)
                yield self.half[h].wait(g)
                if not h and g == g0 and n:
                    yield self.acc_empty.wait(n - 1)
            self.commit(self.free(self.ring1, g) if more else lambda: self.acc_full.arrive(n))

    def tile(self, g):
        yield self.sdp.wait(g)
        for h in (0, 1):
            if h:
                self.dp_free.arrive(g)
            yield None
            self.half[h].arrive(g)


def _stuck(kind, lo, hi, seeds=150, **turns):
    """Schedules of 12 items of lo to hi tiles that end stuck."""
    return [s for s in range(seeds) if kind([random.Random(s).randint(lo, hi) for _ in range(12)], **turns).stuck(s)]


@pytest.mark.parametrize("lo,hi", [(1, 1), (1, 2), (2, 2), (3, 3), (0, 6), (20, 30)])
@pytest.mark.parametrize("kind", [DkDv, Dq])
def test_every_schedule_ends(kind, lo, hi):
    turns = {"last_half_turns": _turns("kLastHalfTurns")} if kind is Dq else {}
    assert _stuck(kind, lo, hi, 150 if hi < 20 else 30, acc_turns=_turns("kAccTurns"), **turns) == []


def test_every_schedule_of_the_causal_dq_ends():
    """The layer template's dQ kernel: the same roles, one item a block."""
    turns = _turns("kLastHalfTurns", "attention_bwd_tc.cu")
    assert not any(Dq([40], acc_turns=1, last_half_turns=turns).stuck(s) for s in range(300))


@pytest.mark.parametrize("kind,lo,hi,turns", [(DkDv, 1, 1, dict(acc_turns=1)),
                                              (Dq, 1, 1, dict(acc_turns=1, last_half_turns=2)),
                                              (Dq, 3, 3, dict(acc_turns=2, last_half_turns=1))])
def test_one_barrier_loses_a_phase(kind, lo, hi, turns):
    """What the turns are for: with one barrier some schedules get stuck."""
    assert _stuck(kind, lo, hi, **turns)
