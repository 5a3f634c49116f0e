"""A model of the synchronisation of the linear kernel's CTA pairs, run on the CPU under random
interleavings.  The actors are the kernel's: the two CTAs' producers, the leader's issuer, and the
eight epilogue warps of either CTA; the copies and the products complete asynchronously.  The
barriers are mbarriers as the kernel sets them up (arrival counts, transaction bytes, parity waits).

Checked: a stage is filled only after its products are done, the products read the K block that
belongs to them in both CTAs, an accumulator is written only after all sixteen warps have it out
and read only when it is whole, no waiter misses a phase, and everything ends."""
import random

import pytest

STAGES, BYTES = 6, 2


class Bar:
    """count arrivals and zero outstanding bytes end a phase."""

    def __init__(self, count):
        self.count, self.pending, self.tx, self.phase = count, count, 0, 0

    def step(self, arrivals=0, tx=0):
        self.pending -= arrivals
        self.tx += tx
        assert self.pending >= 0, "an arrival too many"
        if self.pending == 0 and self.tx == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def done(self, parity, seen):
        """try_wait.parity; `seen` is the number of phases the waiter has to find complete."""
        ok = (self.phase & 1) != parity
        if ok:
            assert self.phase == seen, "a waiter saw a barrier in another phase than it waits for"
        return ok


class Pair:
    def __init__(self, items, rng, acc_empty_count=16, peer_waits=True, buffers=2):
        self.items, self.rng, self.peer_waits, self.buffers = items, rng, peer_waits, buffers
        self.full = [Bar(1) for _ in range(STAGES)]                       # the leader's
        self.empty = [[Bar(1) for _ in range(STAGES)] for _ in range(2)]  # each CTA's
        self.acc_full = [[Bar(1) for _ in range(2)] for _ in range(2)]
        self.acc_empty = [Bar(acc_empty_count) for _ in range(2)]         # the leader's
        self.smem = [[None] * STAGES for _ in range(2)]                   # K block a stage holds
        self.reading = [[0] * STAGES for _ in range(2)]                   # products that still read it
        self.acc = [[None, 0] for _ in range(2)]                          # item, warps that have to read it
        self.asyncs = []                                                  # copies: any order
        self.tensor = []                                                  # products and commits: in order
        self.read = []

    def producer(self, cta):
        g = 0
        for it, n in enumerate(self.items):
            for kb in range(n):
                s = g % STAGES
                if g >= STAGES and (cta == 0 or self.peer_waits):
                    while not self.empty[cta][s].done((g // STAGES - 1) & 1, g // STAGES):
                        yield
                if cta == 0:
                    self.full[s].step(arrivals=1, tx=2 * BYTES)
                    yield

                def land(s=s, block=(it, kb)):
                    assert self.reading[cta][s] == 0, "a stage is overwritten under its products"
                    self.smem[cta][s] = block
                    self.full[s].step(tx=-BYTES)
                self.asyncs.append(land)
                g += 1
                yield

    def issuer(self):
        g = 0
        for it, n in enumerate(self.items):
            buf = it % self.buffers
            use = it // self.buffers
            if use > 0:
                while not self.acc_empty[buf].done((use - 1) & 1, use):
                    yield
            for kb in range(n):
                s = g % STAGES
                while not self.full[s].done((g // STAGES) & 1, g // STAGES + 1):
                    yield
                for cta in range(2):
                    assert self.smem[cta][s] == (it, kb), "the products read another K block"
                    self.reading[cta][s] += 1

                def product(s=s, it=it, kb=kb, buf=buf):
                    assert self.acc[buf][1] == 0, "an accumulator is overwritten before it is out"
                    self.acc[buf][0] = it
                    for cta in range(2):
                        self.reading[cta][s] -= 1
                        self.empty[cta][s].step(arrivals=1)
                self.tensor.append(product)
                g += 1
                yield

            def whole(buf=buf):
                self.acc[buf][1] = 16
                for cta in range(2):
                    self.acc_full[cta][buf].step(arrivals=1)
            self.tensor.append(whole)
            yield

    def epilogue(self, cta, warp):
        for it in range(len(self.items)):
            buf, use = it % self.buffers, it // self.buffers
            while not self.acc_full[cta][buf].done(use & 1, use + 1):
                yield
            assert self.acc[buf][0] == it, "an epilogue warp reads another tile's accumulator"
            yield
            assert self.acc[buf][0] == it, "an accumulator changed while it was read"
            self.acc[buf][1] -= 1
            self.acc_empty[buf].step(arrivals=1)
            self.read.append((cta, warp, it))
            yield

    def run(self, limit=400000):
        actors = [self.producer(0), self.producer(1), self.issuer(),
                  *(self.epilogue(c, w) for c in range(2) for w in range(8))]
        for _ in range(limit):
            choices = len(actors) + (2 if self.asyncs else 0) + (2 if self.tensor else 0)
            if choices == 0:
                break
            i = self.rng.randrange(choices)
            if i < len(actors):
                if next(actors[i], "end") == "end":
                    actors.pop(i)
            elif self.asyncs and i < len(actors) + 2:
                self.asyncs.pop(self.rng.randrange(len(self.asyncs)))()
            elif self.tensor:
                self.tensor.pop(0)()
        else:
            raise AssertionError("the pair did not end")
        assert len(self.read) == 16 * len(self.items)


@pytest.mark.parametrize("seed", range(12))
def test_pairs_protocol(seed):
    rng = random.Random(seed)
    items = [rng.choice([1, 2, 5, 7, 16]) for _ in range(rng.randint(1, 9))]
    Pair(items, rng).run()


MISTAKES = {"the accumulator is handed back by one CTA's warps alone": dict(acc_empty_count=8),
            "the other CTA fills its stages without waiting": dict(peer_waits=False),
            "one accumulator for barriers meant for two": dict(buffers=1)}


@pytest.mark.parametrize("what", MISTAKES)
def test_planted_mistakes_are_caught(what):
    if what.startswith("one accumulator"):
        # a tile whose products start before the last one is out
        class Early(Pair):
            def issuer(self):
                self.acc_empty[0].done = lambda parity, seen: True
                yield from super().issuer()
        make = lambda rng: Early([7] * 6, rng, buffers=1)
    else:
        make = lambda rng: Pair([7] * 6, rng, **MISTAKES[what])
    caught = 0
    for seed in range(20):
        try:
            make(random.Random(seed)).run()
        except AssertionError:
            caught += 1
    assert caught >= 15, (what, caught)


class AbortingPair(Pair):
    """The same with bounded waits, as the kernel gives up: a wait that is over its bound sets its CTA's
    flag, and each wait of that CTA ends on it; the issuer signals the end of its products, whatever
    happened.  When all warps of a CTA are through and its flag is set, the leader's producer waits for
    the copies of its last stages, and the other CTA's gives its own some time.  Time is the scheduler's
    steps; a copy lands within COPY of them, and a product is done within as many.

    one_deadline: the drain has one bound for all stages.  drains: "flag" as above; "own": a producer
    drains only when its own wait ended early; "never"."""
    COPY, DRAIN, REST = 150, 1500, 300

    def __init__(self, items, rng, bound, one_deadline=True, drains="flag"):
        super().__init__(items, rng)
        self.bound, self.one_deadline, self.drains = bound, one_deadline, drains
        self.now, self.flag, self.drain = 0, [False, False], [Bar(1), Bar(1)]
        self.live, self.drained = [10, 10], 0

    def wait(self, cta, bar, parity, seen):
        """The generator's value is whether the phase was complete in time."""
        t0 = self.now
        while not bar.done(parity, seen):
            if self.flag[cta] or self.now - t0 > self.bound:
                self.flag[cta] = True
                return False
            yield
        return True

    def fill(self, cta):
        """The copies; (K blocks that were asked for, whether that is all of them)."""
        g = 0
        for it, n in enumerate(self.items):
            for kb in range(n):
                s = g % STAGES
                if g >= STAGES and not (yield from self.wait(cta, self.empty[cta][s], (g // STAGES - 1) & 1, g // STAGES)):
                    return g, False
                if cta == 0:
                    self.full[s].step(arrivals=1, tx=2 * BYTES)
                    yield

                def land(s=s, block=(it, kb)):
                    self.smem[cta][s] = block
                    self.full[s].step(tx=-BYTES)
                self.asyncs.append((self.now, land))
                g += 1
                yield
        return g, True

    def producer(self, cta):
        g, ok = yield from self.fill(cta)
        while self.live[cta] > 1 and self.drains != "own":
            yield
        if self.drains == "never" or (ok if self.drains == "own" else not self.flag[cta]):
            return
        t0 = self.now
        if cta == 0:
            for x in range(max(0, g - STAGES), g):
                since = t0 if self.one_deadline else self.now
                while not self.full[x % STAGES].done((x // STAGES) & 1, x // STAGES + 1) and self.now - since <= self.DRAIN:
                    yield
            self.drained = self.now - t0
        else:
            while self.now - t0 < self.REST:
                yield

    def products(self):
        g = 0
        for it, n in enumerate(self.items):
            buf, use = it % 2, it // 2
            if use > 0 and not (yield from self.wait(0, self.acc_empty[buf], (use - 1) & 1, use)):
                return
            for kb in range(n):
                s = g % STAGES
                if not (yield from self.wait(0, self.full[s], (g // STAGES) & 1, g // STAGES + 1)):
                    return
                for cta in range(2):
                    assert self.smem[cta][s] == (it, kb), "the products read another K block"

                def product(s=s):
                    for cta in range(2):
                        self.empty[cta][s].step(arrivals=1)
                self.tensor.append((self.now, product))
                g += 1
                yield

            def whole(buf=buf):
                for cta in range(2):
                    self.acc_full[cta][buf].step(arrivals=1)
            self.tensor.append((self.now, whole))
            yield

    def issuer(self, cta):
        if cta == 0:
            yield from self.products()
            self.tensor.append((self.now, lambda: [b.step(arrivals=1) for b in self.drain]))
            yield
        t0 = self.now
        while not self.drain[cta].done(0, 1) and self.now - t0 <= 100 * self.DRAIN:
            yield

    def epilogue(self, cta, warp):
        for it in range(len(self.items)):
            buf, use = it % 2, it // 2
            if not (yield from self.wait(cta, self.acc_full[cta][buf], use & 1, use + 1)):
                return
            yield
            self.acc_empty[buf].step(arrivals=1)
            self.read.append((cta, warp, it))
            yield

    def run(self, limit=400000):
        actors = [(c, a) for c in range(2) for a in (self.producer(c), self.issuer(c), *(self.epilogue(c, w) for w in range(8)))]
        for self.now in range(limit):
            late = [q for q in (self.asyncs, self.tensor) if q and self.now - q[0][0] > self.COPY]
            i = self.rng.randrange(len(actors) + 2)
            if late:
                late[0].pop(0)[1]()
            elif i < len(actors):
                if next(actors[i][1], "end") == "end":
                    self.live[actors.pop(i)[0]] -= 1
                    if not actors:                       # both CTAs are at their last barrier
                        break
            elif i == len(actors) and self.asyncs:
                self.asyncs.pop(self.rng.randrange(len(self.asyncs)))[1]()
            elif i > len(actors) and self.tensor:
                self.tensor.pop(0)[1]()
        else:
            raise AssertionError("the pair did not end")
        assert not self.asyncs, "a copy is under way when its CTA ends"
        assert not self.tensor, "a product is under way when its CTA ends"
        # a step belongs to one of up to 22 choices, so the last look may come some hundred steps late
        assert self.drained <= self.DRAIN + 300, "the drain takes more than its bound"
        return any(self.flag)


def aborts(**how):
    """Pairs whose waits run out at any point, so that producers stop at different blocks."""
    for seed in range(200):
        rng = random.Random(seed)
        items = [rng.choice([1, 2, 5, 7, 16]) for _ in range(rng.randint(2, 9))]
        yield AbortingPair(items, rng, rng.choice([5, 20, 60, 100, 150, 250]), **how)


def test_pairs_protocol_abort():
    """The pair ends, with nothing under way, and the drain keeps to its bound."""
    assert sum(pair.run() for pair in aborts()) >= 100


@pytest.mark.parametrize("mistake,said", [(dict(one_deadline=False), "the drain takes more"), (dict(drains="never"), "a copy is"),
                                          (dict(drains="own"), "a copy is")],
                         ids=["a bound for each stage", "no drain", "a drain only for the producer's own waits"])
def test_planted_mistakes_of_an_abort_are_caught(mistake, said):
    caught = 0
    for pair in aborts(**mistake):
        try:
            pair.run()
        except AssertionError as e:
            assert said in str(e)
            caught += 1
    assert caught >= 5, caught
