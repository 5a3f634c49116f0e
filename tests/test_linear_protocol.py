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
