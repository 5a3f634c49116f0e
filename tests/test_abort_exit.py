"""A model of how a CTA of the attention and projection kernels ends when a wait runs out: a producer
asks for copies into a ring of stages, an issuer multiplies them, readers take the results out.  A wait
over its bound sets the CTA's flag, and every wait then ends.  Checked under random interleavings:
nothing that writes to the CTA's memory is under way when its last warp is through.  Copies land, and
products end, at random; a role that waits for its own before it ends is modelled with a bound that a
copy never reaches."""
import random

import pytest

STAGES = 3


class Cta:
    """always: the producer and the issuer wait for their last copies and products; else only when a
    wait of their own ran out."""

    def __init__(self, blocks, rng, bound, always=True):
        self.blocks, self.rng, self.bound, self.always = blocks, rng, bound, always
        self.now, self.flag, self.copies, self.products = 0, False, [], []
        self.full, self.empty, self.out = set(), set(), set()       # blocks whose phase is complete

    def wait(self, done, key):
        t0 = self.now
        while key not in done:
            if self.flag or self.now - t0 > self.bound:
                self.flag = True
                return False
            yield
        return True

    def producer(self):
        ok, g = True, 0
        while g < self.blocks and ok:
            if g >= STAGES:
                ok = yield from self.wait(self.empty, g - STAGES)
            if ok:
                self.copies.append(g)
                g += 1
            yield
        while (self.always or not ok) and self.copies:
            yield

    def issuer(self):
        ok, g = True, 0
        while g < self.blocks and ok:
            ok = yield from self.wait(self.full, g)
            if ok:
                self.products.append(g)
                g += 1
            yield
        while (self.always or not ok) and self.products:
            yield

    def reader(self):
        for g in range(self.blocks):
            if not (yield from self.wait(self.out, g)):
                return
            yield

    def run(self):
        roles = [self.producer(), self.issuer(), self.reader(), self.reader()]
        while roles:
            self.now += 1
            i = self.rng.randrange(len(roles) + 2)
            if i < len(roles):
                if next(roles[i], "end") == "end":
                    roles.pop(i)
            elif i == len(roles) and self.copies:
                self.full.add(self.copies.pop(self.rng.randrange(len(self.copies))))
            elif i > len(roles) and self.products:
                g = self.products.pop(0)
                self.empty.add(g)
                self.out.add(g)
        return self.flag, bool(self.copies or self.products)


def ends(always):
    rng = random.Random(3)
    return [Cta(rng.randint(1, 12), rng, rng.choice([3, 10, 30, 100]), always).run() for _ in range(2000)]


def test_nothing_is_under_way_at_the_end():
    got = ends(True)
    assert sum(gave_up for gave_up, _ in got) >= 500
    assert not any(left for _, left in got)


def test_waiting_only_after_an_own_wait_ran_out_is_caught():
    assert sum(left for _, left in ends(False)) >= 20
