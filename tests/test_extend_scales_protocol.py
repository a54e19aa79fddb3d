"""A random-interleaving model of the 8-bit extend kernel's K producer (host only): the K ring of four
stages beside the ring of eight steps' scales, which nothing releases, and what is left in flight when
a wait gives up.

The copies of a step (K, and two of scales on one barrier) land in any order and at any time.  S(t)
needs K(t) and P(t - 2), and an item's first two S steps the P of the item before; P(t) needs S(t) and
the scales of step t, in each of two tiles.  The producer fills step u once S of step u - 4 is complete
in both.  Checked: an entry of scales is never refilled before both tiles are done with it, no wait
tests a phase other than the next or the one before, and, from an abort at any moment, the waits that
the producer makes before it leaves cover every copy in flight.
"""
import random

import pytest

STAGES, RING = 4, 8


class Model:
    def __init__(self, items, seed):
        self.rnd = random.Random(seed)
        self.n = sum(items)
        self.first = []                     # per step: the first step of its item
        for n in items:
            self.first += [len(self.first)] * n
        self.filled = 0                     # steps the producer has issued
        self.flying = set()                 # (step, which copy)
        self.s = [0, 0]                     # S steps complete per tile
        self.p = [0, 0]                     # P steps complete per tile

    def landed(self, u, what):
        return u < self.filled and all((u, c) not in self.flying for c in what)

    def moves(self):
        out = [("land", c) for c in self.flying]
        u = self.filled
        if u < self.n and (u < STAGES or min(self.s) > u - STAGES):
            out.append(("fill", u))
        for x in range(2):
            t = self.s[x]
            if t < self.n and self.landed(t, ["K"]):
                need = t - 2 if t - 2 >= self.first[t] else self.first[t] - 1
                if self.p[x] > need:
                    out.append(("S", x))
            t = self.p[x]
            if t < self.s[x] and self.landed(t, ["sc0", "sc1"]):
                out.append(("P", x))
        return out

    def step(self):
        moves = self.moves()
        if not moves:
            return False
        kind, what = self.rnd.choice(sorted(moves, key=repr))
        if kind == "land":
            self.flying.discard(what)
        elif kind == "fill":
            if what >= RING:                # the entry's last user, and its barrier's phase
                assert min(self.p) > what - RING, "scales refilled while they are read"
                assert self.landed(what - RING, ["sc0", "sc1"]), "two phases of one barrier open"
            self.flying |= {(what, c) for c in ("K", "sc0", "sc1")}
            self.filled += 1
        elif kind == "S":
            self.s[what] += 1
        else:
            self.p[what] += 1
        return True

    def drain(self, scale_steps):
        """What flies on after the producer's last waits: the K barriers of the last STAGES steps, the
        scale barriers of the last `scale_steps`."""
        waited = {(u, "K") for u in range(max(0, self.filled - STAGES), self.filled)}
        for u in range(max(0, self.filled - scale_steps), self.filled):
            waited |= {(u, "sc0"), (u, "sc1")}
        return self.flying - waited


def random_items(rnd):
    return [rnd.randint(1, 9) for _ in range(rnd.randint(1, 6))]


@pytest.mark.parametrize("block", range(8))
def test_every_item_list_runs_to_its_end(block):
    for seed in range(block * 40, block * 40 + 40):
        items = random_items(random.Random(seed))
        m = Model(items, seed)
        while m.step():
            pass
        assert m.p == [m.n, m.n] and not m.flying


@pytest.mark.parametrize("block", range(8))
def test_no_copy_is_in_flight_when_an_aborted_producer_leaves(block):
    keys_only = 0
    for seed in range(block * 100, block * 100 + 100):
        rnd = random.Random(seed)
        m = Model(random_items(rnd), seed)
        for _ in range(rnd.randint(1, 60)):
            if not m.step():
                break
        assert not m.drain(RING)
        keys_only += bool(m.drain(0))
    assert keys_only  # waiting for the K stages alone leaves copies of scales in flight
