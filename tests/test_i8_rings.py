"""The 8-bit product's converter sets and their barriers (csrc/i8_tc.cuh), on
the CPU: the protocol of producer, two converter sets and MMA issuer, run step
by step in random order with barriers that answer parity waits as the hardware
does (a wait on parity p passes when the phase in progress has the other
parity).  For the ring depths of both configurations no stage may be read
before it holds its step's load, no slot overwritten before its MMAs ran, and
everything must finish.  The same check finds the order of waits that is
wrong for odd rings."""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "dense_fp32_matrix_03_gb300", "csrc", "i8_tc.cuh")


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return self.phase & 1 != parity


def simulate(slots, ring, steps, seed, slot_first=True):
    """One ring (weights or tokens) into the widened slots.  Loads land in any
    order.  Returns True when every step finished, "stale" at the first wrong
    read or write, False when nothing can move."""
    rng = random.Random(seed)
    full = [Barrier(1) for _ in range(ring)]
    empty = [Barrier(1) for _ in range(ring)]
    ready = [Barrier(1) for _ in range(slots)]
    slot_empty = [Barrier(1) for _ in range(slots)]
    stage, slot = [None] * ring, [None] * slots
    flying, done = [], []

    def producer():
        for n in range(steps):
            while not empty[n % ring].passed((n // ring & 1) ^ 1):
                yield
            flying.append(n)
            yield

    def loads():
        while True:
            if flying and rng.random() < 0.5:
                n = flying.pop(rng.randrange(len(flying)))
                stage[n % ring] = n
                full[n % ring].arrive()
            yield

    def converter(which):
        for n in range(which, steps, 2):
            waits = [(slot_empty[n % slots], (n // slots & 1) ^ 1), (full[n % ring], n // ring & 1)]
            for bar, parity in waits if slot_first else waits[::-1]:
                while not bar.passed(parity):
                    yield
            if stage[n % ring] != n or slot[n % slots] is not None:
                done.append("stale")
                return
            slot[n % slots] = n
            yield
            empty[n % ring].arrive()
            ready[n % slots].arrive()
            yield

    def mma():
        for n in range(steps):
            while not ready[n % slots].passed(n // slots & 1):
                yield
            yield
            if slot[n % slots] != n:
                done.append("stale")
                return
            slot[n % slots] = None
            slot_empty[n % slots].arrive()
            yield
        done.append(True)

    roles = {"p": producer(), "l": loads(), "a": converter(0), "b": converter(1), "m": mma()}
    speed = {r: rng.choice([1, 1, 3, 10]) for r in roles}
    for _ in range(4000 * steps):
        name = rng.choices(list(roles), [speed[r] for r in roles])[0]
        next(roles[name], None)
        if done:
            return done[0]
        if rng.random() < 0.02:
            speed[rng.choice(list(roles))] = rng.choice([1, 1, 3, 10])
    return False


def depths():
    text = open(SOURCE).read()
    found = {}
    for name in ("Narrow", "Wide"):
        m = re.search(rf"using {name} = Cfg<(\d+), (\d+), (\d+), (\d+), (\d+), (\d+)>", text)
        assert m, name
        found[name] = tuple(int(x) for x in m.groups())
    return found


@pytest.mark.parametrize("which", ["Narrow", "Wide"])
def test_shipped_depths(which):
    _, _, slots, wring, tring, _ = depths()[which]
    for ring in (wring, tring):
        assert ring % 2 == 0 or ring >= slots
        for seed in range(60):
            assert simulate(slots, ring, 40, seed) is True, (slots, ring, seed)


@pytest.mark.parametrize("slots,ring", [(2, 3), (3, 3), (3, 5), (4, 4), (4, 2), (3, 2)])
def test_rule_of_the_depths(slots, ring):
    assert all(simulate(slots, ring, 40, seed) is True for seed in range(40))


@pytest.mark.parametrize("slots,ring,slot_first", [(3, 3, False), (4, 3, True), (4, 3, False)])
def test_unsound_orders_are_found(slots, ring, slot_first):
    assert any(simulate(slots, ring, 40, seed, slot_first) is not True for seed in range(200))
