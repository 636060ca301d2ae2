"""A model of the barrier protocol of the token attention kernel (la_cache_token.cu): the copying
warp and the four that compute, written out as their sequences of waits, arrivals and accesses, run
by a scheduler that interleaves them at random and lets copies land at random times in any order.
A wait passes by its barrier's parity, as on the hardware: a warp that skipped a stage's filling
passes too early if the one before has not landed.  Checked: every run ends; each reader finds the
tile, q, operands and sums it was meant for, from its first access to its last.  Planted
mistakes have to fail it."""
import random

import pytest

from test_prompt_protocol_cpu import Bar, Fault


class Model:
    """units: the key tiles of each unit of a block's share.  groups: row groups (1: two warps take a
    tile, the other two the next; 2: all four take every tile)."""

    def __init__(self, units, stages, groups, seed, mistake=None):
        self.units, self.stages, self.groups, self.mistake = units, stages, groups, mistake
        self.rng = random.Random(seed)
        some = lambda n, k, c: [Bar(f"{n}[{i}]", c) for i in range(k)]  # noqa: E731
        sharers = 1 if mistake == "a stage that one warp releases" else 2 * groups
        self.full, self.empty = some("full", stages, 1), some("empty", stages, sharers)
        self.q_full, self.q_empty = some("q_full", 2, 1), some("q_empty", 2, 4)
        self.four = Bar("four", 4)
        self.copies = []                       # (buffer, place, contents, barrier) in flight
        self.stage, self.raw = [None] * stages, [None] * 2
        self.operands, self.sums = [None] * 4, [None] * 4
        self.done = []

    def expect(self, got, want, what):
        if got != want:
            raise Fault(f"{what}: {got} instead of {want}")

    def copy(self, buffer, place, contents, bar):
        buffer[place] = None
        self.copies.append((buffer, place, contents, bar))

    def copying(self):
        it = 0
        for u, n in enumerate(self.units):
            if u >= 2 and self.mistake != "no wait for q to be read":
                yield self.q_empty[u & 1], (u >> 1) - 1
            self.copy(self.raw, u & 1, u, self.q_full[u & 1])
            for i in range(n):
                s = it % self.stages
                if it >= self.stages and self.mistake != "no wait for a stage":
                    yield self.empty[s], it // self.stages - 1
                self.copy(self.stage, s, (u, i), self.full[s])
                it += 1
                yield None

    def sync(self, phase):
        yield self.four.arrive
        yield self.four, phase

    def computing(self, w):
        it = phase = 0
        for u, n in enumerate(self.units):
            yield self.q_full[u & 1], u >> 1
            self.expect(self.raw[u & 1], u, "q")
            yield None
            self.operands[w] = u
            self.expect(self.raw[u & 1], u, "q, at the end")
            yield self.q_empty[u & 1].arrive
            if self.mistake != "no barrier before the tiles":
                yield from self.sync(phase)
                phase += 1
            for i in range(n):
                s, k = it % self.stages, it // self.stages
                it += 1
                if self.groups == 1 and (i ^ (w >> 1)) & 1 and self.mistake != "all warps take every stage":
                    continue
                if i and self.rng.random() < 0.2:      # a chain ends: sums into the warp's buffer
                    self.sums[w] = (u, "some")
                yield self.full[s], k
                for _ in range(2):
                    self.expect(self.stage[s], (u, i), f"stage {s}")
                    self.expect(self.operands, [u] * 4, "operands")
                    yield None
                yield self.empty[s].arrive
            self.sums[w] = (u, "all")
            if self.mistake != "no barrier at the end":
                yield from self.sync(phase)
                phase += 1
            for _ in range(2):
                self.expect(self.sums, [(u, "all")] * 4, "sums")
                yield None
            self.done.append((u, w))

    def run(self):
        roles = [self.computing(w) for w in range(4)] + [self.copying()]
        speed = [self.rng.choice([0.05, 0.3, 1.0]) for _ in range(len(roles) + 1)]
        at = [next(r, StopIteration) for r in roles]
        idle = 0
        while any(a is not StopIteration for a in at):
            idle += 1
            if idle > 20000:
                raise Fault("no progress")
            k = self.rng.randrange(len(roles) + 1)
            if self.rng.random() > speed[k]:
                continue
            if k == len(roles):
                if self.copies:
                    buffer, place, contents, bar = self.copies.pop(self.rng.randrange(len(self.copies)))
                    buffer[place] = contents
                    bar.arrive()
                    idle = 0
                continue
            a = at[k]
            if a is StopIteration or (isinstance(a, tuple) and not a[0].passed(a[1])):
                continue
            if a is not None and not isinstance(a, tuple):
                a()
            at[k], idle = next(roles[k], StopIteration), 0
        assert sorted(self.done) == [(u, w) for u in range(len(self.units)) for w in range(4)]
        if self.copies:
            raise Fault("copies in flight at the end")


def units_of(rng):
    return [rng.choice([1, 1, 2, 3, 4, 5, 6, 7, 13]) for _ in range(rng.randint(1, 8))]


# stages and row groups as the kernel has them for d = 128 and 64
@pytest.mark.parametrize("stages,groups", [(4, 1), (3, 2), (6, 1), (5, 2)])
def test_protocol(stages, groups):
    rng = random.Random(stages)
    for seed in range(150):
        Model(units_of(rng), stages, groups, seed).run()


@pytest.mark.parametrize("stages,groups,mistake", [
    (3, 1, None),                       # an odd number of stages, two pairs of warps in turn
    (5, 1, None),
    (4, 1, "a stage that one warp releases"), (3, 2, "a stage that one warp releases"),
    (4, 1, "no wait for a stage"), (4, 1, "no wait for q to be read"),
    (4, 1, "no barrier before the tiles"), (4, 1, "no barrier at the end"),
    (4, 1, "all warps take every stage"),
])
def test_planted_protocol_mistakes(stages, groups, mistake):
    rng, caught = random.Random(1), 0
    for seed in range(80):
        try:
            Model(units_of(rng), stages, groups, seed, mistake).run()
        except Fault:
            caught += 1
    assert caught > 0
