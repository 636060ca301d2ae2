"""A model of the barrier protocol of the prompt attention kernel (la_cache_prompt.cu): its warps
written out as their sequences of waits, arrivals and products, run by a scheduler that
interleaves them at random and executes products in issue order at random times.  Checked: every run
ends; no wait meets its barrier two phases ahead (a parity could not tell); each product and
each reader finds the operand version it was meant for.  Planted mistakes have to fail it."""
import random

import pytest


class Fault(Exception):
    pass


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.phases = name, count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phases = self.count, self.phases + 1

    def passed(self, phase):
        if self.phases >= phase + 2:
            raise Fault(f"{self.name}: waiting for phase {phase}, {self.phases} are over")
        return self.phases == phase + 1


class Model:
    """units: for each unit of a block's share the key tiles of row tile 0 and of row tile 1."""

    def __init__(self, units, slots, seed, mistake=None):
        self.units, self.slots, self.mistake = units, slots, mistake
        self.rng = random.Random(seed)
        two = lambda n, c: [Bar(f"{n}[{t}]", c) for t in range(2)]  # noqa: E731
        self.kv_full = [Bar(f"kv_full[{i}]", 4) for i in range(slots)]
        self.kv_empty = [Bar(f"kv_empty[{i}]", 1) for i in range(slots)]
        self.q_full, self.s_full, self.p_full, self.o_full = two("q", 4), two("s", 1), two("p", 4), two("o", 1)
        self.e_full, self.e_empty = two("e_full", 1), two("e_empty", 8)
        self.queue = []                                   # products and commits in issue order
        self.slot = [[None] * 4 for _ in range(slots)]    # what each converting warp wrote
        self.q = [[None] * 4 for _ in range(2)]
        self.p = [[None] * 4 for _ in range(2)]
        self.s, self.o, self.e = [None, None], [None, None], [None, None]
        self.named = [0, 0]                               # the converting warps' block barrier
        self.stored = set()

    def expect(self, got, want, what):
        if got != want:
            raise Fault(f"{what}: {got} instead of {want}")

    def unread(self, kind, key):
        """No product still to run reads this buffer."""
        if any(op[0] == kind and key in op[1] for op in self.queue):
            raise Fault(f"{key} written under a product that reads it")

    def softmax(self, t, w):
        it = used = 0
        for seg, c in enumerate(self.units):
            if c[t]:
                self.unread("mma", ("q", t))
                self.q[t][w] = seg
                yield self.q_full[t].arrive
            k = seg & 1
            if self.mistake == "one e barrier":
                yield self.e_full[0], seg
                self.expect(self.e[k], seg, "scale references")
                yield self.e_empty[0].arrive
            else:
                yield self.e_full[k], seg >> 1
                self.expect(self.e[k], seg, "scale references")
                yield self.e_empty[k].arrive
            for i in range(c[t]):
                yield self.s_full[t], it
                self.expect(self.s[t], (seg, i), f"scores {t}")
                if i and self.rng.random() < 0.3:          # the maximum grows: O is rescaled
                    self.expect(self.o[t], (seg, i - 1), f"O {t} to rescale")
                self.p[t][w] = (seg, i)
                yield self.p_full[t].arrive
                it += 1
            if c[t]:
                if self.mistake != "no wait for the output":
                    yield self.o_full[t], used
                used += 1
                self.expect(self.o[t], (seg, c[t] - 1), f"output {t}")
            self.stored.add((seg, t, w))

    def block_sync(self):
        """The barrier of the four converting warps."""
        mine = self.named[0] // 4
        self.named[0] += 1
        while self.named[0] < 4 * (mine + 1):
            yield None

    def convert(self, w):
        u = 0
        for seg, c in enumerate(self.units):
            yield from self.block_sync()
            if seg >= 2 and self.mistake == "one e barrier":
                yield self.e_empty[0], seg - 2
            elif seg >= 2 and (w == 0 or self.mistake == "every converting warp waits"):
                yield self.e_empty[seg & 1], (seg >> 1) - 1
            if w == 0:
                self.e[seg & 1] = seg
                yield (self.e_full[0 if self.mistake == "one e barrier" else seg & 1]).arrive
            yield from self.block_sync()
            for i in range(max(c)):
                for kind in "kv":
                    s = u % self.slots
                    if u >= self.slots and self.mistake != "no wait for a slot":
                        yield self.kv_empty[s], u // self.slots - 1
                    self.unread("mma", ("slot", s))
                    self.slot[s][w] = (seg, i, kind)
                    yield self.kv_full[s].arrive
                    u += 1

    def scores(self, t, u, seg, i):
        s = u % self.slots

        def run():
            self.expect(self.slot[s], [(seg, i, "k")] * 4, f"slot {s}")
            self.expect(self.q[t], [seg] * 4, f"q {t}")
            if i:
                self.expect(self.p[t], [(seg, i - 1)] * 4, f"weights {t} before new scores")
            self.s[t] = (seg, i)
        self.queue += [("mma", (("slot", s), ("q", t)), run), ("commit", (), self.s_full[t].arrive)]

    def issue(self):
        u, it, units = 0, [0, 0], [0, 0]
        commit = lambda b: self.queue.append(("commit", (), b.arrive))  # noqa: E731
        for seg, c in enumerate(self.units):
            n = max(c)
            for t in range(2):
                if c[t]:
                    yield self.q_full[t], units[t]
                    yield self.kv_full[u % self.slots], u // self.slots
                    units[t] += 1
                    self.scores(t, u, seg, 0)
            if n:
                commit(self.kv_empty[u % self.slots])
            for i in range(n):
                v = u + 1
                for t in range(2):
                    if i >= c[t]:
                        continue
                    if self.mistake != "no wait for weights":
                        yield self.p_full[t], it[t]
                    yield self.kv_full[v % self.slots], v // self.slots
                    it[t] += 1

                    def run(t=t, i=i, seg=seg, s=v % self.slots):
                        self.expect(self.slot[s], [(seg, i, "v")] * 4, f"slot {s}")
                        self.expect(self.p[t], [(seg, i)] * 4, f"weights {t}")
                        if i:
                            self.expect(self.o[t], (seg, i - 1), f"O {t}")
                        self.o[t] = (seg, i)
                    self.queue.append(("mma", (("slot", v % self.slots),), run))
                    if i + 1 < c[t]:
                        yield self.kv_full[(u + 2) % self.slots], (u + 2) // self.slots
                        self.scores(t, u + 2, seg, i + 1)
                    else:
                        commit(self.o_full[t])
                commit(self.kv_empty[v % self.slots])
                if i + 1 < n:
                    commit(self.kv_empty[(u + 2) % self.slots])
                u += 2

    def run(self):
        roles = [self.softmax(t, w) for t in range(2) for w in range(4)]
        roles += [self.convert(w) for w in range(4)] + [self.issue()]
        speed = [self.rng.choice([0.05, 0.3, 1.0]) for _ in roles] + [self.rng.choice([0.05, 0.3, 1.0])]
        at = [next(r, StopIteration) for r in roles]
        idle = 0
        while any(a is not StopIteration for a in at) or self.queue:
            k = self.rng.randrange(len(roles) + 1)
            idle += 1
            if idle > 20000:
                raise Fault("no progress")
            if self.rng.random() > speed[k]:
                continue
            if k == len(roles):
                if self.queue:
                    self.queue.pop(0)[2]()
                    idle = 0
                continue
            a = at[k]
            if a is StopIteration:
                continue
            if isinstance(a, tuple):
                if not a[0].passed(a[1]):
                    continue
            elif a is not None:
                a()
            new = next(roles[k], StopIteration)
            if a is not None or new is not None:
                idle = 0
            at[k] = new
        assert self.stored == {(s, t, w) for s in range(len(self.units)) for t in range(2) for w in range(4)}


def units_of(rng):
    kinds = [(1, 1), (1, 2), (0, 1), (0, 0), (3, 3), (4, 5), (2, 0), (9, 10), (1, 0)]
    return [rng.choice(kinds) for _ in range(rng.randint(1, 9))]


@pytest.mark.parametrize("slots", [5, 8])
def test_protocol(slots):
    rng = random.Random(slots)
    for seed in range(150):
        Model(units_of(rng), slots, seed).run()


@pytest.mark.parametrize("mistake", ["one e barrier", "every converting warp waits",
                                     "no wait for the output", "no wait for a slot",
                                     "no wait for weights"])
def test_planted_protocol_mistakes(mistake):
    rng, caught = random.Random(1), 0
    for seed in range(150):
        try:
            Model(units_of(rng), 8, seed, mistake).run()
        except Fault:
            caught += 1
    assert caught > 0
