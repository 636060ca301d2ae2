"""A model of the barrier protocol of the prompt attention kernel (la_cache_prompt.cu): its warps
written out as their sequences of waits, arrivals and products, run by a scheduler that
interleaves them at random and executes products in issue order at random times.  A wait passes by its
barrier's parity, as on the hardware, so one that is two phases off passes too early or never.
Checked: every run ends; each product and each reader finds the operand version it was meant for.
Planted mistakes have to fail it."""
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
        """As the hardware tells it: by the parity of the phase under way."""
        return self.phases % 2 != phase % 2


class Model:
    """units: for each unit of a block's share the key tiles that row tile 0 and row tile 1 see."""

    PLANS = 4

    def __init__(self, units, slots, seed, mistake=None):
        self.units, self.slots, self.mistake = units, slots, mistake
        self.rng = random.Random(seed)
        some = lambda n, k, c: [Bar(f"{n}[{t}]", c) for t in range(k)]  # noqa: E731
        self.kv_full, self.kv_empty = some("kv_full", slots, 8), some("kv_empty", slots, 1)
        self.q_full, self.s_full, self.o_full = some("q", 2, 4), some("s", 2, 1), some("o", 2, 1)
        self.p_full = some("p", 4, 4)                     # for each row tile its two halves
        self.u_full, self.u_empty = some("u_full", self.PLANS, 1), some("u_empty", self.PLANS, 17)
        self.queue = []                                   # products and commits in issue order
        self.slot = [[None] * 8 for _ in range(slots)]    # what each converting warp wrote
        self.q = [[None] * 4 for _ in range(2)]
        self.p = [[None] * 4 for _ in range(4)]
        self.s, self.o = [None] * 2, [None] * 2
        self.plan = [None] * self.PLANS
        self.stored = set()

    def expect(self, got, want, what):
        if got != want:
            raise Fault(f"{what}: {got} instead of {want}")

    def unread(self, key):
        """No product still to run reads this buffer."""
        if any(key in op[0] for op in self.queue):
            raise Fault(f"{key} written under a product that reads it")

    def unit(self, seg):
        k = seg % self.PLANS
        yield self.u_full[k], seg // self.PLANS
        self.expect(self.plan[k], seg, "plan")
        if seg < len(self.units):
            yield self.u_empty[k].arrive

    def planner(self):
        for seg in range(len(self.units) + 1):
            k = seg % self.PLANS
            if seg >= self.PLANS and self.mistake != "no wait for the readers of a plan":
                yield self.u_empty[k], seg // self.PLANS - 1
            self.plan[k] = seg
            yield self.u_full[k].arrive

    def softmax(self, t, w):
        it = used = 0
        for seg, c in enumerate(self.units):
            yield from self.unit(seg)
            if c[t]:
                self.unread(("q", t))
                self.q[t][w] = seg
                yield self.q_full[t].arrive
            for i in range(c[t]):
                yield self.s_full[t], it
                self.expect(self.s[t], (seg, i), f"scores {t}")
                if i and self.rng.random() < 0.3:          # the maximum grows: O is rescaled
                    self.expect(self.o[t], (seg, i - 1), f"O {t} to rescale")
                for h in range(2):
                    self.expect(self.s[t], (seg, i), f"scores {t}, half {h}")
                    self.p[2 * t + h][w] = (seg, i)
                    yield self.p_full[2 * t + (0 if self.mistake == "one barrier for both halves" else h)].arrive
                it += 1
            if c[t]:
                if self.mistake != "no wait for the output":
                    yield self.o_full[t], used
                used += 1
                self.expect(self.o[t], (seg, c[t] - 1), f"output {t}")
                self.unread(("q", t))                      # rows go out through the q tile
            self.stored.add((seg, t, w))
        yield from self.unit(len(self.units))

    def convert(self, w):
        u = 0
        for seg, c in enumerate(self.units):
            yield from self.unit(seg)
            for i in range(max(c)):
                for kind in "kv":
                    s = u % self.slots
                    if u >= self.slots and self.mistake != "no wait for a slot":
                        yield self.kv_empty[s], u // self.slots - 1
                    self.unread(("slot", s))
                    self.slot[s][w] = (seg, i, kind)
                    yield self.kv_full[s].arrive
                    u += 1
        yield from self.unit(len(self.units))

    def scores(self, t, s, seg, i):
        def run():
            self.expect(self.slot[s], [(seg, i, "k")] * 8, f"slot {s}")
            self.expect(self.q[t], [seg] * 4, f"q {t}")
            if i:
                self.expect(self.o[t], (seg, i - 1), f"weights {t} under new scores have met V")
            self.s[t] = (seg, i)
        self.queue += [((("slot", s), ("q", t)), run), ((), self.s_full[t].arrive)]

    def issue(self):
        u, tiles, units = 0, [0, 0], [0, 0]
        commit = lambda b: self.queue.append(((), b.arrive))  # noqa: E731
        full = lambda k: (self.kv_full[k % self.slots], k // self.slots)  # noqa: E731
        for seg, c in enumerate(self.units):
            yield from self.unit(seg)
            n = max(c)
            if not n:
                continue
            yield full(u)
            for t in range(2):
                if c[t]:
                    if self.mistake != "no wait for q":
                        yield self.q_full[t], units[t]
                    units[t] += 1
                    self.scores(t, u % self.slots, seg, 0)
            commit(self.kv_empty[u % self.slots])
            u += 1
            for i in range(n):
                v, u = u, u + 1
                yield full(v)
                if i + 1 < n:
                    yield full(u)
                for t in range(2):
                    if i >= c[t]:
                        continue
                    for h in range(2):
                        if self.mistake == "one barrier for both halves":
                            yield self.p_full[2 * t], 2 * tiles[t] + h
                        elif self.mistake != "no wait for weights":
                            yield self.p_full[2 * t + h], tiles[t]

                        def run(t=t, i=i, h=h, seg=seg, s=v % self.slots):
                            self.expect(self.slot[s], [(seg, i, "v")] * 8, f"slot {s}")
                            self.expect(self.p[2 * t + h], [(seg, i)] * 4, f"weights {t}")
                            if h:
                                self.o[t] = (seg, i)
                            elif i:
                                self.expect(self.o[t], (seg, i - 1), f"O {t}")
                        self.queue.append(((("slot", v % self.slots),), run))
                    tiles[t] += 1
                    if i + 1 < c[t]:
                        self.scores(t, u % self.slots, seg, i + 1)
                    else:
                        commit(self.o_full[t])
                commit(self.kv_empty[v % self.slots])
                if i + 1 < n:
                    commit(self.kv_empty[u % self.slots])
                    u += 1
        yield from self.unit(len(self.units))

    def run(self):
        roles = [self.softmax(t, w) for t in range(2) for w in range(4)]
        roles += [self.convert(w) for w in range(8)] + [self.issue(), self.planner()]
        speed = [self.rng.choice([0.05, 0.3, 1.0]) for _ in roles] + [self.rng.choice([0.05, 0.3, 1.0])]
        at = [next(r, StopIteration) for r in roles]
        idle = 0
        while any(a is not StopIteration for a in at) or self.queue:
            k = self.rng.randrange(len(roles) + 1)
            idle += 1
            if idle > 40000:
                raise Fault("no progress")
            if self.rng.random() > speed[k]:
                continue
            if k == len(roles):
                if self.queue:
                    self.queue.pop(0)[1]()
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
    kinds = [(1, 1), (1, 2), (0, 1), (0, 0), (3, 3), (4, 5), (2, 0), (9, 10), (1, 0), (6, 7)]
    return [rng.choice(kinds) for _ in range(rng.randint(1, 9))]


@pytest.mark.parametrize("slots", [5, 8])
def test_protocol(slots):
    rng = random.Random(slots)
    for seed in range(100):
        Model(units_of(rng), slots, seed).run()


@pytest.mark.parametrize("mistake", ["no wait for the readers of a plan", "no wait for q",
                                     "one barrier for both halves", "no wait for the output",
                                     "no wait for a slot", "no wait for weights"])
def test_planted_protocol_mistakes(mistake):
    rng, caught = random.Random(1), 0
    for seed in range(60):
        try:
            Model(units_of(rng), 8, seed, mistake).run()
        except Fault:
            caught += 1
    assert caught > 0
