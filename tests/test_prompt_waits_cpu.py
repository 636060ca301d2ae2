"""The prompt attention kernel's bounded waits on its model (test_prompt_protocol_cpu): a wait gives
up after a limit, which ends its role and, through the abort flag, all others; only the waits for
a unit to be written down or read go on for as long as tiles are converted.  Units that take far
longer than the limit are worked through, and when a role stops the others all end."""
import random

import pytest

from test_prompt_protocol_cpu import Fault, Model

LIMIT = 6000   # steps that a wait lasts; a tile takes about 300 to 1000


class Timed(Model):
    """Waits with a limit.  `dies`: (role, after so many of its steps).  Mistakes: "limit alone", the
    waits for a unit have no more than the limit; "no look at the tiles", they have none."""

    def ticks(self):
        return sum(b.phases for b in self.kv_full)

    def run(self, dies=None):
        roles = [self.softmax(t, w) for t in range(2) for w in range(4)]
        roles += [self.convert(w) for w in range(8)] + [self.issue(), self.planner()]
        at = [next(r) for r in roles]
        n, now, abort = len(roles), 0, False
        since, seen, steps = [0] * n, [None] * n, [0] * n
        gone = set()
        while any(a is not StopIteration for k, a in enumerate(at) if k not in gone) or self.queue:
            now += 1
            if now > 3_000_000:
                raise Fault("roles that never end")
            k = self.rng.randrange(n + 1)
            if k == n:
                if self.queue:
                    self.queue.pop(0)[1]()
                continue
            a = at[k]
            if k in gone or a is StopIteration:
                continue
            if isinstance(a, tuple) and not a[0].passed(a[1]):
                if abort:
                    at[k] = StopIteration
                elif now - since[k] > LIMIT:
                    working = a[0].name.startswith("u_") and self.mistake != "limit alone"
                    if working and (self.ticks() != seen[k] or self.mistake == "no look at the tiles"):
                        since[k], seen[k] = now, self.ticks()
                    else:
                        at[k], abort = StopIteration, True
                continue
            if a is not None and not isinstance(a, tuple):
                a()
            steps[k] += 1
            if dies and dies[0] == k and steps[k] > dies[1]:
                gone.add(k)
                continue
            at[k] = next(roles[k], StopIteration)
            since[k], seen[k] = now, None
        return abort


# the second row tile has no rows: its warps wait for the first's, unit after unit
LONG = [(40, 0)] * 7


def test_units_longer_than_the_limit():
    for seed in range(2):
        model = Timed(LONG, 5, seed)
        assert not model.run()
        assert model.stored == {(s, t, w) for s in range(len(LONG)) for t in range(2) for w in range(4)}


def test_the_limit_alone_would_give_up_such_units():
    assert Timed(LONG, 5, 0, "limit alone").run()


@pytest.mark.parametrize("role", [0, 5, 8, 15, 16, 17])   # softmax, converting, issuing, planning
def test_all_roles_end_when_one_stops(role):
    rng, given_up = random.Random(role), 0
    for seed in range(4):
        units = [(rng.randint(1, 6), rng.randint(0, 6)) for _ in range(7)]
        given_up += Timed(units, 5, seed).run(dies=(role, rng.randint(1, 25)))
    assert given_up > 0


def test_waits_without_a_look_at_the_tiles_would_not_end():
    with pytest.raises(Fault, match="never end"):
        Timed([(3, 0)] * 7, 5, 0, "no look at the tiles").run(dies=(17, 3))
