"""The barrier protocol of the tree attention's pipeline, simulated: two producers, two
MMA issuers, the softmax, unordered copies and the in-order queue of the tensor pipe,
each delayed at will. Every tile has to be read whole and before it is overwritten, no
barrier may get an arrival that its phase does not expect, and nothing may wait for
good. One ring that both producers fill in turns, instead of one each, breaks all of
this when a commit comes late: the model has to see that."""

import random

import pytest

NK, NV = 2, 3


class Broken(Exception):
    pass


class Bar:
    """An mbarrier: arrivals and pending copies of a phase; waits name a phase by parity."""

    def __init__(self):
        self.pending, self.copies, self.phase = 1, 0, 0

    def arrive(self, copies=0):
        if self.pending == 0:
            raise Broken("an arrival too many")
        self.pending -= 1
        self.copies += copies
        self._turn()

    def landed(self):
        self.copies -= 1
        self._turn()

    def _turn(self):
        if self.pending == 0 and self.copies == 0:
            self.phase += 1
            self.pending = 1

    def done(self, parity):
        return (self.phase & 1) != parity


def simulate(seed, runs, one_ring=False):
    rng = random.Random(seed)
    n = NK + NV
    full, empty = [Bar() for _ in range(n)], [Bar() for _ in range(n)]
    q_full, q_empty = Bar(), Bar()
    s_full, p_full, o_done = ([Bar(), Bar()] for _ in range(3))
    held, readers, q_held, q_readers = [None] * n, [0] * n, [None], [0]
    copies, queue, now = [], [], [None]

    def place(kind, i):
        if one_ring:
            at = 2 * i + (kind == "V")
            return at % n, (at // n) & 1
        return (i % NK, (i // NK) & 1) if kind == "K" else (NK + i % NV, (i // NV) & 1)

    def copy(cell, at, value, busy, bar):
        if busy[at]:
            raise Broken("overwritten while read")
        cell[at] = None

        def land():
            if busy[at]:
                raise Broken("landed while read")
            cell[at] = value
            bar.landed()
        copies.append(land)

    def producer(kind):
        i, q_phase = 0, 0
        for r, tiles in enumerate(runs):
            if kind == "K":
                while not q_empty.done(q_phase ^ 1):
                    yield
                q_full.arrive(1)
                yield
                copy(q_held, 0, r, q_readers, q_full)
                q_phase ^= 1
            for _ in range(tiles):
                st, ph = place(kind, i)
                while not empty[st].done(ph ^ 1):
                    yield
                full[st].arrive(1)
                yield
                copy(held, st, (kind, i), readers, full[st])
                yield
                i += 1

    def scores():
        i, q_phase = 0, 0
        for r, tiles in enumerate(runs):
            while not q_full.done(q_phase):
                yield
            q_phase ^= 1
            for t in range(tiles):
                while i >= 2 and not o_done[i & 1].done(((i - 2) >> 1) & 1):
                    yield
                st, ph = place("K", i)
                while not full[st].done(ph):
                    yield
                for step in [("mma", st, ("K", i), r), s_full[i & 1], empty[st]] + [q_empty] * (t == tiles - 1):
                    queue.append(step)
                    yield
                i += 1

    def outputs():
        i = 0
        for _ in range(sum(runs)):
            st, ph = place("V", i)
            while not full[st].done(ph):
                yield
            while not p_full[i & 1].done((i >> 1) & 1):
                yield
            for step in (("mma", st, ("V", i), None), o_done[i & 1], empty[st]):
                queue.append(step)
                yield
            i += 1

    def softmax():
        i = 0
        for tiles in runs:
            for t in range(tiles):
                while not s_full[i & 1].done((i >> 1) & 1):
                    yield
                yield
                rescale = t > 0 and rng.random() < 0.3
                while rescale and not o_done[(i - 1) & 1].done(((i - 1) >> 1) & 1):
                    yield
                p_full[i & 1].arrive()
                yield
                while t > 0 and not rescale and not o_done[(i - 1) & 1].done(((i - 1) >> 1) & 1):
                    yield
                i += 1
            while not o_done[(i - 1) & 1].done(((i - 1) >> 1) & 1):
                yield

    threads = {"K": producer("K"), "V": producer("V"), "S": scores(), "PV": outputs(), "softmax": softmax()}
    slow = dict.fromkeys([*threads, "copies", "queue"], 1)
    for step in range(150_000):
        if not threads and not queue and now[0] is None:
            return
        if step % 500 == 0:
            slow = {k: rng.choice([1, 1, 3, 10, 30, 300]) for k in slow}
        name = rng.choice(list(slow))
        if rng.random() > 1 / slow[name]:
            continue
        if name == "copies":
            if copies:
                copies.pop(rng.randrange(len(copies)))()
        elif name == "queue":
            if now[0] is not None:
                _, st, _, r = now[0]
                readers[st] -= 1
                q_readers[0] -= r is not None
                now[0] = None
            elif queue:
                step_ = queue.pop(0)
                if isinstance(step_, Bar):
                    step_.arrive()
                    continue
                _, st, want, r = now[0] = step_
                if held[st] != want or (r is not None and q_held[0] != r):
                    raise Broken("read something else")
                readers[st] += 1
                q_readers[0] += r is not None
        elif name in threads and next(threads[name], "end") == "end":
            del threads[name]
    raise Broken("waits for good")


def runs_of(seed):
    rng = random.Random(seed + 999)
    return [rng.randint(1, 9) for _ in range(rng.randint(1, 6))]


@pytest.mark.parametrize("block", range(6))
def test_protocol_holds_under_any_delay(block):
    for seed in range(10 * block, 10 * block + 10):
        simulate(seed, runs_of(seed))


def test_the_model_sees_what_one_ring_breaks():
    broken = 0
    for seed in range(30):
        try:
            simulate(seed, runs_of(seed), one_ring=True)
        except Broken:
            broken += 1
    assert broken > 0
