"""The barrier protocol of the tree attention's pipeline, simulated: two producers, two
MMA issuers, the softmax, unordered copies and the in-order queue of the tensor pipe,
each delayed at will. Every tile has to be read whole and before it is overwritten, no
barrier may get an arrival that its phase does not expect, and nothing may wait for
good. One query tile has an issuer of scores and one of outputs; two have an issuer each,
of both, and share K, V and Q. One ring that both producers fill in turns, instead of one each, breaks all of
this when a commit comes late: the model has to see that."""

import random

import pytest

NK, NV = 2, 3


class Broken(Exception):
    pass


class Bar:
    """An mbarrier: arrivals and pending copies of a phase; waits name a phase by parity."""

    def __init__(self, count=1):
        self.count, self.pending, self.copies, self.phase = count, count, 0, 0

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
            self.pending = self.count

    def done(self, parity):
        return (self.phase & 1) != parity


def simulate(seed, runs, one_ring=False, nx=1):
    rng = random.Random(seed)
    n = NK + NV
    full, empty = [Bar() for _ in range(n)], [Bar(nx) for _ in range(n)]
    q_full, q_empty = Bar(), Bar(nx)
    s_full, p_full, o_done = ([[Bar(), Bar()] for _ in range(nx)] for _ in range(3))
    buffers, writing = [[None, None] for _ in range(nx)], [0] * nx      # scores or weights of a tile; outputs
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

    def scores(x, i, r):
        while i >= 2 and not o_done[x][i & 1].done(((i - 2) >> 1) & 1):
            yield
        st, ph = place("K", i)
        while not full[st].done(ph):
            yield
        for step in (("mma", st, ("K", i), r, x), s_full[x][i & 1], empty[st]):
            queue.append(step)
            yield

    def outputs(x, i):
        st, ph = place("V", i)
        while not full[st].done(ph):
            yield
        while not p_full[x][i & 1].done((i >> 1) & 1):
            yield
        for step in (("mma", st, ("V", i), None, x), o_done[x][i & 1], empty[st]):
            queue.append(step)
            yield

    def issuer(x, which):
        i = 0
        for r, tiles in enumerate(runs):
            while "S" in which and not q_full.done(r & 1):
                yield
            for t in range(tiles + (2 if which == "both S, PV" else 0)):
                if which == "both S, PV":
                    if t >= 2:
                        yield from outputs(x, i + t - 2)
                    if t < tiles:
                        yield from scores(x, i + t, r)
                else:
                    yield from (scores(x, i + t, r) if which == "S" else outputs(x, i + t))
                if "S" in which and t == tiles - 1:
                    queue.append(q_empty)
                    yield
            i += tiles

    def softmax(x):
        i = 0
        for tiles in runs:
            for t in range(tiles):
                while not s_full[x][i & 1].done((i >> 1) & 1):
                    yield
                if buffers[x][i & 1] != ("S", i):
                    raise Broken("other scores")
                yield
                rescale = t > 0 and rng.random() < 0.3
                while rescale and not o_done[x][(i - 1) & 1].done(((i - 1) >> 1) & 1):
                    yield
                if rescale and writing[x]:
                    raise Broken("outputs rescaled while written")
                buffers[x][i & 1] = ("P", i)
                p_full[x][i & 1].arrive()
                yield
                i += 1
            while tiles > 1 and not o_done[x][i & 1].done(((i - 2) >> 1) & 1):
                yield
            while not o_done[x][(i - 1) & 1].done(((i - 1) >> 1) & 1):
                yield
            if writing[x]:
                raise Broken("outputs read while written")

    threads = {"K": producer("K"), "V": producer("V")}
    for x in range(nx):
        threads |= {f"{which} {x}": issuer(x, which) for which in (("S", "PV") if nx == 1 else ("both S, PV",))}
        threads[f"softmax {x}"] = softmax(x)
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
                _, st, (_, i), r, x = now[0]
                readers[st] -= 1
                q_readers[0] -= r is not None
                if r is not None:
                    buffers[x][i & 1] = ("S", i)
                else:
                    writing[x] = 0
                now[0] = None
            elif queue:
                step_ = queue.pop(0)
                if isinstance(step_, Bar):
                    step_.arrive()
                    continue
                _, st, want, r, x = now[0] = step_
                if r is not None:
                    buffers[x][want[1] & 1] = None
                elif buffers[x][want[1] & 1] != ("P", want[1]):
                    raise Broken("other weights")
                else:
                    writing[x] = 1
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


@pytest.mark.parametrize("query_tiles", [1, 2])
@pytest.mark.parametrize("block", range(6))
def test_protocol_holds_under_any_delay(block, query_tiles):
    for seed in range(10 * block, 10 * block + 10):
        simulate(seed, runs_of(seed), nx=query_tiles)


def test_the_model_sees_what_one_ring_breaks():
    broken = 0
    for seed in range(30):
        try:
            simulate(seed, runs_of(seed), one_ring=True)
        except Broken:
            broken += 1
    assert broken > 0
