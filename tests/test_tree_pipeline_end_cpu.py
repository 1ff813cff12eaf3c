"""The barrier protocol of the tree attention's pipelines up to the CTA's end, for each
form that is built (its rings' lengths and query tiles read from the kernel's source).

As in test_tree_pipeline_cpu.py, but a commit arrives at any time after the MMAs that its
thread issued before it, in no order with that thread's other commits, and the CTA leaves
when its last thread has ended: an arrival or a copy that lands after that lands in memory
that may be another CTA's. So the last phase of every barrier that a commit arrives on has
to have been waited for by a thread that has seen the phase before it (a wait by parity
passes two phases too early as well)."""

import os
import random
import re

import pytest

import paged_kv_cache_345_b200 as pa
from test_tree_pipeline_cpu import Bar, Broken

SOURCE = os.path.join(os.path.dirname(pa.__file__), "csrc", "pa_tree.cu")


def built_forms():
    """{(head_dim, query tiles): (K tiles, V tiles) in flight}"""
    text = open(SOURCE).read()
    rings = []
    for name in ("kNK", "kNV"):
        m = re.search(name + r" = QT == 1 \? \(D == 128 \? (\d+) : (\d+)\) : \(D == 128 \? (\d+) : (\d+)\);", text)
        rings.append([int(x) for x in m.groups()])
    keys = [(128, 1), (64, 1), (128, 2), (64, 2)]
    return {k: (a, b) for k, a, b in zip(keys, *rings)}


FORMS = built_forms()


def simulate(seed, runs, form, end="each issuer"):
    """`end`: who waits for the last "empty" phases. "each issuer": the issuer that commits
    them; "scores": the scores' issuer for V's too; "nobody"."""
    nx = form[1]
    nk, nv = FORMS[form]
    n = nk + nv
    rng = random.Random(seed)
    full, empty = [Bar() for _ in range(n)], [Bar(nx) for _ in range(n)]
    q_full, q_empty = Bar(), Bar(nx)
    s_full, p_full, o_done = ([[Bar(), Bar()] for _ in range(nx)] for _ in range(3))
    buffers, writing = [[None, None] for _ in range(nx)], [0] * nx
    held, readers, q_held, q_readers = [None] * n, [0] * n, [None], [0]
    copies, mmas, running, commits = [], [], [None], []
    by = {}      # per issuer: MMAs that it issued, those that are done
    clock = [0]

    def place(kind, i):
        return (i % nk, (i // nk) & 1) if kind == "K" else (nk + i % nv, (i // nv) & 1)

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
        i = 0
        for r, tiles in enumerate(runs):
            if kind == "K":
                while not q_empty.done((r & 1) ^ 1):
                    yield
                q_full.arrive(1)
                yield
                copy(q_held, 0, r, q_readers, q_full)
            for _ in range(tiles):
                st, ph = place(kind, i)
                while not empty[st].done(ph ^ 1):
                    yield
                full[st].arrive(1)
                yield
                copy(held, st, (kind, i), readers, full[st])
                yield
                i += 1

    def issue(who, step):
        by.setdefault(who, [0, 0])[0] += 1
        mmas.append((who, *step))

    def commit(who, bar):  # lands once what `who` has issued so far is done, some of them late
        late = rng.randint(0, 2000) if rng.random() < 0.2 else 0
        commits.append((who, by.get(who, [0, 0])[0], bar, clock[0] + late))

    def scores(who, x, i, r):
        while i >= 2 and not o_done[x][i & 1].done(((i - 2) >> 1) & 1):
            yield
        st, ph = place("K", i)
        while not full[st].done(ph):
            yield
        issue(who, (st, ("K", i), r, x))
        yield
        for bar in (s_full[x][i & 1], empty[st]):
            commit(who, bar)
            yield

    def outputs(who, x, i):
        st, ph = place("V", i)
        while not full[st].done(ph):
            yield
        while not p_full[x][i & 1].done((i >> 1) & 1):
            yield
        issue(who, (st, ("V", i), None, x))
        yield
        for bar in (o_done[x][i & 1], empty[st]):
            commit(who, bar)
            yield

    def last_phases(kinds, total, runs_seen):
        left = []  # (a lane each: all at once)
        for kind in kinds:
            first, size = (0, nk) if kind == "K" else (nk, nv)
            if kind == "Q":
                left.append((q_empty, (runs_seen - 1) & 1))
            else:
                left += [(empty[first + at], ((total - at + size - 1) // size - 1) & 1) for at in range(min(size, total))]
        while left:
            left = [w for w in left if not w[0].done(w[1])]
            yield

    def issuer(x, which):
        who, i = f"{which} {x}", 0
        for r, tiles in enumerate(runs):
            while "S" in which and not q_full.done(r & 1):
                yield
            for t in range(tiles + (2 if which == "S PV" else 0)):
                if which == "S PV":
                    if t >= 2:
                        yield from outputs(who, x, i + t - 2)
                    if t < tiles:
                        yield from scores(who, x, i + t, r)
                else:
                    yield from (scores(who, x, i + t, r) if which == "S" else outputs(who, x, i + t))
                if "S" in which and t == tiles - 1:
                    commit(who, q_empty)
                    yield
            i += tiles
        waits = {"each issuer": {"S": "KQ", "PV": "V", "S PV": "KVQ" if x == 0 else ""},
                 "scores": {"S": "KVQ", "PV": "", "S PV": "KVQ" if x == 0 else ""},
                 "nobody": {}}[end].get(which, "")
        yield from last_phases(waits, i, len(runs))

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
                if t == tiles - 1:  # (a ragged last tile: V's rows past the context become zeros)
                    st, ph = place("V", i)
                    while not full[st].done(ph):
                        yield
                    if held[st] != ("V", i):
                        raise Broken("zeros into another tile")
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
        for which in ("S", "PV") if nx == 1 else ("S PV",):
            threads[f"{which} {x}"] = issuer(x, which)
        threads[f"softmax {x}"] = softmax(x)
    slow = dict.fromkeys([*threads, "copies", "pipe", "commits"], 1)
    for step in range(300_000):
        clock[0] = step
        if not threads:
            if mmas or running[0] is not None or copies or commits:
                raise Broken("left with something still to arrive")
            return
        if step % 500 == 0:
            slow = {k: rng.choice([1, 1, 3, 10, 30, 300]) for k in slow}
        name = rng.choice(list(slow))
        if rng.random() > 1 / slow[name]:
            continue
        if name == "copies":
            if copies:
                copies.pop(rng.randrange(len(copies)))()
        elif name == "commits":
            ready = [c for c in commits if by.get(c[0], [0, 0])[1] >= c[1] and c[3] <= step]
            if ready:
                c = rng.choice(ready)
                commits.remove(c)
                c[2].arrive()
        elif name == "pipe":
            if running[0] is not None:
                who, st, (_, i), r, x = running[0]
                readers[st] -= 1
                q_readers[0] -= r is not None
                by[who][1] += 1
                if r is not None:
                    buffers[x][i & 1] = ("S", i)
                else:
                    writing[x] = 0
                running[0] = None
            elif mmas:
                _, st, want, r, x = running[0] = mmas.pop(0)
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
    rng = random.Random(seed + 4242)
    return [rng.randint(1, 15) for _ in range(rng.randint(1, 5))]


def broken(form, end, seeds):
    count = 0
    for seed in range(seeds):
        try:
            simulate(seed, runs_of(seed), form, end)
        except Broken:
            count += 1
    return count


def end_in_source():
    """Who waits for V's last "empty" phases where scores and outputs have an issuer each:
    the kernel says in one place which of a warp's lanes (one a place in the rings) wait."""
    return "each issuer" if re.search(r"QT == 2 \? warp == 2 : \(lane < NK\) == \(warp == 2\)", open(SOURCE).read()) else "scores"


@pytest.mark.parametrize("block", range(4))
@pytest.mark.parametrize("form", FORMS)
def test_protocol_holds_to_the_end_under_any_delay(form, block):
    for seed in range(50 * block, 50 * block + 50):
        simulate(seed, runs_of(seed), form, end_in_source())


@pytest.mark.parametrize("form", FORMS)
def test_the_model_sees_a_cta_that_leaves_too_early(form):
    assert broken(form, "nobody", 12) > 0


def test_the_model_sees_a_wait_of_another_warp_that_passes_two_phases_early():
    assert broken((128, 1), "scores", 200) > 0
