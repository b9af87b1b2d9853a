"""The d_weight pass's schedule, checked on the host: units follow one another without rounds of their own.

The agents and barriers are those of test_bwd_schedule_cpu; what differs is the order of the work.  A group's
supertiles are numbered through all of its units; step s forms tiles s c .. s c + c - 1 (one per pair) and accumulates those of
step s - 1, which may end one unit and begin the next.  Where a unit ends inside a step, the pair accumulates up to its
end, then computes its own next logit tile, then goes on with the next unit, so that the accumulator is stored under the
logit tile; the epilogue stores that accumulator before it forms the step's tile.  All other accumulators are stored after
the step's tile.  The model replays that order under random interleavings and checks that every run finishes, that no
barrier runs two phases past a waiter, that no slot is read early or overwritten, and that every unit's tiles are
accumulated in order, from its first to its last, with its predecessor's accumulator stored before."""
import random

import pytest

from test_bwd_schedule_cpu import G_SLOTS, NST, Bar, Violation, _all_bars, _wait


def steps(nys, c):
    """Per step: own tiles (k, y) by pair, accumulated tiles of the step before, and how many of these come first."""
    tiles = [(k, y) for k, ny in enumerate(nys) for y in range(ny)]
    out = []
    n = -(-len(tiles) // c)
    for s in range(n + 1):
        own = [tiles[s * c + j] if s * c + j < len(tiles) else None for j in range(c)]
        acc = tiles[(s - 1) * c:s * c] if s > 0 else []
        ends = [i for i, (k, y) in enumerate(acc) if y == nys[k] - 1]
        mid = bool(ends) and ends[0] + 1 < len(acc)
        out.append((own, acc, ends[0] + 1 if mid else 0))
    return out


def agents(j, c, nys, nk, B, S):
    plan = steps(nys, c)

    def until(cond):
        while not cond():
            yield

    def producer():
        k_acq, cnt = 0, [0] * c

        def acquire():
            nonlocal k_acq
            s, u = k_acq % NST, k_acq // NST
            yield from _wait(B[j]["empty"][s], u - 1)
            B[j]["full"][s].arrive()
            k_acq += 1

        def load(wr):
            g, u = cnt[wr] % G_SLOTS, cnt[wr] // G_SLOTS
            yield from until(lambda: S["seen"][j][wr] >= cnt[wr] + 1)
            for _ in range(4):
                yield from acquire()
                if S["fills"][wr][g] != u + 1:
                    raise Violation("a slot read before it was written, or after it was overwritten")
            S["loaded"][j][wr][g] += 1
            cnt[wr] += 1
        for own, acc, before in plan:
            for wr in range(before):
                yield from load(wr)
            if own[j] is not None:
                for _ in range(nk):
                    yield from acquire()
            for wr in range(before, len(acc)):
                yield from load(wr)

    def poller():
        cnt = [0] * c
        for _, acc, _ in plan:
            for wr in range(len(acc)):
                g, u = cnt[wr] % G_SLOTS, cnt[wr] // G_SLOTS
                yield from until(lambda: S["ready"][wr][g] >= u + 1)
                S["seen"][j][wr] = cnt[wr] + 1
                cnt[wr] += 1

    def mma():
        k_con, m_all, cnt = 0, 0, [0] * c

        def consume():
            nonlocal k_con
            yield from _wait(B[j]["full"][k_con % NST], k_con // NST)
            k_con += 1
            return (k_con - 1) % NST

        def accumulate(wr, k, y):
            if y == 0:
                yield from _wait(B[j]["accempty"], k - 1)
                if S["stored"][j] != k:
                    raise Violation("an accumulator begun before the last one was stored")
            if S["acc"][j] != (k, y):
                raise Violation("tiles out of order")
            g = cnt[wr] % G_SLOTS
            for q in range(4):
                s = yield from consume()
                if q == 3:
                    S["free"][wr][g] += 1
                B[j]["empty"][s].arrive()
            cnt[wr] += 1
            last = y == nys[k] - 1
            S["acc"][j] = (k + 1, 0) if last else (k, y + 1)
            if last:
                B[j]["accfull"].arrive()
        for own, acc, before in plan:
            for wr in range(before):
                yield from accumulate(wr, *acc[wr])
            if own[j] is not None:
                yield from _wait(B[j]["tempty"], m_all - 1)
                for _ in range(nk):
                    s = yield from consume()
                    B[j]["empty"][s].arrive()
                B[j]["tfull"].arrive()
                m_all += 1
            for wr in range(before, len(acc)):
                yield from accumulate(wr, *acc[wr])

    def epilogue():
        m_all = 0

        def store(k):
            yield from _wait(B[j]["accfull"], k)
            S["stored"][j] += 1
            B[j]["accempty"].arrive()
        for own, acc, before in plan:
            ends = [k for k, y in acc if y == nys[k] - 1]
            if before:
                yield from store(ends.pop(0))
            if own[j] is not None:
                g, u = m_all % G_SLOTS, m_all // G_SLOTS
                yield from until(lambda: S["free"][j][g] >= c * u)
                yield from _wait(B[j]["tfull"], m_all)
                for q in range(c):
                    if S["loaded"][q][j][g] < u:
                        raise Violation("a slot overwritten before it was read")
                S["fills"][j][g] += 1
                B[j]["tempty"].arrive()
                S["ready"][j][g] += 1
                m_all += 1
            for k in ends:
                yield from store(k)
    return [producer(), poller(), mma(), epilogue()]


def run(c, nys, nk, seed):
    B = [{"full": [Bar(1) for _ in range(NST)], "empty": [Bar(1) for _ in range(NST)], "tfull": Bar(1), "tempty": Bar(1),
          "accfull": Bar(1), "accempty": Bar(1)} for _ in range(c)]
    S = {"ready": [[0] * G_SLOTS for _ in range(c)], "free": [[0] * G_SLOTS for _ in range(c)],
         "fills": [[0] * G_SLOTS for _ in range(c)], "seen": [[0] * c for _ in range(c)],
         "loaded": [[[0] * G_SLOTS for _ in range(c)] for _ in range(c)], "stored": [0] * c, "acc": [(0, 0)] * c}
    live = [a for j in range(c) for a in agents(j, c, nys, nk, B, S)]
    rng, stalled = random.Random(seed), 0

    def state():
        return [(b.phases, b.count) for cta in B for b in _all_bars(cta)], str(S)
    while live:
        a, before = rng.choice(live), state()
        try:
            next(a)
            stalled = 0 if state() != before else stalled + 1
        except StopIteration:
            live.remove(a)
            stalled = 0
        if stalled > 400 * 4 * c + 1000:
            raise AssertionError("deadlock")
    assert S["stored"] == [len(nys)] * c and S["acc"] == [(len(nys), 0)] * c


@pytest.mark.parametrize("c", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("ny,units", [(1, 7), (2, 5), (3, 4), (4, 4), (5, 3), (9, 3), (16, 2)])
def test_units_in_a_row(c, ny, units):
    for seed in range(3):
        run(c, [ny] * units, nk=3, seed=seed)


@pytest.mark.parametrize("ny,units", [(24, 2), (1, 20), (9, 4)])
def test_groups_of_16(ny, units):
    run(16, [ny] * units, nk=2, seed=1)


def test_whole_rounds_are_the_old_order():
    """Units of whole rounds: no accumulator is stored before the step's tile."""
    assert all(before == 0 for c in (1, 2, 4) for _, _, before in steps([2 * c] * 3, c))

