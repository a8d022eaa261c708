"""The barriers of the tensor-core attention kernel, played through on the CPU.

The kernel's roles (producers, converters, the MMA thread, softmax warps) wait for phases of shared-memory
barriers by parity alone. Here each role is a generator that yields the phase it waits for and arrives where
the kernel does, at random speeds; a barrier that is waited for by parity before its phase is over, one that
gets more arrivals than its count, and a stop of all roles are mistakes. Two earlier forms of the protocol are
planted to show that they are found.
"""
import random

import pytest


class Mistake(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        if self.left == 0:
            raise Mistake("more arrivals than the phase takes")
        self.left -= 1
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.count

    def by_parity(self, phase):
        return self.phase & 1 != phase & 1


class Stage(Barrier):
    """A raw stage's `full`: one arrival, and the phase ends when the copies land, some time after it."""

    def __init__(self):
        super().__init__(1)
        self.booked = False

    def arrive(self):
        if self.booked:
            raise Mistake("a stage booked twice in one phase")
        self.booked = True

    def land(self):
        if self.booked:
            self.booked = False
            self.phase += 1


def play(seed, row_tiles, tiles, stages, jobs, producers=None, end="own barrier"):
    r = random.Random(seed)
    soft = 4 * row_tiles
    full, empty = [Stage() for _ in range(stages)], [Barrier(4) for _ in range(stages)]
    k_full, k_free, q_ready, job_done = Barrier(4), Barrier(1), Barrier(soft), Barrier(1)
    v_full, v_free, o_done = ([Barrier(n) for _ in range(2)] for n in (4, 1, 1))
    s_full, p_ready = ([Barrier(n) for _ in range(4)] for n in (1, 4))
    total, events = tiles * jobs, r.random()
    warps = min(3, stages // 2) if producers is None else producers

    def producer(mine):
        for t in range(mine, total, warps):
            for u in (2 * t, 2 * t + 1):
                if u // stages:
                    yield empty[u % stages], u // stages - 1
            for u in (2 * t, 2 * t + 1):
                full[u % stages].arrive()

    def converter():
        for t in range(total):
            for which in range(2):
                u = 2 * t + which
                if which == 0 and t >= 1:
                    yield k_free, t - 1
                if which == 1 and t >= 2:
                    yield v_free[t & 1], (t >> 1) - 1
                yield full[u % stages], u // stages
                empty[u % stages].arrive()
                (k_full if which == 0 else v_full[t & 1]).arrive()

    def mma():
        t = 0

        def scores(rt, h):
            s_full[2 * rt + h].arrive()
            if rt == row_tiles - 1 and h == 1:
                k_free.arrive()

        for job in range(jobs):
            yield q_ready, job
            yield k_full, t
            steps = [(i % row_tiles, i // row_tiles) for i in range(2 * row_tiles)]
            for s in steps:
                scores(*s)
            for tile in range(tiles):
                for i, (rt, h) in enumerate(steps):
                    yield p_ready[2 * rt + h], t
                    if i == 0:
                        yield v_full[t & 1], t >> 1
                    o_done[rt].arrive()
                    if rt == row_tiles - 1 and h == 1:
                        v_free[t & 1].arrive()
                    if tile + 1 < tiles:
                        if i == 0:
                            yield k_full, t + 1
                        scores(rt, h)
                t += 1
            job_done.arrive()

    def softmax(rt):
        t = 0
        for job in range(jobs):
            q_ready.arrive()
            for tile in range(tiles):
                for h in range(2):
                    yield s_full[2 * rt + h], t
                    if (tile or h) and r.random() < events:       # the reference moves: the sums are rescaled
                        yield o_done[rt], 2 * t + h - 1
                    p_ready[2 * rt + h].arrive()
                t += 1
            if end == "own barrier":
                yield job_done, job
            else:                                                  # the last two phases of one barrier
                yield o_done[rt], 2 * t - 2
                yield o_done[rt], 2 * t - 1

    roles = [mma()] + [producer(i) for i in range(warps)] + [converter() for _ in range(4)] + [softmax(i // 4) for i in range(soft)]
    speed = {id(x): r.choice([0.05, 0.3, 1.0]) for x in roles}
    waits, alive = {id(x): None for x in roles}, list(roles)
    while alive:
        could = False
        for x in r.sample(alive, len(alive)):
            w = waits[id(x)]
            if w is not None and not w[0].by_parity(w[1]):
                continue
            could = True
            if r.random() > speed[id(x)]:
                continue
            if w is not None and w[0].phase <= w[1]:
                raise Mistake("a wait ended before its phase")
            try:
                waits[id(x)] = next(x)
            except StopIteration:
                alive.remove(x)
        for s in full:
            if s.booked:
                could = True
                if r.random() < 0.5:
                    s.land()
        if not could:
            raise Mistake("every role waits")


@pytest.mark.parametrize("row_tiles", [1, 2])
@pytest.mark.parametrize("stages", [2, 3, 4, 5, 8])
def test_protocol(row_tiles, stages):
    for seed in range(12):
        play(seed, row_tiles, [1, 2, 3, 7][seed % 4], stages, 1 + seed % 3)


def test_more_producers_than_the_ring_takes_are_found():
    with pytest.raises(Mistake):
        for seed in range(40):
            play(seed, 2, 9, 3, 1, producers=3)


def test_waiting_for_two_phases_of_one_barrier_is_found():
    with pytest.raises(Mistake):
        for seed in range(40):
            play(seed, 1, 5, 8, 2, end="two phases")
