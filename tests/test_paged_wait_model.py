"""A model of how the decode kernel's teams use their rings of stages, and of
how they give up when a wait runs out: what is armed, what is on the way, and
who leaves when, under every order of steps that a seeded scheduler tries.  The
rules are those of mbarriers: a phase takes as many arrivals as the team has
warps, and completes when they and their copies are in; an arrival on a phase
that has had all of its arrivals is an error."""

import random

import pytest


class Misuse(Exception):
    pass


class Phase:
    def __init__(self, warps):
        self.warps = self.missing = warps
        self.copies = self.index = 0

    def arrive(self, copies):
        if self.missing == 0:
            raise Misuse("armed while its copies are on the way")
        self.missing -= 1
        self.copies += copies
        self.advance()

    def land(self):
        self.copies -= 1
        self.advance()

    def advance(self):
        if self.missing == 0 and self.copies == 0:
            self.index, self.missing = self.index + 1, self.warps

    def done(self, parity):
        return self.index & 1 != parity


def play(seed, carries_on=False):
    """One team at work; True if it gave up.  `carries_on` plants the mistake
    of going on after a wait that ran out."""
    rng = random.Random(seed)
    warps, stages, blocks = rng.choice([1, 2, 4]), rng.choice([2, 3, 4, 8]), rng.randint(0, 30)
    runs_out = rng.choice([0, 0.02, 0.2, 0.9])
    ring, on_the_way = [Phase(warps) for _ in range(stages)], []
    flags, abort, arrived, left = [False] * stages, [False], [0] * warps, []

    def warp(w):
        fifo, issued = [None] * stages, 0

        def issue(stage):
            nonlocal issued
            fifo[stage] = issued < blocks
            if not fifo[stage]:
                return
            issued += 1
            copies = (2 if w == 0 else 0) + rng.randint(0, 1)      # K and V, query rows
            ring[stage].arrive(copies)
            on_the_way.extend([stage] * copies)

        for i in range(stages - 1):
            issue(i)
            yield
        stage, fill, parity = 0, stages - 1, 0
        while True:
            arrived[w] += 1                       # the team's barrier
            step = arrived[w]
            while min(arrived) < step:
                yield
            yield
            if not fifo[stage]:
                break
            while not ring[stage].done(parity):
                if abort[0] or rng.random() < runs_out:
                    abort[0] = flags[stage] = True
                    break
                yield
            yield
            if flags[fill] and not carries_on:
                break
            issue(fill)
            yield
            fill, stage = (fill + 1) % stages, stage + 1
            if stage == stages:
                stage, parity = 0, parity ^ 1
        gave_up = flags[fill]
        left.append((step, gave_up))
        if gave_up and not carries_on:
            stage -= 1
            if stage < 0:
                stage, parity = stages - 1, parity ^ 1
            for _ in range(stages):
                if not fifo[stage]:
                    break
                while not ring[stage].done(parity):
                    yield
                stage += 1
                if stage == stages:
                    stage, parity = 0, parity ^ 1

    team = {w: warp(w) for w in range(warps)}
    for _ in range(10 ** 6):
        if not team:
            break
        if on_the_way and rng.random() < 0.4:
            ring[on_the_way.pop(rng.randrange(len(on_the_way)))].land()
            continue
        w = rng.choice(list(team))
        try:
            next(team[w])
        except StopIteration:
            del team[w]
    assert not team, "stuck"
    assert len(set(left)) == 1, "warps left at different steps, or for different reasons"
    if on_the_way:
        raise Misuse("left while copies are on the way")
    return left[0][1]


def test_giving_up_leaves_nothing_behind():
    gave_up = [play(seed) for seed in range(3000)]
    assert 300 < sum(gave_up) < 2700


def test_the_model_sees_a_team_that_carries_on():
    with pytest.raises(Misuse):
        for seed in range(200):
            play(seed, carries_on=True)
