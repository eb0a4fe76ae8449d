"""A model of how the warps of a team of the decode kernel walk their range of
the work.  They meet at a barrier for every block, so they have to agree on the
number of blocks whatever the lengths do meanwhile: lengths that change during a
call give wrong numbers, but may not leave a warp waiting for others that are
gone."""

import random

import pytest


class Stuck(Exception):
    pass


def play(seed, each_reads=False):
    """Steps of one team; `each_reads` plants the mistake of warps that read the
    lengths for themselves."""
    rng = random.Random(seed)
    warps, batch = rng.choice([2, 4]), rng.randint(1, 8)
    lens = [rng.randint(1, 5) for _ in range(batch)]
    common, at, gone, steps = [None, None], [0] * warps, [], [0] * warps

    def warp(w):
        entered = 0

        def meet():
            at[w] += 1
            me = at[w]
            while any(x < me for x in at):
                yield

        left, b, off, units = rng_range, 0, 0, 0
        while left > 0:
            if off >= units:
                if entered and b + 1 >= batch:
                    break
                b += entered > 0
                if each_reads:
                    units = lens[b]
                else:
                    place = entered & 1
                    if w == 0:
                        common[place] = lens[b]
                    yield from meet()
                    yield
                    units = common[place]
                entered, off = entered + 1, 0
            yield
            off, left = off + 1, left - 1
            steps[w] += 1
            yield from meet()              # the block's barrier
        gone.append(w)

    rng_range = rng.randint(1, 30)
    team = {w: warp(w) for w in range(warps)}
    for _ in range(20000):
        if not team:
            return steps
        if rng.random() < 0.2:
            lens[rng.randrange(batch)] = rng.randint(1, 5)
            continue
        w = rng.choice(list(team))
        try:
            next(team[w])
        except StopIteration:
            del team[w]
    raise Stuck(f"{gone} are gone, the others wait")


def test_warps_that_share_what_one_reads_stay_together():
    for seed in range(2000):
        assert len(set(play(seed))) == 1


def test_warps_that_read_for_themselves_part():
    with pytest.raises(Stuck):
        for seed in range(200):
            play(seed, each_reads=True)
