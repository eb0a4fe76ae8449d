"""A model of how fa_paged_extend's query loader gives up (CPU): two halves of rows, each
armed and filled when its readers have freed it, and what is left on the way when a wait
runs out between them.  The rules of mbarriers are those of the decode kernel's model."""

import os
import random
import re

import pytest

from test_paged_wait_model import Misuse, Phase
from varlen_flashattention_backward_gb300 import build as fb


def play(seed, counts_late=False):
    """One CTA at work; True if it gave up.  `counts_late` plants the mistake of counting
    the halves of a block when both are filled."""
    rng = random.Random(seed)
    items = [(rng.random() < 0.7, rng.random() < 0.7) for _ in range(rng.randint(0, 12))]
    runs_out = rng.choice([0, 0.02, 0.2, 0.9])
    query, frees, on_the_way, abort = [Phase(1), Phase(1)], [0, 0], [], [False]

    def loader():
        freed, filled, shared, ok = [0, 0], [0, 0], False, True
        for both, two in items:
            for w in (0, 1) if both else (0,):
                for half in (0, 1) if w == 0 and shared else (w,):
                    while ok and frees[half] < freed[half]:
                        if abort[0] or rng.random() < runs_out:
                            abort[0], ok = True, False
                        yield
                if not ok:
                    break
                if not counts_late:
                    filled[w] += 1
                copies = rng.randint(1, 3)
                query[w].arrive(copies)
                on_the_way.extend([w] * copies)
                yield
            if not ok:
                break
            shared = not both and two
            freed[0] += 1
            freed[1] += both or two
            if counts_late:
                filled[0] += 1
                filled[1] += both
        for w in (0, 1):
            while filled[w] and not query[w].done((filled[w] - 1) & 1):
                yield

    def reader(w):
        used = [0, 0]
        for both, two in items:
            rows = w if both else 0
            if both or w == 0 or two:
                while query[rows].index <= used[rows]:
                    if abort[0]:
                        return
                    yield
                frees[w] += 1
            used[0] += 1
            used[1] += both
            yield

    team = {name: run for name, run in (("loader", loader()), (0, reader(0)), (1, reader(1)))}
    while "loader" in team:
        if on_the_way and rng.random() < 0.3:
            query[on_the_way.pop(rng.randrange(len(on_the_way)))].land()
            continue
        name = rng.choice(list(team))
        try:
            next(team[name])
        except StopIteration:
            del team[name]
    if on_the_way:
        raise Misuse("left while copies are on the way")
    return abort[0]


def test_giving_up_leaves_nothing_behind():
    gave_up = [play(seed) for seed in range(3000)]
    assert 300 < sum(gave_up) < 2700


def test_the_model_sees_halves_that_are_counted_late():
    with pytest.raises(Misuse):
        for seed in range(500):
            play(seed, counts_late=True)


def test_the_kernel_counts_a_half_before_it_is_filled():
    with open(os.path.join(fb.CSRC, "paged_extend_tc.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    counted = [m.start() for m in re.finditer(r"\+\+filled\[", text)]
    armed = text.index("mbar_arrive_expect_tx(bar(c->query[w]), M::kQ);")
    waits = text.rindex("if (!ok) break;", 0, armed)
    assert len(counted) == 1 and waits < counted[0] < armed


def test_the_kernel_waits_for_every_phase_that_it_began():
    # Whether its copies were TMA's or pieces, which the barrier counts in by an arrival of
    # its own: the waits at the end make no difference.
    with open(os.path.join(fb.CSRC, "paged_extend_tc.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    ends = re.findall(r"&never\)", text)
    assert len(ends) == 3                       # K and V, the query rows, the MMAs
    drain = text[text.index("void drain("):]
    drain = drain[:drain.index("&never")]
    assert "if (" not in drain
    rows = text[text.index("if (filled[w] > 0)"):]
    assert re.match(r"if \(filled\[w\] > 0\) mbar_wait\(", rows)
