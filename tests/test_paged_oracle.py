"""CPU pins of the paged-cache oracle: hand-worked plans, the conservation of
pages over many calls, and single-token attention against the packed one."""

import numpy as np
import pytest

import oracle
from oracle import paged as po

from _paged import make_table


def test_plan_by_hand():
    # Pages of 4; ring of 6 whose free pages are 5, 0, 3 (from position 4 on,
    # around the end).
    table = np.array([[1, -1, -1], [2, 4, -1], [-1, -1, -1]], np.int32)
    ring = np.array([3, 9, 9, 9, 5, 0], np.int32)
    r = oracle.paged_plan(table, [3, 6, 0], [2, -3, 5], ring, [4, 3], 4, 8)
    assert r["error"] == 0
    assert r["cu"].tolist() == [0, 2, 2, 7]
    assert r["seq_lens"].tolist() == [5, 3, 5]
    # Request 0 takes page 5 for its fifth token, request 2 takes 0 and 3;
    # request 1 gives page 4 back behind the ring's end (position 1).
    assert r["block_table"].tolist() == [[1, 5, -1], [2, 4, -1], [0, 3, -1]]
    assert r["slots"].tolist() == [1 * 4 + 3, 5 * 4, 0, 1, 2, 3, 3 * 4, -1]
    assert r["free_pages"].tolist() == [3, 4, 9, 9, 5, 0]
    assert r["free_state"].tolist() == [1, 1]


def test_plan_refusals_by_hand():
    table = np.full((4, 2), -1, np.int32)
    table[0, 0] = 0
    ring = np.array([1, 2, 0, 0], np.int32)
    # 0 fits in its page; 1 takes both free pages; 2 finds none; 3 would pass
    # its two pages.
    r = oracle.paged_plan(table, [1, 0, 0, 0], [1, 3, 1, 5], ring, [0, 2], 2, 64)
    assert r["error"] == po.EXHAUSTED | po.ROW_FULL
    assert r["seq_lens"].tolist() == [2, 3, 0, 0]
    assert r["slots"][:10].tolist() == [1, 2, 3, 4, -1, -1, -1, -1, -1, -1]
    # A request that needs no page is granted behind one that finds none.
    r = oracle.paged_plan(table, [1, 0, 0, 0], [1, 4, 4, 0], ring, [0, 0], 2, 64)
    assert r["error"] == po.EXHAUSTED and r["seq_lens"].tolist() == [2, 0, 0, 0]
    r = oracle.paged_plan(table, [1, 0, 0, 0], [1, 2, 0, 0], ring, [0, 2], 2, 2)
    assert r["error"] == po.ROWS and r["slots"].tolist() == [1, -1]
    assert oracle.paged_plan(table, [1, -1, 5, 0], [0] * 4, ring, [0, 2], 2, 0)["error"] == \
        po.BAD_LENGTH
    for state in ([-1, 2], [4, 2], [0, 5], [0, -1]):
        r = oracle.paged_plan(table, [1, 0, 0, 0], [1, 0, 0, 0], ring, state, 2, 4)
        assert r["error"] & po.BAD_POOL and r["seq_lens"].tolist() == [1, 0, 0, 0]
        assert (r["slots"] == -1).all() and (r["block_table"] == table).all()


@pytest.mark.parametrize("page", [1, 3, 16])
def test_pages_are_conserved(page):
    rng = np.random.default_rng(page)
    batch, width, n = 9, 7, 30
    table, lens = np.full((batch, width), -1, np.int32), np.zeros(batch, np.int64)
    ring, state = rng.permutation(n).astype(np.int32), np.array([11, n])
    for _ in range(200):
        delta = rng.integers(-3 * page, 3 * page + 2, batch)
        r = oracle.paged_plan(table, lens, delta, ring, state, page, 1000)
        assert r["error"] & ~(po.EXHAUSTED | po.ROW_FULL) == 0
        table, lens, ring, state = (r[k] for k in ("block_table", "seq_lens", "free_pages",
                                                   "free_state"))
        held = [int(table[b, i]) for b in range(batch) for i in range(-(-int(lens[b]) // page))]
        free = [int(ring[(state[0] + i) % n]) for i in range(state[1])]
        assert sorted(held + free) == list(range(n))
        used = r["slots"][r["slots"] >= 0]
        assert len(set(used.tolist())) == len(used) and np.isin(used // page, held).all()


def test_write_then_read():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 5, 2, 8))
    cache = np.zeros((3, 4, 2, 8))
    kc, vc, err = oracle.paged_write(k, v, [11, -1, 0, 5, 12], cache, cache)
    assert err == po.BAD_SLOT
    assert (kc[2, 3] == k[0]).all() and (vc[0, 0] == v[2]).all() and (kc[1, 1] == k[3]).all()
    assert np.count_nonzero(kc.any(axis=(2, 3))) == 3


@pytest.mark.parametrize("window", [2 ** 31 - 1, 5, 0])
def test_decode_is_the_last_row_of_the_packed_forward(window):
    rng = np.random.default_rng(1)
    lens, page, heads, heads_kv, dim = [13, 1, 8, 0], 4, 4, 2, 8
    total = sum(lens)
    q, k, v = (rng.standard_normal((total, h, dim)) for h in (heads, heads_kv, heads_kv))
    y, m, l = oracle.varlen_forward(q, k, v, lens, lens, 0.3, window, 0)
    table, _ = make_table(rng, lens, page, 12)
    kc, vc = np.full((2, 12, page, heads_kv, dim), np.nan)
    cu, last = np.cumsum([0] + lens), []
    for b, n in enumerate(lens):
        slots = [table[b, j // page] * page + j % page for j in range(n)]
        kc, vc, _ = oracle.paged_write(k[cu[b]:], v[cu[b]:], slots, kc, vc)
        last.append(cu[b + 1] - 1)
    r = oracle.paged_decode(q[last], kc, vc, table, lens, 0.3, window)
    some = [0, 1, 2]
    rows = [last[b] for b in some]
    stat = lambda x: np.asarray(x)[rows].reshape(3, heads, -1)[..., 0]  # noqa: E731
    np.testing.assert_allclose(r["y"][some], y[rows], rtol=1e-12)
    np.testing.assert_allclose(r["max"][some], stat(m), rtol=1e-12)
    np.testing.assert_allclose(r["sum"][some], stat(l), rtol=1e-12)
    assert (r["y"][3] == 0).all() and (r["max"][3] == -np.inf).all() and r["error"] == 0
