"""Rows that are computed once more, because a value that they do not see is not finite:
what stays as it was, and how long many of them take."""

import numpy as np
import pytest
import torch

from test_extend_gpu import BIG, DTYPES, Case
from varlen_flashattention_backward_gb300 import binding as fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_statistics_are_those_of_finite_values(dtype, value):
    # Bit for bit: masked scores are no part of them.
    for key, pre in ((60, 20), (150, BIG), (170, 33), (0, 5)):
        c = Case([100, 3, 260], [77, 600, 0], 4, 2, 64, dtype, page=24)
        _, *want, _ = c.run(pre)
        for b in (0, 2):
            at = c.table[b, key // 24], key % 24
            c.cache[1][at[0], at[1], 1, 5] = value
        y, *got, error = c.run(pre)
        assert error == 0
        for a, z in zip(got, want):
            assert torch.equal(a, z)
        c.check(pre)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("columns", [slice(None), slice(5, 6)])
def test_a_cache_full_of_nan(dtype, columns):
    # Every row is flagged, and all warps of a span share them.  The bounds on the time are
    # two to three times what it takes with one column, and an eighth of it (16 bits; a half,
    # fp32) with one warp at work.
    c = Case([4096, 3] if dtype == "fp32" else [8192, 3], [20000, 50], 8, 2, 64, dtype, page=24)
    args = c.on_device()
    args[2][..., columns] = float("nan")
    y, _, _ = fa.paged_extend(*args, c.scale)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    fa.paged_extend(*args, c.scale, y=y)
    end.record()
    torch.cuda.synchronize()
    assert y[..., columns].isnan().all()
    rest = np.setdiff1d(np.arange(64), np.arange(64)[columns])
    assert y[..., torch.from_numpy(rest).to(y.device)].isfinite().all()
    assert start.elapsed_time(end) < (700 if dtype == "fp32" else 1500)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("batch,heads,heads_kv", [(31, 4, 2), (33, 2, 2), (700, 4, 1), (2048, 2, 2)])
def test_rows_of_many_requests(dtype, batch, heads, heads_kv):
    # The last key of some requests, which their earlier rows do not see.
    new = np.arange(batch) % 4
    c = Case(new, [20] * batch, heads, heads_kv, 32, dtype, page=4)
    for b in {0, 1, 2, 3, 30, 31, 32, batch // 2, batch - 1} | set(range(5, batch, 7)):
        if b < batch:
            last = int(c.lens[b]) - 1
            c.cache[1][c.table[b, last // 4], last % 4, b % heads_kv, 3] = float("nan")
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_row_whose_first_scores_are_minus_infinity(dtype):
    # It sees NaN with weight 0 first and finite values then, which makes NaN, beside values
    # that it does not see; a row that sees no other scores stays 0.
    c = Case([40, 3], [60, 90], 2, 1, 64, dtype, page=16)
    c.q[:] = c.q.abs().clamp(min=0.1)
    for b in range(2):
        for j in range(int(c.lens[b])):
            at = c.table[b, j // 16], j % 16, 0
            if j < 50 or b == 1:
                c.cache[0][at] = -float("inf")
            if j < 50 or j >= int(c.lens[b]) - 1:
                c.cache[1][at] = float("nan")
    y, top, total, error = c.run()
    assert error == 0 and y[:40].isnan().all() and (total[:40] > 0).all()
    assert (y[40:43] == 0).all() and (total[40:43] == 0).all() and (top[40:43] == -float("inf")).all()
    y, _, total, _ = c.run(after=-60)            # row i sees keys 0 to i
    assert (y[:40] == 0).all() and (total[:40] == 0).all()
    y, _, total, _ = c.run(after=-20)            # 0 to 40 + i
    assert (y[:10] == 0).all() and (total[:10] == 0).all() and y[10:40].isnan().all()
