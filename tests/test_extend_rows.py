"""Bounds of rows that descend: requests could share rows, whose results would go by the
order of the CTAs, so the call does nothing (fa_paged_extend)."""

import numpy as np
import pytest

import oracle
from varlen_flashattention_backward_gb300 import binding as fa


def test_the_oracle_does_nothing():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 8, 4, 1, 8))
    q, table = rng.standard_normal((20, 2, 8)), np.arange(8).reshape(2, 4)
    for cu, rows, error in (([0, 5, 20], range(20), 0), ([2, 5, 5], range(2, 5), 0), ([0, 5, 60], range(20), 4),
                            ([-4, 5, 9], range(9), 4), ([0, 9, 5], (), 4), ([5, 4, 9], (), 4), ([-1, -2, 3], (), 4),
                            ([30, 29, 40], (), 4)):
        ref = oracle.paged_extend(q, k, v, table, [16, 9], np.array(cu), 0.3)
        assert ref["error"] == error and np.flatnonzero(ref["owned"]).tolist() == list(rows)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("cu", [[0, 50, 20, 60, 70], [0, 74, 0, 74, 74], [10, 9, 20, 40, 70], [-1, -2, 20, 40, 60],
                                [0, 30, 40, 100, 99], [2 ** 40, 3, 4, 5, 6], [0, 1, 2, 3, -2 ** 62]])
def test_rows_that_descend(dtype, cu):
    from test_extend_gpu import Case
    c = Case([30, 10, 20, 10], [100, 300, 20, 7], 4, 2, 64, dtype, pad=4)
    c.cu = np.array(cu, np.int64)
    c.check(error=fa.FA_PAGED_ROWS)
    c.lens[1] = -1
    c.check(error=fa.FA_PAGED_ROWS | fa.FA_PAGED_BAD_LENGTH)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_the_last_of_2048_requests_descends(dtype):
    from test_extend_gpu import Case
    c = Case([1] * 2048, [3] * 2048, 4, 2, 32, dtype, page=4)
    c.check()
    c.cu[2048] = 2046
    c.check(error=fa.FA_PAGED_ROWS)
    c.cu[2047:] = 2046, 2048
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_every_request_descends(dtype):
    from test_extend_gpu import Case
    c = Case([1] * 2048, [3] * 2048, 64, 1, 32, dtype, page=4)
    c.cu = np.arange(2048, -1, -1, dtype=np.int64)
    c.check(error=fa.FA_PAGED_ROWS)
    c.cu[::2], c.cu[1::2] = 2048, 0
    c.check(error=fa.FA_PAGED_ROWS)
