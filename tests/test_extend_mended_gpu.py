"""Rows that are computed once more, because a value that they do not see is not finite:
what stays as it was."""

import pytest
import torch

from test_extend_gpu import BIG, DTYPES, Case

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
