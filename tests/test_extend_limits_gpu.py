"""Chunk attention at the ends of its types' ranges."""

import numpy as np
import pytest
import torch

from _paged import f64
from test_extend_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 192])
@pytest.mark.parametrize("new,past,at", [(1, 383, 300), (1, 383, 100), (200, 300, 310), (3, 9000, 8500),
                                         (700, 0, 90)])
def test_large_values_behind_small_ones(dtype, dim, new, past, at):
    """One key counts 2^7 times as much as each before it and holds values of 2^122: its
    product is 2^129 where the weights are relative to the keys before it, and 2^122
    where they are relative to the largest, as the sums of the definition are.  Every
    result is below 2^122."""
    c = Case([new], [past], 2, 1, dim, dtype, page=16)
    c.q[:] = 1
    c.cache[0][:] = 0
    c.cache[1][:] = 0
    key = c.table[0, at // 16], at % 16, 0
    c.cache[0][key] = 7 * np.log(2) / (c.scale * dim)
    c.cache[1][key] = 2.0 ** 122
    y = c.check()
    assert torch.isfinite(y).all() and f64(y).max() > 2.0 ** 115


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new,past", [([1, 5], [300, 90]), ([200], [300]), ([3], [9000])])
def test_small_values(dtype, new, past):
    # Down to the smallest normal values of bf16 and fp32, about 2^-126.
    c = Case(new, past, 4, 2, 64, dtype, page=16)
    c.cache[1][:] = c.cache[1].double() * 2.0 ** -118
    c.check()
