"""Chunk attention at the ends of its ranges: values at the top of the type's, and
windows at the far end of the longest request."""

import numpy as np
import pytest
import torch

from _extend import check_extend
from _paged import DTYPE, f64
from test_extend_gpu import BIG, DEV, DTYPES, Case, dev
from varlen_flashattention_backward_gb300 import binding as fa

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


@pytest.mark.parametrize("dim", [32, 128, 192])
@pytest.mark.parametrize("unseen", [None, float("nan"), float("inf")])
def test_many_large_values_beside_one_that_is_not_finite(dim, unseen):
    # 200 keys and more that weigh alike, each 2^121, sum up to 2^128 and more where weights are
    # 1.  In bf16 they are 2^-8, in rows that are computed once more too.
    c = Case([100, 70], [200, 300], 2, 1, dim, "bf16", page=16)
    c.cache[0][:] = 0
    c.cache[1][:] = 2.0 ** 121
    if unseen is not None:
        for b, key in ((0, 290), (1, 365)):
            c.cache[1][c.table[b, key // 16], key % 16, 0, 3] = unseen
    y = c.check()
    if unseen is not None:
        assert (f64(y[:90, :, 3]) == 2.0 ** 121).all() and not np.isfinite(f64(y[90:100, :, 3])).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new,past", [([1, 5], [300, 90]), ([200], [300]), ([3], [9000])])
def test_small_values(dtype, new, past):
    # Down to the smallest normal values of bf16 and fp32, about 2^-126.
    c = Case(new, past, 4, 2, 64, dtype, page=16)
    c.cache[1][:] = c.cache[1].double() * 2.0 ** -118
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [32, 64, 192])
@pytest.mark.parametrize("new,past", [([1], [0]), ([5, 200], [3, 300]), ([3], [9000]), ([300], [0])])
def test_scores_of_minus_infinity_beside_values_that_are_not_finite(dtype, dim, new, past):
    # y = 0, whatever the values are; next to them a head whose keys are finite.
    c = Case(new, past, 4, 2, dim, dtype, page=16)
    c.q[:] = c.q.abs().clamp(min=0.1)
    c.cache[0][:, :, 0] = -float("inf")
    c.cache[1][:, ::2, 0] = float("inf")
    c.cache[1][:, 1::3, 0] = float("nan")
    y, top, total, error = c.run()
    own = slice(0, int(c.cu[-1]))
    assert error == 0 and (y[own, :2] == 0).all()
    assert (top[own, :2] == -float("inf")).all() and (total[own, :2] == 0).all()
    c.q[:, :2] = 0.0      # (out of the oracle's way)
    c.cache[0][:, :, 0] = 0.0
    c.cache[1][:, :, 0] = 0.0
    ref = c.oracle()
    check_extend({k: x if k in ("error", "owned", "keys") else x[:, 2:] for k, x in ref.items()}, dim, dtype,
                 y[:, 2:], top[:, 2:], total[:, 2:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_windows_at_the_end_of_the_longest_request(dtype):
    # 2^30 keys: one page, named over and over.  A row at the last of them sees key 0 where
    # the window ends 2^30 - 1 keys before it, and none where it ends before that.
    page, pages = 65536, 16384
    g = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randn(1, page, 1, 32, generator=g, device=DEV).to(DTYPE[dtype])
    v = torch.randn(1, page, 1, 32, generator=g, device=DEV).to(DTYPE[dtype])
    q = torch.randn(1, 2, 32, generator=g, device=DEV).to(DTYPE[dtype])
    table = torch.zeros(1, pages, dtype=torch.int32, device=DEV)
    lens, cu = dev(np.array([2 ** 30], np.int32)), dev(np.array([0, 1], np.int64))
    for pre in (BIG, 2 ** 30, 2 ** 40):
        y, top, total = fa.paged_extend(q, k, v, table, lens, cu, 0.2, pre, 1 - 2 ** 30, stats=True)
        assert torch.equal(y[0, 0], v[0, 0, 0]) and torch.equal(y[0, 1], v[0, 0, 0])
        # exp2 of the rounding of one score, 2^-24 of it, and its own error of 2^-22.
        score = 0.2 * float((q.double().abs() * k[0, 0].double().abs()).sum(-1).max())
        assert float((total - 1).abs().max()) <= score * 2.0 ** -24 + 2.0 ** -22
        for after in (-2 ** 30, -2 ** 31, -2 ** 40):
            y, top, total = fa.paged_extend(q, k, v, table, lens, cu, 0.2, pre, after, stats=True)
            assert (y == 0).all() and (top == -float("inf")).all() and (total == 0).all()
