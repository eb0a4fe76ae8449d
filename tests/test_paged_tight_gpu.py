"""GPU tests of single-token attention against bounds that follow from each
row's number of keys, for short rows and for long ones."""

import numpy as np
import pytest
import torch

import oracle
from varlen_flashattention_backward_gb300 import binding as fa
from varlen_flashattention_backward_gb300 import build as fb

from _paged import DTYPE, f64, make_cache, make_table, to_device
from _paged_bounds import check_tight, depth

DEV = torch.device("cuda:0")
BIG = 2 ** 31 - 1
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fb.build()
    fa.lib()
    torch.cuda.set_device(DEV)


def run(dtype, lens, heads, heads_kv, dim, page, gain, window=BIG, seed=0, wide=40000):
    rng = np.random.default_rng(seed)
    lens = np.array(lens)
    pages = sum(-(-int(n) // page) for n in lens) + 2
    k, v = make_cache(rng, pages, page, heads_kv, dim, dtype)
    table, _ = make_table(rng, lens, page, pages)
    q = torch.from_numpy(gain * rng.standard_normal((len(lens), heads, dim)).astype(np.float32))
    q = q.to(DTYPE[dtype])
    ref = oracle.paged_decode(f64(q), f64(k), f64(v), table, lens, dim ** -0.5, window)
    kd, vd = to_device((k, v), DEV)
    keys = np.minimum(lens, window + 1)
    v_max = float(v.float().abs().max())
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    in_a_row, parts = depth(lens, heads, heads_kv, dtype, sms, window)
    # As wide as the longest request, and wider, where all are cut into ranges.
    for width in (table.shape[1], max(table.shape[1], wide // page)):
        t = np.full((len(lens), width), -1, np.int32)
        t[:, :table.shape[1]] = table
        y, top, total = fa.paged_decode(
            q.to(DEV), kd, vd, torch.from_numpy(t).to(DEV),
            torch.from_numpy(lens).to(DEV, torch.int32), dim ** -0.5, pre_tokens=window, stats=True)
        check_tight(ref, keys, v_max, dim, dtype, y, top, total, in_a_row=in_a_row, parts=parts)


SHORT = [1, 0, 2, 3, 15, 16, 17, 60, 200]


@pytest.mark.parametrize("gain", [0.1, 1.0])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 192])
@pytest.mark.parametrize("dtype,heads,heads_kv", [
    ("fp32", 2, 2), ("fp32", 4, 1), ("fp32", 24, 2), ("bf16", 8, 2), ("bf16", 12, 1), ("bf16", 32, 1),
    ("bf16", 64, 1), ("fp16", 4, 4), ("fp16", 16, 1), ("fp16", 24, 1), ("fp16", 48, 1)])
def test_short_rows(dtype, heads, heads_kv, dim, page, gain):
    run(dtype, SHORT, heads, heads_kv, dim, page, gain, seed=dim + heads)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("gain", [0.1, 2.0])
def test_windows(dtype, gain):
    run(dtype, [900, 41, 7, 300], 8, 2, 64, 16, gain, window=40, seed=1)


@pytest.mark.parametrize("dtype,heads", [("fp32", 2), ("bf16", 4), ("bf16", 32), ("fp16", 4), ("fp16", 16)])
def test_long_rows(dtype, heads):
    run(dtype, [20000, 4097, 0, 1, 700], heads, 1, 64, 64, 1.0, seed=heads, wide=70000)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_the_longest_rows(dtype):
    run(dtype, [131072, 65536], 2, 1, 32, 256, 0.5, seed=3, wide=140000)
