"""What the bounds of ``_paged_bounds`` notice: weights that lose their second
16-bit part, or digits, on ordinary inputs."""

import numpy as np
import pytest

import oracle

from _paged import f64, make_cache, make_table
from _paged_bounds import DTYPE, check_tight, emulate, half_step

LENS = [1, 0, 3, 17, 60, 200]


def inputs(dtype, gain=0.1, dim=64, heads=8, heads_kv=2, page=16):
    import torch
    rng = np.random.default_rng(4)
    pages = sum(-(-n // page) for n in LENS) + 1
    k, v = make_cache(rng, pages, page, heads_kv, dim, dtype)
    table, _ = make_table(rng, LENS, page, pages)
    q = torch.from_numpy(gain * rng.standard_normal((len(LENS), heads, dim)).astype(np.float32))
    args = (f64(q.to(DTYPE[dtype])), f64(k), f64(v), table, LENS, dim ** -0.5)
    return args, float(v.float().abs().max()), dim


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("gain", [0.1, 1.0])
def test_two_parts_keep_the_bound_and_one_does_not(dtype, gain):
    args, v_max, dim = inputs(dtype, gain)
    ref = oracle.paged_decode(*args)
    check_tight(ref, LENS, v_max, dim, dtype, emulate(*args, dtype))
    with pytest.raises(AssertionError, match="of its bound"):
        check_tight(ref, LENS, v_max, dim, dtype, emulate(*args, dtype, parts=1))


def test_twelve_digits_do_not_keep_the_fp32_bound():
    args, v_max, dim = inputs("fp32")
    ref = oracle.paged_decode(*args)
    check_tight(ref, LENS, v_max, dim, "fp32", emulate(*args, "fp32", digits=24))
    with pytest.raises(AssertionError, match="of its bound"):
        check_tight(ref, LENS, v_max, dim, "fp32", emulate(*args, "fp32", digits=12))


@pytest.mark.parametrize("dtype,x,want", [
    ("bf16", 1.0, 2.0 ** -8), ("bf16", 1.99, 2.0 ** -8), ("bf16", 2.0, 2.0 ** -7), ("fp16", 1.0, 2.0 ** -11),
    ("fp16", 0.0, 2.0 ** -25), ("fp16", 2.0 ** -20, 2.0 ** -25), ("fp32", 3.0, 2.0 ** -23)])
def test_half_a_step(dtype, x, want):
    assert half_step(np.array(x), dtype) == want
