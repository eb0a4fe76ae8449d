"""GPU tests of the decode kernel's bounded waits: with a limit of one
nanosecond on healthy copies some wait runs out; the call then ends by itself,
says FA_PAGED_TIMEOUT, and leaves nothing behind that the next call would
notice."""

import numpy as np
import pytest
import torch

from varlen_flashattention_backward_gb300 import binding as fa
from varlen_flashattention_backward_gb300 import build as fb

from _paged import DTYPE

DEV = torch.device("cuda:0")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fb.build()
    fa.lib()
    torch.cuda.set_device(DEV)


def inputs(dtype, heads, heads_kv, dim, lens, page, width):
    g = torch.Generator(device=DEV).manual_seed(2)
    draw = lambda *s: torch.randn(*s, generator=g, device=DEV).to(DTYPE[dtype])  # noqa: E731
    have = [-(-n // page) for n in lens]
    n = sum(have)
    table = np.full((len(lens), max(max(have), width)), -1, np.int32)
    order, at = np.random.default_rng(0).permutation(n), 0
    for b, h in enumerate(have):
        table[b, :h] = order[at:at + h]
        at += h
    args = (draw(len(lens), heads, dim), draw(n, page, heads_kv, dim), draw(n, page, heads_kv, dim),
            torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), 0.125)
    torch.cuda.synchronize()
    return args


def decode(args, **kw):
    error = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = fa.paged_decode(*args, stats=True, error=error, **kw)
    return out, int(error)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


# Teams of one, two and four warps and the fp32 kernel; few requests run
# directly, by one CTA and by clusters, and long ones by ranges.  `surely`: so much
# is on the way at once that some wait takes longer than the GPU's timer needs to
# move; in the others a copy may always be there first.
@pytest.mark.parametrize("dtype,heads,heads_kv,dim,lens,width,surely", [
    ("bf16", 8, 2, 128, [4000] * 60, 0, True), ("bf16", 8, 2, 128, [2000], 0, False),
    ("bf16", 8, 8, 64, [120] * 30, 0, False), ("bf16", 8, 8, 128, [500] * 30, 0, True),
    ("bf16", 8, 8, 128, [8000], 0, True), ("fp16", 16, 1, 192, [5000] * 20, 0, True),
    ("bf16", 32, 1, 64, [5000] * 20, 0, True), ("bf16", 32, 1, 192, [300] * 100, 0, True),
    ("fp16", 64, 1, 128, [3000] * 9, 4000, False), ("bf16", 64, 1, 32, [900] * 4, 0, False),
    ("fp16", 64, 1, 192, [5000] * 60, 0, True), ("fp32", 4, 2, 128, [3000] * 20, 0, True),
    ("fp32", 8, 8, 128, [250] * 30, 0, True), ("fp32", 8, 1, 64, [700], 0, False),
    ("fp32", 1, 1, 192, [700], 3000, False)])
def test_a_wait_that_runs_out_ends_the_call(dtype, heads, heads_kv, dim, lens, width, surely):
    args = inputs(dtype, heads, heads_kv, dim, lens, 16, width)
    want, error = decode(args)
    assert error == 0
    cold = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    expired = 0
    for _ in range(40):
        cold.zero_()               # what the cache held leaves the L2
        _, error = decode(args, wait_timeout_ns=1)
        assert error in (0, fa.FA_PAGED_TIMEOUT)
        expired += error != 0
        got, error = decode(args)
        assert error == 0 and same(got, want)
    assert expired > 0 or not surely
    # A generous limit is none of these.
    got, error = decode(args, wait_timeout_ns=10 ** 9)
    assert error == 0 and same(got, want)


def test_without_an_error_word_the_call_still_ends():
    args = inputs("bf16", 8, 2, 128, [4000] * 60, 16, 0)
    want, _ = decode(args)
    for _ in range(5):
        fa.paged_decode(*args, wait_timeout_ns=1)
    got, error = decode(args)
    assert error == 0 and same(got, want)


def test_pages_that_are_not_whole_blocks_wait_for_no_barrier():
    args = inputs("bf16", 8, 2, 64, [700, 90], 24, 0)
    want, _ = decode(args)
    got, error = decode(args, wait_timeout_ns=1)
    assert error == 0 and same(got, want)
