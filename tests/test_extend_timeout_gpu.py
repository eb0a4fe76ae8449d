"""Waits of chunk attention that do run out: with several long blocks to a CTA, the next
block's query rows wait for the whole of the one before, some hundred microseconds."""

import pytest
import torch

from _paged import DTYPE
from test_extend_gpu import DEV, Case
from varlen_flashattention_backward_gb300 import binding as fa

pytestmark = pytest.mark.gpu

# Head dim, heads, scale, page: rows by TMA and in pieces (groups of 3; a scale below 0),
# keys in boxes of 64, 8 and 4 and in pieces.
CASES = [(128, 8, None, 64), (64, 8, None, 24), (192, 6, None, 100), (96, 8, -0.1, 5), (32, 8, None, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,heads,scale,page", CASES)
@pytest.mark.parametrize("value", [None, float("nan")])
def test_a_wait_that_does_run_out(dtype, dim, heads, scale, page, value):
    c = Case([8192, 3], [20000, 50], heads, 2, dim, dtype, page=page, scale=scale)
    if value is not None:       # rows that would be looked at again, by flags never written
        c.cache[1][:] = value
    q, *rest = c.on_device()
    size = fa.paged_extend_workspace_size(2, c.rows, heads, 2, dim, DTYPE[dtype])
    room = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((c.rows + 600, heads, dim), 7.0, dtype=q.dtype, device=DEV)
    stats = torch.full((2, c.rows + 600, heads, 8), 5.0, device=DEV)
    part = slice(300, 300 + c.rows)

    def run(wait_ns=0):
        error = torch.zeros(1, dtype=torch.int32, device=DEV)
        fa.paged_extend(q, *rest, c.scale, y=out[part], softmax_max=stats[0, part], softmax_sum=stats[1, part],
                        error=error, workspace=room, wait_timeout_ns=wait_ns)
        return int(error)

    assert run() == 0
    want = out.clone(), stats.clone()
    for wait_ns in (1, 1, 10000):
        room.fill_(255)
        assert run(wait_ns) == fa.FA_PAGED_TIMEOUT
        for t, was in ((out, 7), (stats[0], 5), (stats[1], 5)):
            assert (t[:300] == was).all() and (t[300 + c.rows:] == was).all()
    assert run() == 0
    for got, was in zip((out, stats), want):
        assert torch.equal(got.isnan(), was.isnan()) and torch.equal(got.nan_to_num(), was.nan_to_num())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_calls_beside_one_that_gives_up(dtype):
    # CTAs that leave early make room for another stream's, whose shared memory stays theirs.
    long, other = (Case([8192], [20000], 8, 2, 128, dtype, page=64),
                   Case([5] * 60, [700] * 60, 8, 2, 64, dtype, seed=2))
    want = other.run()[0]
    long_args, args = long.on_device(), other.on_device()
    sides = [torch.cuda.Stream(DEV) for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    error = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = []
    for _ in range(5):
        fa.paged_extend(*long_args, long.scale, error=error, stream=sides[0], wait_timeout_ns=1)
        got += [fa.paged_extend(*args, other.scale, stream=sides[1])[0] for _ in range(4)]
    torch.cuda.synchronize()
    assert int(error) == fa.FA_PAGED_TIMEOUT
    for y in got:
        assert torch.equal(y, want)
