"""CPU tests: the paged entry points refuse addresses that are not aligned to
their type, which a kernel could only fault on."""

import pytest

from varlen_flashattention_backward_gb300 import binding as fa
from varlen_flashattention_backward_gb300 import build as fb

from test_paged_abi import DECODE, P, PLAN, WRITE, call


@pytest.fixture(scope="module", autouse=True)
def built():
    fb.build()
    fa.lib()


FOUR = ["block_table", "seq_lens", "delta", "free_pages", "seq_lens_out", "error"]
EIGHT = ["free_state", "slots", "cu_tokens", "free_state_out"]


@pytest.mark.parametrize("name,off", [(n, 2) for n in FOUR] + [(n, 4) for n in EIGHT])
def test_plan(name, off):
    assert call("fa_paged_plan", PLAN, **{name: P + off}) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("name,off", [("slots", 4), ("error", 1)])
def test_write(name, off):
    assert call("fa_paged_write", WRITE, **{name: P + off}) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("name,off", [("block_table", 2), ("seq_lens", 1), ("error", 2)])
def test_decode(name, off):
    assert call("fa_paged_decode", DECODE, **{name: P + off}) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("name", ["softmax_max", "softmax_sum"])
def test_decode_statistics(name):
    stats = dict(softmax_max=P, softmax_sum=P)
    stats[name] = P + 2
    assert call("fa_paged_decode", DECODE, **stats) == fa.FA_ERR_INVALID
