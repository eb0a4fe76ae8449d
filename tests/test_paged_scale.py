"""CPU tests of the scales that fa_paged_decode takes: its kernels hold scale
and scale * log2(e) in 32 bits, so neither may be infinite there."""

import pytest

from varlen_flashattention_backward_gb300 import binding as fa
from varlen_flashattention_backward_gb300 import build as fb

from test_paged_abi import DECODE

LARGEST = (2 - 2 ** -23) * 2.0 ** 127


@pytest.fixture(scope="module", autouse=True)
def built():
    fb.build()
    fa.lib()


def decode(scale):
    # Refused for its scale, or, behind that check, for its workspace.
    args = {**DECODE, "scale": scale, "max_pages": 4096, "table_stride": 4096}
    return fa.lib().fa_paged_decode(fa._pack_decode(*args.values()), None)


@pytest.mark.parametrize("scale", [1e39, -1e39, 1.7e308, LARGEST, -LARGEST, LARGEST / 1.4426])
def test_scales_that_pass_the_range_of_fp32(scale):
    assert decode(scale) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("scale", [0.0, -0.5, 1e-300, 1e38, -1e38, LARGEST / 1.4427])
def test_scales_inside_it(scale):
    assert decode(scale) == fa.FA_ERR_WORKSPACE
