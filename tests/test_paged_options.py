"""CPU tests of fa_paged_decode_ex: its checks are those of fa_paged_decode, and
its options are packed as the header lays them out."""

import os
import re

import pytest

from varlen_flashattention_backward_gb300 import binding as fa
from varlen_flashattention_backward_gb300 import build as fb

from test_paged_abi import DECODE


@pytest.fixture(scope="module", autouse=True)
def built():
    fb.build()
    fa.lib()


def call(options, **kw):
    args = {k: v or 0 for k, v in {**DECODE, **kw}.items()}
    return fa.lib().fa_paged_decode_ex(fa._pack_decode(*args.values()), options, None)


def test_options_are_packed_as_the_header_lays_them_out():
    with open(os.path.join(fb.INCLUDE, "fa_varlen.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} fa_paged_decode_options;", text).group(1)
    assert [d.strip() for d in body.split(";") if d.strip()] == ["int64_t wait_timeout_ns"]
    assert len(fa._pack_options(1)) == 8


@pytest.mark.parametrize("options", [None, fa._pack_options(0), fa._pack_options(1000),
                                     fa._pack_options(-5)])
def test_refusals_are_those_of_decode(options):
    assert fa.lib().fa_paged_decode_ex(None, options, None) == fa.FA_ERR_NULLPTR
    assert call(options, q=None) == fa.FA_ERR_NULLPTR
    assert call(options, batch=0) == fa.FA_ERR_INVALID
    assert call(options, reserved=1) == fa.FA_ERR_INVALID
    assert call(options, max_pages=4096, table_stride=4096) == fa.FA_ERR_WORKSPACE
