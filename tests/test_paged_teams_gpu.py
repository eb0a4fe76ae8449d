"""GPU tests of decode with many query heads on one key head, where a warp takes
16 of them or a team of two or four warps shares the keys (fp32: 8 at a time):
every type and head dim, pages that TMA copies and pages that it does not, run
directly and by ranges."""

import pytest
import torch

from varlen_flashattention_backward_gb300 import binding as fa
from varlen_flashattention_backward_gb300 import build as fb

from test_paged_gpu import DEV, run_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fb.build()
    fa.lib()
    torch.cuda.set_device(DEV)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 192])
@pytest.mark.parametrize("heads", [12, 17, 32, 40, 64])
@pytest.mark.parametrize("page", [16, 24])
def test_many_heads_on_one(dtype, dim, heads, page):
    run_decode(dtype, [5, 0, 200, 77], heads, 1, dim, page, seed=heads + dim)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("dim,heads", [(32, 64), (96, 32), (128, 48), (192, 32), (192, 64)])
def test_many_heads_over_long_requests(dtype, dim, heads):
    # More blocks than a team has stages, so that its ring goes round; two key heads,
    # a window, head-major pages.
    run_decode(dtype, [1500, 900, 0, 1777], 2 * heads, 2, dim, 32, layout="HND", window=1400,
               seed=dim + heads)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,heads", [(64, 65), (128, 130), (192, 96)])
def test_groups_cut_into_pieces(dtype, dim, heads):
    # Above 64 the group is cut, the last piece partly empty.
    run_decode(dtype, [300, 31, 1000], heads, 1, dim, 16, layout="both", seed=heads)
