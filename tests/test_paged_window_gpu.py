"""GPU test of a window that is not a plain int: its value counts at each call,
not the object."""

import pytest
import torch

from varlen_flashattention_backward_gb300 import binding as fa
from varlen_flashattention_backward_gb300 import build as fb

DEV = torch.device("cuda:0")
pytestmark = pytest.mark.gpu


def test_a_window_that_is_changed_in_place():
    fb.build()
    g = torch.Generator(device=DEV).manual_seed(0)
    k, v = (torch.randn(600, 16, 2, 64, generator=g, device=DEV).bfloat16() for _ in range(2))
    q = torch.randn(1, 8, 64, generator=g, device=DEV).bfloat16()
    table = torch.arange(600, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([9600], dtype=torch.int32, device=DEV)
    window = torch.tensor(20)
    small = fa.paged_decode(q, k, v, table, lens, 0.125, pre_tokens=window)[0]
    # Now the call runs by ranges, which need a workspace.
    window.fill_(9000)
    large = fa.paged_decode(q, k, v, table, lens, 0.125, pre_tokens=window)[0]
    torch.cuda.synchronize()
    assert fa.paged_decode_workspace_size(1, 8, 2, 64, q.dtype, 16, 600, 20) == 0
    assert fa.paged_decode_workspace_size(1, 8, 2, 64, q.dtype, 16, 600, 9000) > 0
    assert torch.equal(small, fa.paged_decode(q, k, v, table, lens, 0.125, pre_tokens=20)[0])
    assert torch.equal(large, fa.paged_decode(q, k, v, table, lens, 0.125, pre_tokens=9000)[0])
