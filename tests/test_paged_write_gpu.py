"""GPU tests of large fa_paged_write calls, in which a thread takes two pieces
of each row: above 152 * 256 * 4 pieces of 16 bytes, or, where rows start off
16-byte boundaries, of one element.  Copies, so everything is compared exactly."""

import numpy as np
import pytest
import torch

import oracle
from varlen_flashattention_backward_gb300 import binding as fa
from varlen_flashattention_backward_gb300 import build as fb

from _paged import DTYPE, check_decode, f64, make_cache, to_device

DEV = torch.device("cuda:0")
TWO_EACH = 152 * 256 * 4
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fb.build()
    fa.lib()
    torch.cuda.set_device(DEV)


def pieces(tokens, heads, dim, dtype, shift):
    wide = 4 if dtype == "fp32" else 2
    return tokens * heads * dim * wide // (wide if shift else 16)


def write(dtype, tokens, heads, dim, page, layout, shift, seed):
    rng = np.random.default_rng(seed)
    num_pages = tokens // page + 3
    cache = make_cache(rng, num_pages, page, heads, dim, dtype, layout)
    row = heads * dim
    width = 2 * row + 8 + 5 * (shift > 0)      # odd with a shift: every alignment occurs
    x = torch.from_numpy(rng.standard_normal((tokens, width)).astype(np.float32)).to(DTYPE[dtype])
    rows = [x[:, shift + i * row:shift + (i + 1) * row].unflatten(1, (heads, dim)) for i in (0, 1)]
    xd = x.to(DEV)
    rows_d = [xd[:, shift + i * row:shift + (i + 1) * row].unflatten(1, (heads, dim)) for i in (0, 1)]
    slots = rng.permutation(num_pages * page)[:tokens].astype(np.int64)
    slots[rng.random(tokens) < 0.1] = -1
    slots[-1] = num_pages * page               # one behind the cache
    slots[0] = num_pages * page - 1            # the cache's last
    slots[1:][slots[1:] == slots[0]] = -1
    kd, vd = to_device(cache, DEV)
    error = torch.zeros(1, dtype=torch.int32, device=DEV)
    fa.paged_write(*rows_d, torch.from_numpy(slots).to(DEV), kd, vd, error=error)
    # The definition, in copies of whole rows of bits.
    used = torch.from_numpy((slots >= 0) & (slots < num_pages * page))
    at = torch.from_numpy(slots)[used]
    for got, want, new in zip((kd, vd), cache, rows):
        want = want.clone()
        want[at // page, at % page] = new[used]
        assert torch.equal(got.cpu(), want)
    assert int(error) == fa.FA_PAGED_BAD_SLOT


@pytest.mark.parametrize("dtype,tokens,heads,dim,page,layout,shift", [
    ("bf16", 1301, 8, 128, 16, "NHD", 0), ("bf16", 2601, 5, 96, 24, "HND", 0),
    ("fp16", 13001, 3, 32, 7, "both", 0), ("fp32", 701, 5, 192, 16, "HND", 0),
    ("fp32", 3333, 3, 64, 1, "NHD", 0), ("bf16", 20011, 1, 64, 5, "NHD", 0),
    ("bf16", 40, 32, 192, 16, "NHD", 1), ("bf16", 555, 3, 96, 16, "HND", 1),
    ("fp16", 333, 5, 96, 24, "both", 3), ("fp32", 1717, 1, 96, 16, "NHD", 1),
    ("fp32", 291, 7, 128, 5, "both", 2), ("fp16", 159, 8, 128, 16, "HND", 4)])
def test_two_pieces_each(dtype, tokens, heads, dim, page, layout, shift):
    assert pieces(tokens, heads, dim, dtype, shift) > TWO_EACH
    write(dtype, tokens, heads, dim, page, layout, shift, tokens)


@pytest.mark.parametrize("dtype,heads,dim,shift", [("bf16", 8, 128, 0), ("fp32", 1, 32, 0),
                                                   ("fp16", 1, 64, 1), ("fp32", 4, 32, 1)])
@pytest.mark.parametrize("more", [0, 1])
def test_both_sides_of_the_border(dtype, heads, dim, shift, more):
    row = pieces(1, heads, dim, dtype, shift)
    tokens = TWO_EACH // row + more
    assert (pieces(tokens, heads, dim, dtype, shift) > TWO_EACH) == bool(more)
    write(dtype, tokens, heads, dim, 16, "NHD", shift, row + more)


def test_pages_of_one_token_behind_32_bits():
    # 2^26 + 9 pages of one token of 2 x 32 values: the last lie behind 2^32 elements,
    # 2^33 bytes, of each cache.
    heads, dim, n = 2, 32, (1 << 26) + 9
    assert (n - 1) * heads * dim >= 1 << 32
    k = torch.empty(n, 1, heads, dim, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    rng = np.random.default_rng(0)
    slots = np.array([n - 1, 3, n - 2, (1 << 25) + 1, 0, n - 9, (1 << 26) - 1, 77], np.int64)
    tokens = len(slots)
    rows = torch.from_numpy(rng.standard_normal((2, tokens, heads, dim)).astype(np.float32)).bfloat16()
    fa.paged_write(rows[0].to(DEV), rows[1].to(DEV), torch.from_numpy(slots).to(DEV), k, v)
    at = torch.from_numpy(slots).to(DEV)
    assert torch.equal(k[at, 0].cpu(), rows[0]) and torch.equal(v[at, 0].cpu(), rows[1])
    q = torch.from_numpy(rng.standard_normal((1, 4, dim)).astype(np.float32)).bfloat16()
    table = slots.astype(np.int32)[None]
    ref = oracle.paged_decode(f64(q), f64(rows[0])[:, None], f64(rows[1])[:, None],
                              np.arange(tokens, dtype=np.int32)[None], [tokens], 0.2)
    y, top, total = fa.paged_decode(q.to(DEV), k, v, torch.from_numpy(table).to(DEV),
                                    torch.tensor([tokens], dtype=torch.int32, device=DEV), 0.2,
                                    stats=True)
    check_decode(ref, float(rows[1].float().abs().max()), dim, "bf16", y, top, total)
