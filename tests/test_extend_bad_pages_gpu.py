"""Bad table entries of chunk attention where they count and where they do not: the
error word speaks of keys that some row sees, not of their neighbours in a tile."""

import pytest

from test_extend_gpu import BIG, DTYPES, Case
from varlen_flashattention_backward_gb300 import binding as fa

pytestmark = pytest.mark.gpu

BAD = (-1, 2 ** 30)


def case(new, length, dim, dtype, page):
    return Case(new, [length - n for n in new], 4, 2, dim, dtype, page=page, seed=length)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 192])
@pytest.mark.parametrize("page", [16, 12, 5])
@pytest.mark.parametrize("bad", BAD)
def test_pages_that_a_window_has_left_behind(dtype, dim, page, bad):
    # The first key that any row sees lies inside a tile (of 32, 64 or 128 keys): entries
    # of the pages before its own name nothing.
    for first in (115, 98, 131, 197):
        c = case([2], 320, dim, dtype, page)
        c.table[0, :first // page] = bad
        c.check(318 - first)
        c.table[0, first // page] = bad
        c.check(318 - first, error=fa.FA_PAGED_BAD_PAGE)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 192])
@pytest.mark.parametrize("page", [16, 12, 5])
@pytest.mark.parametrize("bad", BAD)
def test_pages_that_the_rows_have_not_come_to(dtype, dim, page, bad):
    # Rows that see nothing of the last keys.
    for last in (206, 140, 101, 290):
        c = case([3, 7], 320, dim, dtype, page)
        c.table[0, last // page + 1:] = bad
        c.table[1, last // page + 1:] = bad
        c.check(BIG, last - 319)
        c.table[1, last // page] = bad
        c.check(BIG, last - 319, error=fa.FA_PAGED_BAD_PAGE)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", BAD)
def test_windows_without_a_key(dtype, bad):
    # No row sees anything, though windows of several rows span keys between them.
    for pre, after in ((5, -6), (-3, 2), (40, -70)):
        c = case([90, 1], 320, 64, dtype, 16)
        c.table[:] = bad
        y = c.check(pre, after)
        assert (y == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_two_blocks_with_a_gap(dtype):
    # A window of one key behind each row: those between the requests' rows are seen, the rest not.
    c = case([70, 300], 600, 64, dtype, 16)
    c.table[0, :(600 - 70 - 90) // 16] = -1
    c.table[1, :(600 - 300 - 90) // 16] = -1
    c.table[:, (600 - 90) // 16 + 1:] = -1
    c.check(90, -90)
