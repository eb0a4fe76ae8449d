"""Bounds on the errors of single-token attention over the cache that follow from
the number of keys a row sees, and a plain emulation of how the 16-bit kernels
multiply weights and values, to show what such bounds notice."""

from __future__ import annotations

import numpy as np
import torch

from _paged import DTYPE, f64

U = 2.0 ** -24          # half a step of fp32


def half_step(x, dtype):
    """Half the distance of neighbouring numbers of the type at |x|."""
    digits, lowest = {"bf16": (7, -126), "fp16": (10, -14), "fp32": (23, -126)}[dtype]
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** lowest)))
    return 2.0 ** (e - digits - 1)


def depth(lens, heads, heads_kv, dtype, sms, window=2 ** 31 - 1):
    """(blocks that one team takes in a row, parts that a row is cut into), at
    most.  A direct call gives a team 8 blocks; otherwise the blocks of all
    requests and key heads (the group in pieces of up to 64 heads, fp32 8), one more
    for each of them, are dealt evenly to 2 to 16 teams per multiprocessor."""
    keys = np.minimum(np.asarray(lens, np.int64), window + 1)
    blocks = keys // (8 if dtype == "fp32" else 16) + 3
    pieces = heads_kv * -(-heads // heads_kv // (8 if dtype == "fp32" else 64))
    return max(8, int(-(-blocks.sum() * max(1, pieces) // (2 * sms)))) + 1, 16 * sms


def tight_bounds(ref, keys, v_max, dim, dtype, in_a_row=10 ** 9, parts=10 ** 9):
    """Largest errors of (y, max, sum relative to the kernel's own maximum)
    against float64.  `keys` [batch]: the keys that each row sees.

    w = |scale| max_j sum_d |q_d k_jd| bounds a row's scores.  The keys are b blocks of 16
    (fp32: 8), one more where the first is not whole; a team takes r <= b of them in a
    row, and c <= b parts are joined.

    Scores: `dim` products are added in some order, each addition off by u on
    the CUDA cores and, where tensor cores may cut off, 2 u (products of 16-bit
    numbers are exact there): a dim u w, a = 1 or 2.  The product with the scale,
    that constant, and the subtraction of the maximum (a difference of at most 2 w):
    4 u w more.  The same in the exponent of e: ds = (a dim + 4) u w.
    exp2 is off by 2^-22 = 4 u of its value.

    Maxima: a weight meets a factor at each block behind it whose maximum is larger,
    and at each join: 5 u for a factor (4 u) and its product, in a join one more of each
    and an addition, and a last stage over CTAs or warps; the exponents add up to at
    most 2 w: df = (5 r + 7 c + 16) u + 2 u w.

    Sums of weights: 4 additions in a block's lanes of which one goes on, 3 at a
    part's end, one in each join: dl = (r + c + 8) u.

    Products with values: fp32 adds one key at a time, then the parts:
    dp = (8 r + c + 8) u.  A tensor product adds 16 terms to what was there, 17
    additions of 2 u each at worst, r times, twice with 16 rows, and the parts:
    dp = (2 * 34 r + c + 8) u.  The weight in two 16-bit numbers: its first
    part leaves at most 2^-8 (bf16) or 2^-11 (fp16) of the binade below, the second
    half a step of that: 2^-17 and 2^-23 of the weight, and fp16, scaled by
    2^15, never less than 2^-40 of the largest.

    y = sum p v / sum p with |v| <= v_max, 3 roundings (two parts added, 1 / sum,
    product), then one to the type.  2^-8 more for products of errors, which
    are all below 2^-9."""
    tc = dtype != "fp32"
    n = np.asarray(keys, np.float64)[:, None]
    b = np.ceil(n / (16 if tc else 8)) + 1
    r, c = np.minimum(b, in_a_row), np.minimum(b, parts)
    w = ref["weight"]
    ds = ((2 if tc else 1) * dim + 4) * U * w
    dw = ds + 4 * U + (5 * r + 7 * c + 16) * U + 2 * U * w
    dl = (r + c + 8) * U
    dp = ((68 * r if tc else 8 * r) + c + 8) * U
    if tc:
        dp = dp + (2.0 ** -17 if dtype == "bf16" else 2.0 ** -23 + n * 2.0 ** -40)
    assert (dw + dl + dp < 2.0 ** -9).all()
    more = 1 + 2.0 ** -8
    y = np.abs(ref["y"])
    e = more * ((dw + dp)[..., None] * v_max + (dw + dl + 3 * U)[..., None] * y)
    dy = e + half_step(y + e, dtype)
    dm = ds + 2 * U * np.abs(np.where(np.isfinite(ref["max"]), ref["max"], 0))
    return dy, dm, more * (dw + dl + dm) * ref["sum"]


def check_tight(ref, keys, v_max, dim, dtype, y, top=None, total=None, **deep):
    dy, dm, dt = tight_bounds(ref, keys, v_max, dim, dtype, **deep)
    err = np.abs(f64(y) - ref["y"])
    assert (err <= dy).all(), f"y off by {(err / dy).max():.3g} of its bound"
    if top is None:
        return
    top, total = f64(top)[..., 0], f64(total)[..., 0]
    empty = ref["max"] == -np.inf
    assert (top[empty] == -np.inf).all() and (total[empty] == 0).all()
    got, want = top[~empty], ref["max"][~empty]
    assert (np.abs(got - want) <= dm[~empty]).all()
    moved = ref["sum"][~empty] * np.exp(want - got)
    assert (np.abs(total[~empty] - moved) <= dt[~empty]).all()


def emulate(q, k_pages, v_pages, block_table, seq_lens, scale, dtype, parts=2, digits=None):
    """y with the weights as the sum of `parts` numbers of the type (or rounded
    to `digits` binary digits), all else in float64, rounded to the type once."""
    t = DTYPE[dtype]
    rounded = lambda x: f64(torch.from_numpy(np.asarray(x)).to(t))  # noqa: E731
    batch, heads, dim = q.shape
    page, group = k_pages.shape[1], heads // k_pages.shape[2]
    y = np.zeros((batch, heads, dim))
    for b, length in enumerate(seq_lens):
        pos = np.arange(length)
        at = np.asarray(block_table[b])[pos // page], pos % page
        for h in range(heads if length else 0):
            s = scale * (k_pages[at][:, h // group] @ q[b, h])
            p = np.exp(s - s.max())
            if digits:
                step = 2.0 ** (np.floor(np.log2(p)) - digits + 1)
                used = np.round(p / step) * step
            else:
                used = rounded(p)
                if parts == 2:
                    used = used + rounded(p - used)
            y[b, h] = used @ v_pages[at][:, h // group] / p.sum()
    return torch.from_numpy(y).to(t)
