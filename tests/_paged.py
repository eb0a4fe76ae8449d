"""Shared pieces of the paged-cache tests: seeded caches, and the bounds that
the single-token attention is held to."""

from __future__ import annotations

import numpy as np
import torch

DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def f64(t) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def make_cache(rng, num_pages, page, heads_kv, dim, dtype, layout="NHD", fill=None):
    """CPU k and v caches viewed as [pages, page, heads, dim]; `fill` puts one
    value everywhere.  Layouts: token-major, head-major, K beside V."""
    def draw(shape):
        x = rng.standard_normal(shape).astype(np.float32)
        if fill is not None:
            x[:] = fill
        return torch.from_numpy(x).to(DTYPE[dtype])
    if layout == "NHD":
        return (draw((num_pages, page, heads_kv, dim)), draw((num_pages, page, heads_kv, dim)))
    if layout == "HND":
        return (draw((num_pages, heads_kv, page, dim)).transpose(1, 2),
                draw((num_pages, heads_kv, page, dim)).transpose(1, 2))
    both = draw((num_pages, 2, page, heads_kv, dim))
    return both[:, 0], both[:, 1]


def to_device(cache, dev):
    """The cache on the device with the same strides."""
    k, v = cache
    if k.untyped_storage().data_ptr() == v.untyped_storage().data_ptr():
        both = torch.stack([k, v], dim=1).to(dev)
        return both[:, 0], both[:, 1]
    if not k.is_contiguous():
        return tuple(x.transpose(1, 2).contiguous().to(dev).transpose(1, 2) for x in cache)
    return tuple(x.to(dev) for x in cache)


def make_table(rng, lens, page, num_pages, width=None):
    """Distinct pages in random order for each request, -1 behind them."""
    have = [-(-max(0, int(x)) // page) for x in lens]
    width = max(1, max(have)) if width is None else width
    order = rng.permutation(num_pages)
    table, at = np.full((len(lens), width), -1, np.int32), 0
    for b, n in enumerate(have):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:].astype(np.int32)


def decode_bounds(ref, v_max, dim, dtype):
    """Largest errors of (y, max, sum) against float64, as arrays.

    u = 2^-24 is half a step of fp32.  With w = scale * sum_d |q_d k_d|, a dot
    product of `dim` terms in fp32, in any order, is off by at most
    dim * u * w; tensor cores may cut off instead of rounding, which doubles
    u: ds = 2 (dim + 4) u w, the 4 for the products with the scale and with
    log2(e) and the subtraction of the maximum (both at most |s| <= w).
    exp of that is off by ds, plus 4 u for exp2's own error (2 ulp).  A weight
    that goes to the tensor cores as a sum of two 16-bit numbers keeps 2 * 8
    bits of bf16 or 2 * 11 of fp16: rounding the remainder leaves 2^-17 (bf16)
    of the weight; 2^-16 covers it and fp16's floor 2^-25 for each of the two.
    The sum of weights adds up to 2^12 keys here, in any order at most
    2^12 * u of it.  y is a quotient of two such sums, with |v| <= v_max:
    dy = 2 dp v_max, and its own rounding of eps / 2 (bf16 2^-8, fp16 2^-11,
    fp32 2^-24)."""
    u = 2.0 ** -24
    w = ref["weight"]
    ds = 2 * (dim + 4) * u * w
    dp = ds + 4 * u + 2.0 ** 12 * u + (2.0 ** -16 if dtype != "fp32" else 0.0)
    half = torch.finfo(DTYPE[dtype]).eps / 2
    # fp16 loses relative precision below 2^-14: half a step there is 2^-25.
    floor = 2.0 ** -25 if dtype == "fp16" else 0.0
    dy = 2 * dp[..., None] * v_max * (1 + half) + half * np.abs(ref["y"]) + floor
    return dy, ds + 4 * u * np.abs(np.where(np.isfinite(ref["max"]), ref["max"], 0)), dp * ref["sum"] + ds * ref["sum"]


def check_decode(ref, v_max, dim, dtype, y, top=None, total=None):
    dy, dm, dt = decode_bounds(ref, v_max, dim, dtype)
    # A NaN among the keys that a row sees makes its whole row NaN; a row whose
    # scores pass fp32's range, or that sees an infinite value, is not compared.
    nan = np.isnan(ref["sum"])
    assert np.isnan(f64(y)[nan]).all()
    with np.errstate(invalid="ignore"):
        fine = ~nan & np.isfinite(ref["y"]).all(-1) & (ref["weight"] < 2.0 ** 127)
    err = np.abs(f64(y) - ref["y"])[fine]
    assert (err <= dy[fine]).all(), f"y off by {(err / dy[fine]).max():.3g} of its bound"
    if top is None:
        return
    top, total = f64(top), f64(total)
    assert np.isnan(total[nan]).all()
    top, total, dm, dt = top[fine], total[fine], dm[fine], dt[fine]
    ref = {key: ref[key][fine] for key in ("max", "sum")}
    assert (top == top[..., :1]).all() and (total == total[..., :1]).all()
    empty = ref["max"] == -np.inf
    assert (top[..., 0][empty] == -np.inf).all() and (total[..., 0][empty] == 0).all()
    got, want = top[..., 0][~empty], ref["max"][~empty]
    assert (np.abs(got - want) <= dm[~empty]).all()
    # The sum is relative to the kernel's own maximum.
    moved = ref["sum"][~empty] * np.exp(want - got)
    assert (np.abs(total[..., 0][~empty] - moved) <= 2 * dt[~empty]).all()
