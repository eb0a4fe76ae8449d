"""GPU tests of the paged cache: the plan, the write and the single-token
attention, each against its float64 (or whole-number) oracle, and all three
together as a decoding loop."""

import math

import numpy as np
import pytest
import torch
import torch.nn.functional as F

import oracle
from oracle import paged as po
from varlen_flashattention_backward_gb300 import binding as fa
from varlen_flashattention_backward_gb300 import build as fb

from _paged import DTYPE, check_decode, decode_bounds, f64, make_cache, make_table, to_device

DEV = torch.device("cuda:0")
BIG = 2 ** 31 - 1
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fb.build()
    fa.lib()
    torch.cuda.set_device(DEV)


def dev(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x)).to(DEV, dtype)


# ---------------------------------------------------------------------------
# Plan
# ---------------------------------------------------------------------------

def run_plan(table, lens, delta, ring, state, page, max_tokens, in_place=False):
    t = dict(block_table=dev(table, torch.int32), seq_lens=dev(lens, torch.int32),
             delta=dev(delta, torch.int32), free_pages=dev(ring, torch.int32),
             free_state=dev(state, torch.int64))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.full((max_tokens,), -77, dtype=torch.int64, device=DEV)
    kw = dict(seq_lens_out=t["seq_lens"], free_state_out=t["free_state"]) if in_place else {}
    slots, cu, new, st = fa.paged_plan(**t, page_size=page, max_tokens=max_tokens, slots=slots,
                                       error=err, **kw)
    return dict(slots=slots.cpu().numpy(), cu=cu.cpu().numpy(), seq_lens=new.cpu().numpy(),
                free_state=st.cpu().numpy(), block_table=t["block_table"].cpu().numpy(),
                free_pages=t["free_pages"].cpu().numpy(), error=int(err))


def check_plan(got, ref):
    for key, want in ref.items():
        assert np.array_equal(got[key], want), key


def random_plan(rng, batch, page, width, grow, spare):
    lens = rng.integers(0, width * page + 1, batch)
    have = [-(-int(n) // page) for n in lens]
    n = max(1, sum(have) + spare)
    table, free = make_table(rng, lens, page, n, width)
    head = int(rng.integers(n))
    ring = np.full(n, -1, np.int32)
    ring[(head + np.arange(len(free))) % n] = free
    delta = rng.integers(0, grow + 1, batch)
    kind = rng.random(batch)
    delta = np.where(kind < 0.2, -rng.integers(1, 2 * width * page, batch), delta)
    return table, lens, np.where(kind > 0.8, 0, delta), ring, [head, len(free)]


@pytest.mark.parametrize("batch,page,width,grow,spare,max_tokens", [
    (1, 16, 4, 5, 3, 8), (1, 1, 1, 1, 0, 0), (3, 5, 9, 30, 10, 100), (64, 16, 12, 1, 64, 64),
    (33, 1, 50, 20, 300, 500), (257, 24, 7, 100, 900, 20000), (2048, 16, 3, 40, 3000, 90000),
    (1000, 128, 5, 3, 20, 700), (2047, 1, 4, 2, 0, 4000), (17, 64, 300, 9000, 2000, 70001)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(batch, page, width, grow, spare, max_tokens, in_place):
    rng = np.random.default_rng(batch + page)
    args = random_plan(rng, batch, page, width, grow, spare)
    check_plan(run_plan(*args, page, max_tokens, in_place),
               oracle.paged_plan(*args, page, max_tokens))


@pytest.mark.parametrize("state,lens,delta", [
    ([0, 8], [5, -1, 9, 4], [1, 1, 1, 0]),             # lengths out of range
    ([-1, 4], [1, 2, 3, 4], [1, 1, -1, 9]),            # pools that are none
    ([8, 4], [1, 2, 3, 4], [1, 1, -1, 9]),
    ([2 ** 40, 2], [1, 2, 3, 4], [1, 1, -1, 9]),
    ([0, 9], [1, 2, 3, 4], [1, 1, -1, 9]),
    ([0, 8], [1, 2, 3, 4], [1, 0, -8, 0]),             # no room for what comes back
    ([3, 2], [8, 8, 8, 8], [1, 2 ** 31 - 1, -2 ** 31, 0]),
    ([3, 0], [4, 8, 0, 1], [4, -8, 1, 3]),             # what comes back serves the next call
])
def test_plan_bad_values(state, lens, delta):
    table = np.arange(8, dtype=np.int32).reshape(4, 2)
    ring = np.arange(8, dtype=np.int32)
    args = (table, lens, delta, ring, state, 4, 16)
    check_plan(run_plan(*args), oracle.paged_plan(*args))


def test_plan_bad_page_ids():
    # A half-filled page, a taken page and a ring entry that are no pages.
    table = np.array([[8, 1], [-3, 2], [4, 5]], np.int32)
    ring = np.array([0, 99, 6, 7, -1, 0, 0, 0], np.int32)
    args = (table, [2, 1, 4], [1, 4, 2], ring, [0, 5], 4, 16)
    got, ref = run_plan(*args), oracle.paged_plan(*args)
    check_plan(got, ref)
    assert got["error"] == po.BAD_PAGE


def test_plan_repeats_and_strided_table():
    rng = np.random.default_rng(5)
    table, lens, delta, ring, state = random_plan(rng, 20, 8, 6, 20, 40)
    wide = torch.full((20, 11), 12345, dtype=torch.int32, device=DEV)
    wide[:, 2:8] = dev(table)
    view = wide[:, 2:8]
    t = [view, dev(lens, torch.int32), dev(delta, torch.int32), dev(ring, torch.int32),
         dev(state, torch.int64)]
    first = [x.clone() for x in fa.paged_plan(*t, 8, 300)] + [view.clone(), t[3].clone()]
    again = [x.clone() for x in fa.paged_plan(*t, 8, 300)] + [view.clone(), t[3].clone()]
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    ref = oracle.paged_plan(table, lens, delta, ring, state, 8, 300)
    assert np.array_equal(view.cpu().numpy(), ref["block_table"])
    assert (wide[:, :2] == 12345).all() and (wide[:, 8:] == 12345).all()


# ---------------------------------------------------------------------------
# Write
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("tokens,heads,dim,page,layout,shift", [
    (1, 1, 32, 1, "NHD", 0), (7, 2, 96, 5, "HND", 0), (64, 8, 128, 16, "NHD", 0),
    (300, 5, 192, 24, "both", 0), (33, 4, 64, 16, "HND", 1), (129, 3, 64, 7, "NHD", 3)])
def test_write(dtype, tokens, heads, dim, page, layout, shift):
    rng = np.random.default_rng(tokens)
    pages = tokens // page + 4
    cache = make_cache(rng, pages, page, heads, dim, dtype, layout)
    # Rows inside a wider projection; `shift` elements in, so that rows start
    # off the 16-byte boundaries.
    width = 3 * heads * dim + 5 * shift
    x = torch.from_numpy(rng.standard_normal((tokens, width)).astype(np.float32)).to(DTYPE[dtype])
    rows = [x[:, shift + i * heads * dim:shift + (i + 1) * heads * dim].unflatten(1, (heads, dim))
            for i in (0, 2)]
    xd = x.to(DEV)
    rows_d = [xd[:, shift + i * heads * dim:shift + (i + 1) * heads * dim].unflatten(1, (heads, dim))
              for i in (0, 2)]
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    slots[rng.random(tokens) < 0.2] = -1
    slots[tokens // 2] = pages * page + 3      # behind the cache
    kd, vd = to_device(cache, DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    fa.paged_write(*rows_d, dev(slots), kd, vd, error=err)
    k, v, e = oracle.paged_write(f64(rows[0]), f64(rows[1]), slots, f64(cache[0]), f64(cache[1]))
    assert np.array_equal(f64(kd), k) and np.array_equal(f64(vd), v) and int(err) == e


def test_write_of_no_tokens():
    kd, vd = to_device(make_cache(np.random.default_rng(0), 2, 4, 2, 32, "bf16"), DEV)
    before = kd.clone()
    none = torch.empty(0, 2, 32, dtype=torch.bfloat16, device=DEV)
    fa.paged_write(none, none, torch.empty(0, dtype=torch.int64, device=DEV), kd, vd)
    assert torch.equal(kd, before)


# ---------------------------------------------------------------------------
# Decode
# ---------------------------------------------------------------------------

def run_decode(dtype, lens, heads, heads_kv, dim, page, layout="NHD", window=BIG, scale=None, seed=0,
               spare=3, edit=None, width=None, q_gain=1.0):
    """Runs one call and checks it; `edit(table, kc, vc, lens)` changes the CPU
    inputs first."""
    rng = np.random.default_rng(seed)
    lens = np.array(lens, np.int64)
    num_pages = sum(-(-max(0, int(n)) // page) for n in lens) + spare
    cache = make_cache(rng, num_pages, page, heads_kv, dim, dtype, layout)
    table, _ = make_table(rng, lens, page, num_pages, width)
    # Behind a request's length the cache holds what nobody may see.
    seen = np.zeros((num_pages, page), bool)
    for b, n in enumerate(lens):
        for j in range(max(0, int(n) - 1 - window), int(n)):
            seen[table[b, j // page], j % page] = True
    hidden = torch.from_numpy(~seen)
    v_max = max([1e-30] + [float(cache[1][torch.from_numpy(seen)].float().abs().max())]
                if seen.any() else [1e-30])
    for x, bad in zip(cache, (float("nan"), float("inf"))):
        x[hidden] = bad
        x[hidden & (torch.arange(num_pages)[:, None] % 2 == 0)] = torch.finfo(DTYPE[dtype]).min
    q = torch.from_numpy(q_gain * rng.standard_normal((len(lens), heads, dim)).astype(np.float32))
    q = q.to(DTYPE[dtype])
    if edit:
        edit(table, cache[0], cache[1], lens)
    scale = dim ** -0.5 if scale is None else scale
    kd, vd = to_device(cache, DEV)
    qd, lens_d = q.to(DEV), dev(lens, torch.int32)
    # Once with the table as wide as the longest request, where few and short
    # requests are run directly, and once with a wide one, where all are cut into
    # ranges and joined.
    wide = np.full((len(lens), max(table.shape[1], 40000 // page)), -1, np.int32)
    wide[:, :table.shape[1]] = table
    for tab in (table, wide):
        ref = oracle.paged_decode(f64(q), f64(cache[0]), f64(cache[1]), tab, lens, scale, window)
        size = fa.paged_decode_workspace_size(len(lens), heads, heads_kv, dim, q.dtype, page,
                                              tab.shape[1], window)
        ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        args = (qd, kd, vd, dev(tab, torch.int32), lens_d, scale)
        y, top, total = fa.paged_decode(*args, pre_tokens=window, stats=True, workspace=ws,
                                        error=err)
        check_decode(ref, v_max, dim, dtype, y, top, total)
        assert int(err) == ref["error"]
        again, none, _ = fa.paged_decode(*args, pre_tokens=window)
        assert none is None and np.array_equal(f64(again), f64(y), equal_nan=True)
    return y


RAGGED = [1, 0, 17, 16, 15, 130, 64, 3, 999, 0, 33]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 192])
@pytest.mark.parametrize("heads,heads_kv,page,layout", [
    (2, 2, 16, "NHD"), (8, 2, 24, "HND"), (5, 5, 1, "NHD"), (7, 1, 5, "both"), (16, 1, 64, "NHD"),
    (6, 3, 8, "both"), (4, 4, 32, "HND")])
def test_decode(dtype, dim, heads, heads_kv, page, layout):
    run_decode(dtype, RAGGED, heads, heads_kv, dim, page, layout, seed=dim)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("heads,heads_kv", [(1, 1), (2, 1), (3, 1), (8, 1), (9, 1), (12, 2), (17, 1),
                                            (32, 1), (40, 1), (64, 2), (100, 1), (256, 1), (256, 256)])
def test_decode_groups(dtype, heads, heads_kv):
    run_decode(dtype, [5, 0, 200, 77], heads, heads_kv, 64, 16, seed=heads)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("window", [0, 1, 15, 16, 100, 998, 999, -1, -5])
def test_decode_window(dtype, window):
    run_decode(dtype, RAGGED, 4, 2, 64, 16, window=window, seed=3)


@pytest.mark.parametrize("batch,length", [(1, 1), (1, 4000), (2048, 1), (2048, 9), (500, 40), (3, 2500)])
def test_decode_batches(batch, length):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, length + 1, batch)
    lens[rng.integers(batch)] = length
    run_decode("bf16", lens, 2, 1, 32, 16, seed=batch)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("batch", [152, 153, 304, 305])
def test_decode_one_or_two_waves(dtype, batch):
    # One CTA per request up to twice the GPU's SMs, ranges above.
    lens = np.random.default_rng(batch).integers(0, 200, batch)
    run_decode(dtype, lens, 3, 1, 64, 16, seed=batch)


@pytest.mark.parametrize("dtype,batch,heads,heads_kv,shortest,page", [
    ("bf16", 40, 16, 8, 1500, 16), ("fp16", 100, 64, 2, 1600, 24), ("fp32", 20, 8, 8, 1500, 32)])
def test_decode_large_batches(dtype, batch, heads, heads_kv, shortest, page):
    # Many blocks in each warp's range, and many segments in some.
    lens = np.random.default_rng(batch).integers(shortest, 2500, batch)
    lens[3] = 0
    run_decode(dtype, lens, heads, heads_kv, 32, page, seed=batch)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("gap", [10.25, 15.5, 20.75, 26.5])
@pytest.mark.parametrize("heads", [1, 16])
def test_decode_many_light_keys(dtype, gap, heads):
    # Key 0 weighs 1 and holds zeros; 4096 others weigh 2^-gap each and hold 1024, so
    # y = 4096 1024 2^-gap / (1 + 4096 2^-gap) comes from the light ones alone.  Scores
    # and values are exact.  Besides y's rounding, half a step: the exponent is off by
    # at most three roundings (scale log2 e, a product, a difference) of numbers below
    # 2^5, 3 2^5 2^-24 ln 2 < 2^-17; the weight in two 16-bit parts by 2^-17; exponential,
    # sums (at most 6 blocks of 16 keys in a team, then 64 parts) and quotient by less
    # than 128 2^-23 = 2^-16.  In all 2^-15.
    t, dim, n = DTYPE[dtype], 64, 4097
    k, v = torch.zeros(2, 258, 16, 1, dim)
    k.view(-1, dim)[1:n, 5] = -gap
    v.view(-1, dim)[1:n] = 1024
    q = torch.zeros(1, heads, dim)
    q[:, :, 5] = 1
    qd, kd, vd = (x.to(t).to(DEV) for x in (q, k, v))
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    weight = 4096 * 2.0 ** -gap
    want = weight * 1024 / (1 + weight)
    for width in (257, 3000):          # directly, and by ranges
        table = torch.zeros(1, width, dtype=torch.int32, device=DEV)
        table[0, :257] = torch.arange(257)
        y, _, _ = fa.paged_decode(qd, kd, vd, table, lens, math.log(2.0))
        off = np.abs(f64(y) - want).max() / want
        assert off <= torch.finfo(t).eps / 2 + 2.0 ** -15


def test_decode_all_empty():
    for dtype in DTYPE:
        y = run_decode(dtype, [0, 0, 0], 4, 2, 64, 16)
        assert (y == 0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_decode_sharp_and_flat_scores(dtype):
    run_decode(dtype, [700, 40], 8, 2, 128, 16, q_gain=8.0)
    run_decode(dtype, [700, 40], 8, 2, 128, 16, scale=0.0)
    run_decode(dtype, [700, 40], 8, 2, 128, 16, scale=-0.2)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_decode_scores_of_minus_infinity(dtype):
    # k = -inf in one dimension where q > 0: the key's weight is 0; a request
    # with no other key has none above -inf.
    rng = np.random.default_rng(0)
    k, v = make_cache(rng, 6, 16, 1, 32, dtype)
    q = torch.ones(2, 1, 32, dtype=DTYPE[dtype])
    table = np.array([[0, 1, 2], [3, 4, 5]], np.int32)
    k[0, :, 0, 5] = -np.inf
    k[1, 3, 0, 9] = -np.inf
    k[3:, :, 0, 1] = -np.inf
    lens = np.array([40, 20])
    with np.errstate(invalid="ignore"):
        ref = oracle.paged_decode(f64(q), f64(k), f64(v), table, lens, 0.2)
    finite = k.clone()
    finite[torch.isinf(finite)] = 0
    ref["weight"] = oracle.paged_decode(f64(q), f64(finite), f64(v), table, lens, 0.2)["weight"]
    y, top, total = fa.paged_decode(q.to(DEV), k.to(DEV), v.to(DEV), dev(table), dev(lens, torch.int32),
                                    0.2, stats=True)
    check_decode(ref, float(v.float().abs().max()), 32, dtype, y, top, total)
    assert (y[1] == 0).all() and (top[1] == -np.inf).all() and (total[1] == 0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_decode_infinite_values_stay_in_their_column(dtype):
    # One value of one key head is infinite: its column of that head's queries is
    # infinite (fp32) or NaN, everything else as without it.
    (q, k, v, table, lens, scale), ref, cache = decode_inputs(4, [40, 300], dtype=dtype)
    v[table[1, 2].long(), 5, 1, 7] = float("inf")
    y, top, total = fa.paged_decode(q, k, v, table, lens, scale, stats=True)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[1, 4:, 7] = True
    bad = y[hit]
    assert (bad == float("inf")).all() if dtype == "fp32" else not torch.isfinite(bad).any()
    y[hit] = torch.from_numpy(ref["y"]).to(y)[hit]
    check_decode(ref, float(cache[1].float().abs().max()), 64, dtype, y, top, total)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("page", [4, 16, 48])
def test_decode_bad_pages_and_lengths(dtype, page):
    def edit(table, kc, vc, lens):
        table[0, 1] = -1
        table[1, 0] = kc.shape[0]
        table[2, :] = 2 ** 31 - 1
        lens[3] = -7
        lens[4] = 2 ** 31 - 1      # clamped to the table, whose last entries are -1
    run_decode(dtype, [150, 60, 100, 9, 97], 4, 2, 64, page, edit=edit)


def test_decode_pages_shared_by_requests():
    def edit(table, kc, vc, lens):
        table[1, :5] = table[0, :5]
    run_decode("bf16", [90, 85, 7], 8, 2, 64, 16, edit=edit)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_decode_strided_rows_and_untouched_neighbours(dtype, shift):
    rng = np.random.default_rng(shift)
    b, heads, heads_kv, dim, page = 5, 6, 2, 64, 16
    lens = np.array([20, 0, 300, 1, 64])
    cache = make_cache(rng, 30, page, heads_kv, dim, dtype)
    table, _ = make_table(rng, lens, page, 30)
    row = heads * dim
    wide = torch.from_numpy(rng.standard_normal((b + 2, row + 37)).astype(np.float32)).to(DTYPE[dtype])
    q = wide[1:1 + b, shift:shift + row].unflatten(1, (heads, dim))
    ref = oracle.paged_decode(f64(q), f64(cache[0]), f64(cache[1]), table, lens, 0.125)
    wd, out = wide.to(DEV), torch.full((b + 2, row + 37), 7.0, dtype=DTYPE[dtype], device=DEV)
    y = out[1:1 + b, shift:shift + row].unflatten(1, (heads, dim))
    stat = torch.full((2, b + 2, heads, 8), 7.0, device=DEV)
    wtable = torch.full((b, 40), -9, dtype=torch.int32, device=DEV)
    wtable[:, 3:3 + table.shape[1]] = dev(table)
    got = fa.paged_decode(wd[1:1 + b, shift:shift + row].unflatten(1, (heads, dim)),
                          *to_device(cache, DEV), wtable[:, 3:3 + table.shape[1]],
                          dev(lens, torch.int32), 0.125, y=y, softmax_max=stat[0, 1:1 + b],
                          softmax_sum=stat[1, 1:1 + b])
    assert got[0].data_ptr() == y.data_ptr()
    check_decode(ref, float(cache[1].float().abs().max()), dim, dtype, y, stat[0, 1:1 + b],
                 stat[1, 1:1 + b])
    out[1:1 + b, shift:shift + row] = 7.0
    stat[:, 1:1 + b] = 7.0
    assert (out == 7.0).all() and (stat == 7.0).all()


def test_decode_one_head_key_tensors_with_odd_strides():
    # The stride of an axis with one entry is anything.
    rng = np.random.default_rng(2)
    k, v = make_cache(rng, 1, 16, 1, 64, "bf16")
    kd, vd = (x.to(DEV).as_strided((1, 16, 1, 64), (1, 64, 3, 1)) for x in (k, v))
    q = torch.randn(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    ref = oracle.paged_decode(f64(q), f64(k), f64(v), np.zeros((1, 1), np.int32), [11], 0.1)
    y, top, total = fa.paged_decode(q, kd, vd, dev(np.zeros((1, 1), np.int32)),
                                    dev([11], torch.int32), 0.1, stats=True)
    check_decode(ref, float(v.float().abs().max()), 64, "bf16", y, top, total)


def test_offsets_past_32_bits():
    # A cache of 2^32 + elements: the last pages lie behind 2^32 elements, the
    # slots of a one-token page behind 2^31 bytes.
    page, heads, dim = 16, 8, 128
    n = (1 << 32) // (page * heads * dim) + 8
    k = torch.empty(n, page, heads, dim, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    rng = np.random.default_rng(0)
    rows = torch.from_numpy(rng.standard_normal((2, 50, heads, dim)).astype(np.float32))
    rows = rows.to(torch.bfloat16)
    ids = np.array([n - 1, n - 3, 2, n - 8], np.int32)
    slots = np.concatenate([i * page + np.arange(page) for i in ids.astype(np.int64)])[:50]
    fa.paged_write(rows[0].to(DEV), rows[1].to(DEV), dev(slots), k, v)
    assert torch.equal(k[n - 1].cpu(), rows[0, :16]) and torch.equal(v[n - 8, :2].cpu(), rows[1, 48:])
    q = torch.randn(1, 16, dim, dtype=torch.bfloat16, device=DEV)
    small = np.arange(4, dtype=np.int32)[None]
    pad = np.zeros((14, heads, dim))
    ck, cv = (np.concatenate([f64(x), pad]).reshape(4, page, heads, dim) for x in rows)
    ref = oracle.paged_decode(f64(q), ck, cv, small, [50], 0.09)
    y, top, total = fa.paged_decode(q, k, v, dev(ids[None]), dev([50], torch.int32), 0.09, stats=True)
    check_decode(ref, float(rows[1].float().abs().max()), dim, "bf16", y, top, total)


# ---------------------------------------------------------------------------
# Streams, graphs, and all three together
# ---------------------------------------------------------------------------

def decode_inputs(seed, lens, heads=8, heads_kv=2, dim=64, page=16, dtype="bf16"):
    rng = np.random.default_rng(seed)
    n = sum(-(-x // page) for x in lens) + 2
    cache = make_cache(rng, n, page, heads_kv, dim, dtype)
    table, _ = make_table(rng, lens, page, n)
    q = torch.from_numpy(rng.standard_normal((len(lens), heads, dim)).astype(np.float32))
    q = q.to(DTYPE[dtype])
    ref = oracle.paged_decode(f64(q), f64(cache[0]), f64(cache[1]), table, lens, 0.125)
    return (q.to(DEV), *to_device(cache, DEV), dev(table), dev(lens, torch.int32), 0.125), ref, cache


def test_two_streams_at_once():
    a, ra, ca = decode_inputs(0, [2000, 1500])
    b, rb, cb = decode_inputs(1, [900, 3000, 12])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        outs.append((fa.paged_decode(*a, stream=s1)[0], fa.paged_decode(*b, stream=s2)[0]))
    torch.cuda.synchronize()
    for ya, yb in outs:
        check_decode(ra, float(ca[1].float().abs().max()), 64, "bf16", ya)
        check_decode(rb, float(cb[1].float().abs().max()), 64, "bf16", yb)
        assert torch.equal(ya, outs[0][0]) and torch.equal(yb, outs[0][1])


def test_steps_on_a_stream_without_a_graph():
    """Plan, write and decode launched one behind the other, where each may
    start before the one before it is done: every step sees its own lengths, and
    the cut and joined requests too."""
    torch.manual_seed(3)
    heads, heads_kv, dim, page, b, steps = 8, 2, 64, 16, 3, 60
    n_pages, width = 700, 2600          # a wide table: ranges and a join
    first = [4000, 17, 2000]
    kc, vc = (torch.randn(n_pages, page, heads_kv, dim, dtype=torch.bfloat16, device=DEV)
              for _ in range(2))
    table = torch.full((b, width), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(b, dtype=torch.int32, device=DEV)
    ring = torch.arange(n_pages, dtype=torch.int32, device=DEV)
    state = torch.tensor([0, n_pages], dtype=torch.int64, device=DEV)
    pool = dict(seq_lens_out=lens, free_state_out=state)
    fa.paged_plan(table, lens, dev(first, torch.int32), ring, state, page, sum(first), **pool)
    ones = torch.ones(b, dtype=torch.int32, device=DEV)
    q = torch.randn(steps, b, heads, dim, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.randn(steps, b, heads_kv, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    torch.cuda.synchronize()
    got = []
    for i in range(steps):
        slots, _, _, _ = fa.paged_plan(table, lens, ones, ring, state, page, b, **pool)
        fa.paged_write(k[i], v[i], slots, kc, vc)
        got.append(fa.paged_decode(q[i], kc, vc, table, lens, 0.125, stats=True))
    torch.cuda.synchronize()
    kh, vh, th = f64(kc), f64(vc), table.cpu().numpy()
    v_max = float(np.abs(vh).max())
    for i in (0, 1, 15, 16, 31, steps - 1):
        ref = oracle.paged_decode(f64(q[i]), kh, vh, th, np.array(first) + i + 1, 0.125)
        check_decode(ref, v_max, dim, "bf16", *got[i])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_prompt_then_steps_equal_the_packed_forward(dtype):
    """Prompts through plan and write, then decoding steps (plan, write,
    decode) captured once and replayed: each step's y is the row that the
    packed forward gives for the whole sequence; one request ends on the way
    and its pages serve another."""
    torch.manual_seed(0)
    heads, heads_kv, dim, page, steps = 8, 2, 64, 8, 20
    prompts = [33, 8, 1, 0]
    b, n_pages, width = len(prompts), 24, 10
    dt = DTYPE[dtype]
    total = [p + steps for p in prompts]
    q, k, v = (torch.randn(sum(total), h, dim, device=DEV, dtype=dt) for h in (heads, heads_kv, heads_kv))
    cu = np.concatenate([[0], np.cumsum(total)])
    kc, vc = (torch.full((n_pages, page, heads_kv, dim), float("nan"), dtype=dt, device=DEV)
              for _ in range(2))
    table = torch.full((b, width), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(b, dtype=torch.int32, device=DEV)
    ring = torch.arange(n_pages, dtype=torch.int32, device=DEV)
    state = torch.tensor([0, n_pages], dtype=torch.int64, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pool = dict(seq_lens_out=lens, free_state_out=state, error=err)
    slots, _, _, _ = fa.paged_plan(table, lens, dev(prompts, torch.int32), ring, state, page, 64, **pool)
    pick = np.concatenate([cu[i] + np.arange(p) for i, p in enumerate(prompts)])
    pad = np.zeros(64 - len(pick), np.int64)
    rows = dev(np.concatenate([pick, pad]))
    fa.paged_write(k[rows], v[rows], slots, kc, vc, error=err)
    # One step, captured.
    ones = torch.ones(b, dtype=torch.int32, device=DEV)
    sq, sk, sv = (torch.empty(b, h, dim, dtype=dt, device=DEV) for h in (heads, heads_kv, heads_kv))
    keep = [x.clone() for x in (table, lens, ring, state, kc, vc)]

    def step():
        s, _, _, _ = fa.paged_plan(table, lens, ones, ring, state, page, b, **pool)
        fa.paged_write(sk, sv, s, kc, vc, error=err)
        return fa.paged_decode(sq, kc, vc, table, lens, 0.125, stats=True, error=err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                      # once outside, as for any capture
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((table, lens, ring, state, kc, vc), keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    got = []
    for i in range(steps):
        at = dev(np.array([cu[r] + prompts[r] + i for r in range(b)]))
        sq.copy_(q[at]), sk.copy_(k[at]), sv.copy_(v[at])
        graph.replay()
        got.append([x.clone() for x in out])
    assert int(err) == 0
    assert lens.tolist() == total
    y, smax, ssum = (f64(x) for x in fa.fwd(q, k, v, total, total, 0.125, BIG, 0))
    ry, rm, rl = oracle.varlen_forward(f64(q), f64(k), f64(v), total, total, 0.125, BIG, 0)
    v_max = float(v.float().abs().max())
    for i, (yi, mi, li) in enumerate(got):
        at = [cu[r] + prompts[r] + i for r in range(b)]
        ref = dict(y=ry[at], max=np.asarray(rm)[at].reshape(b, heads, -1)[..., 0],
                   sum=np.asarray(rl)[at].reshape(b, heads, -1)[..., 0])
        weight = np.zeros((b, heads))
        for r in range(b):
            for h in range(heads):
                kk = np.abs(f64(k)[cu[r]:at[r] + 1, h // (heads // heads_kv)])
                weight[r, h] = 0.125 * (kk @ np.abs(f64(q)[at[r], h])).max()
        ref["weight"] = weight
        check_decode(ref, v_max, dim, dtype, yi, mi, li)
        # The library's own forward gives the same rows: two roundings apart.
        dy = decode_bounds(ref, v_max, dim, dtype)[0]
        assert (np.abs(f64(yi) - y[at]) <= 2 * dy).all()
    # Request 1 ends; its pages come back and request 3 takes them.
    held = table[1, :-(-total[1] // page)].tolist()
    free = int(state[1])
    ends = dev([0, -10 ** 9, 0, 0], torch.int32)
    fa.paged_plan(table, lens, ends, ring, state, page, 0, **pool)
    assert int(lens[1]) == 0 and int(state[1]) == free + len(held)
    n = (width - (-(-total[3] // page))) * page
    fa.paged_plan(table, lens, dev([0, 0, 0, n], torch.int32), ring, state, page, 128, **pool)
    taken = table[3, -(-total[3] // page):].tolist()
    assert int(err) == 0 and set(held) <= set(taken) | set(
        ring[(int(state[0]) + torch.arange(int(state[1]))) % n_pages].tolist())


def test_large_plan_in_a_graph():
    """A plan of many rows, updated in place and captured: every replay goes on
    from where the one before ended."""
    rng = np.random.default_rng(4)
    b, page, width, n_pages, max_tokens = 40, 16, 64, 3000, 6000
    table, lens, delta, ring, state = random_plan(rng, b, page, width, 120, n_pages)
    t = [dev(table, torch.int32), dev(lens, torch.int32), dev(delta, torch.int32),
         dev(ring, torch.int32), dev(state, torch.int64)]
    first = [x.clone() for x in t]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        return fa.paged_plan(*t, page, max_tokens, seq_lens_out=t[1], free_state_out=t[4], error=err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(t, first):
        x.copy_(y)
    err.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots, cu, _, _ = step()
    seen = 0
    for _ in range(4):
        graph.replay()
        ref = oracle.paged_plan(table, lens, delta, ring, state, page, max_tokens)
        seen |= ref["error"]
        table, lens, ring, state = (ref[n] for n in ("block_table", "seq_lens", "free_pages",
                                                     "free_state"))
        assert np.array_equal(slots.cpu().numpy(), ref["slots"])
        assert np.array_equal(cu.cpu().numpy(), ref["cu"])
        for x, want in zip((t[0], t[1], t[3], t[4]), (table, lens, ring, state)):
            assert np.array_equal(x.cpu().numpy(), want)
        assert int(err) == seen


def test_decode_with_the_widest_table():
    """A table of 2^30 keys per request, where the line of blocks is measured in
    units of several."""
    rng = np.random.default_rng(9)
    page, width, dim = 65536, 16384, 32
    lens = np.array([70000, 5, 0, 131072, 1000, 65536, 1] + [300] * 57)
    pages = sum(-(-int(n) // page) for n in lens)
    cache = [torch.from_numpy(rng.standard_normal((pages * page, 2, dim), np.float32)).to(torch.bfloat16)
             .view(pages, page, 2, dim) for _ in range(2)]
    table, _ = make_table(rng, lens, page, pages, width)
    q = torch.from_numpy(rng.standard_normal((len(lens), 4, dim)).astype(np.float32)).to(torch.bfloat16)
    ref = oracle.paged_decode(f64(q), f64(cache[0]), f64(cache[1]), table, lens, 0.2)
    kd, vd = (x.to(DEV) for x in cache)
    y, top, total = fa.paged_decode(q.to(DEV), kd, vd, dev(table), dev(lens, torch.int32), 0.2,
                                    stats=True)
    check_decode(ref, float(cache[1].float().abs().max()), dim, "bf16", y, top, total)


def test_two_graphs_replayed_at_once():
    runs = []
    for seed, lens in ((0, [2000, 1500]), (1, [900, 3000, 12])):
        args, ref, cache = decode_inputs(seed, lens)
        args = (*args[:3], F.pad(args[3], (0, 3000), value=-1), *args[4:])   # cut and joined
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        fa.paged_decode(*args, stream=stream)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y = fa.paged_decode(*args)[0]
        runs.append((graph, stream, y, ref, float(cache[1].float().abs().max()), args))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, y, ref, v_max, _ in runs:
        check_decode(ref, v_max, 64, "bf16", y)


def test_statistics_feed_the_backward():
    """A decoding step's y and statistics are those that fa_varlen_bwd takes:
    the gradients of that one row agree with the packed backward's."""
    torch.manual_seed(1)
    heads, heads_kv, dim, page, length = 4, 2, 64, 16, 45
    k, v = (torch.randn(length, heads_kv, dim, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    q, dy = (torch.randn(1, heads, dim, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    kc, vc = (torch.zeros(4, page, heads_kv, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = dev(np.array([[2, 0, 3]], np.int32))
    j = torch.arange(length, device=DEV)
    fa.paged_write(k, v, table[0].long()[j // page] * page + j % page, kc, vc)
    y, top, total = fa.paged_decode(q, kc, vc, table, dev([length], torch.int32), 0.125, stats=True)
    dq, dk, dv = fa.bwd(q, k, v, dy, y, top, total, [1], [length], 0.125, BIG, BIG)
    ref = oracle.varlen_forward(f64(q), f64(k), f64(v), [1], [length], 0.125, BIG, BIG)
    grads = oracle.varlen_backward(f64(q), f64(k), f64(v), f64(dy), *ref, [1], [length], 0.125, BIG, BIG)
    for got, want in zip((dq, dk, dv), grads):
        assert np.abs(f64(got) - want).max() <= 2e-2 * np.abs(want).max()


def test_refusals_on_the_device():
    a, _, _ = decode_inputs(0, [20, 30])
    q, k, v, table, lens, scale = a
    for bad in (dict(y=torch.empty(2, 8, 32, dtype=q.dtype, device=DEV)),
                dict(softmax_max=torch.empty(2, 8, device=DEV)),
                dict(workspace=torch.empty(4096, dtype=torch.uint8)),
                dict(error=torch.zeros(1, dtype=torch.int64, device=DEV))):
        with pytest.raises(ValueError):
            fa.paged_decode(*a, **bad)
    wide = torch.full((2, 4096), -1, dtype=torch.int32, device=DEV)
    with pytest.raises(fa.FaError, match="WORKSPACE"):
        fa.paged_decode(q, k, v, wide, lens, scale,
                        workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        fa.paged_decode(q.float(), k, v, table, lens, scale)
    with pytest.raises(ValueError):
        fa.paged_decode(q, k, v, table, lens.long(), scale)
    with pytest.raises(ValueError):
        fa.paged_decode(q.transpose(0, 1), k, v, table, lens, scale)
    with pytest.raises(fa.FaError, match="INVALID"):
        fa.paged_decode(q[:, :7].contiguous(), k, v, table, lens, scale)
