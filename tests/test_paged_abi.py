"""CPU tests of the paged entry points' argument checks.  Every call here is
refused before anything is launched; the addresses are never read."""

import ctypes
import os
import re

import pytest
import torch

from varlen_flashattention_backward_gb300 import binding as fa
from varlen_flashattention_backward_gb300 import build as fb

P = 1 << 20          # a 16-byte aligned address that no refused call reads
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    fb.build()
    fa.lib()


PLAN = dict(block_table=P, max_pages=8, table_stride=8, seq_lens=P, delta=P, batch=4, free_pages=P,
            free_state=P, num_pages=64, page_size=16, slots=P, max_tokens=64, cu_tokens=P,
            seq_lens_out=P, free_state_out=P, error=0)
WRITE = dict(k=P, v=P, k_stride=512, v_stride=512, slots=P, tokens=4, k_pages=P, v_pages=P,
             num_pages=64, page_size=16, head_num_kv=4, head_dim=128, page_stride=16 * 512,
             token_stride=512, head_stride=128, dtype=2, reserved=0, error=0)
DECODE = dict(q=P, q_stride=1024, k_pages=P, v_pages=P, num_pages=64, page_size=16,
              page_stride=16 * 512, token_stride=512, head_stride=128, block_table=P, max_pages=8,
              table_stride=8, seq_lens=P, batch=4, head_num=8, head_num_kv=4, head_dim=128, dtype=2,
              reserved=0, scale=0.1, pre_tokens=BIG, y=P, y_stride=1024, softmax_max=0,
              softmax_sum=0, error=0, workspace=P, workspace_bytes=0)


def call(name, base, **kw):
    assert set(kw) <= set(base)
    pack = {"fa_paged_plan": fa._pack_plan, "fa_paged_write": fa._pack_write,
            "fa_paged_decode": fa._pack_decode}[name]
    args = {k: v or 0 for k, v in {**base, **kw}.items()}
    return getattr(fa.lib(), name)(pack(*args.values()), None)


def test_the_structs_are_packed_as_the_header_lays_them_out():
    text = open(os.path.join(fb.INCLUDE, "fa_varlen.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, fields, base in (("plan", fa.PLAN_ARGS, PLAN), ("write", fa.WRITE_ARGS, WRITE),
                               ("decode", fa.DECODE_ARGS, DECODE)):
        assert list(base) == fields
        body = re.search(r"typedef struct \{([^}]*)\} fa_paged_%s_args;" % name, text).group(1)
        found, size = [], 0
        for declared in filter(None, (d.strip() for d in body.split(";"))):
            kind, names = re.match(r"(?:const )?(\w+)\s+(.*)", declared, re.S).groups()
            for field in names.split(","):
                found.append(field.strip().lstrip("*"))
                size += 4 if kind == "int32_t" and "*" not in field else 8
        assert found == fields
        assert fa._format(fields).size == size


@pytest.mark.parametrize("name", ["fa_paged_plan", "fa_paged_write", "fa_paged_decode"])
def test_no_arguments(name):
    assert getattr(fa.lib(), name)(None, None) == fa.FA_ERR_NULLPTR


def test_reserved_is_zero():
    assert call("fa_paged_write", WRITE, reserved=1) == fa.FA_ERR_INVALID
    assert call("fa_paged_decode", DECODE, reserved=7) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("null", ["block_table", "seq_lens", "delta", "free_pages", "free_state",
                                  "slots", "cu_tokens", "seq_lens_out", "free_state_out"])
def test_plan_null(null):
    assert call("fa_paged_plan", PLAN, **{null: None}) == fa.FA_ERR_NULLPTR


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(batch=2049), dict(num_pages=0), dict(num_pages=2 ** 31), dict(page_size=0),
    dict(page_size=65537), dict(max_pages=0), dict(max_pages=2 ** 27, table_stride=2 ** 27),
    dict(max_pages=2 ** 62, table_stride=2 ** 62), dict(table_stride=7), dict(table_stride=2 ** 62),
    dict(max_tokens=-1), dict(max_tokens=2 ** 31)])
def test_plan_invalid(bad):
    assert call("fa_paged_plan", PLAN, **bad) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("null", ["k", "v", "slots", "k_pages", "v_pages"])
def test_write_null(null):
    assert call("fa_paged_write", WRITE, **{null: None}) == fa.FA_ERR_NULLPTR


CACHE_BAD = [
    dict(num_pages=0), dict(num_pages=2 ** 31), dict(page_size=0), dict(page_size=65537),
    dict(head_dim=0), dict(head_dim=769), dict(page_stride=8191 + 2), dict(token_stride=516),
    dict(head_stride=64), dict(head_stride=132), dict(token_stride=-512), dict(page_stride=0),
    dict(page_stride=2 ** 55), dict(k_pages=P + 8), dict(v_pages=P + 2), dict(dtype=3),
    dict(dtype=-1)]


@pytest.mark.parametrize("bad", CACHE_BAD + [
    dict(head_num_kv=0), dict(head_num_kv=257), dict(tokens=-1), dict(tokens=2 ** 31),
    dict(k_stride=511), dict(v_stride=0), dict(k_stride=2 ** 61), dict(k=P + 1), dict(v=P + 1)])
def test_write_invalid(bad):
    assert call("fa_paged_write", WRITE, **bad) == fa.FA_ERR_INVALID


def test_unsupported_head_dim():
    strides = dict(page_stride=16 * 512, token_stride=512, head_stride=128)
    for d in (8, 80, 256):
        s = dict(strides, head_stride=max(128, d), token_stride=4 * max(128, d),
                 page_stride=64 * max(128, d))
        assert call("fa_paged_write", WRITE, head_dim=d, **s) == fa.FA_ERR_UNSUPPORTED
        assert call("fa_paged_decode", DECODE, head_dim=d, **s) == fa.FA_ERR_UNSUPPORTED


def test_write_of_nothing_launches_nothing():
    assert call("fa_paged_write", WRITE, tokens=0, k=None, v=None, slots=None) == fa.FA_OK
    # ... but is checked
    assert call("fa_paged_write", WRITE, tokens=0, page_size=0) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("null", ["q", "k_pages", "v_pages", "block_table", "seq_lens", "y"])
def test_decode_null(null):
    assert call("fa_paged_decode", DECODE, **{null: None}) == fa.FA_ERR_NULLPTR


def test_decode_statistics_come_together():
    assert call("fa_paged_decode", DECODE, softmax_max=P) == fa.FA_ERR_NULLPTR
    assert call("fa_paged_decode", DECODE, softmax_sum=P) == fa.FA_ERR_NULLPTR


@pytest.mark.parametrize("bad", CACHE_BAD + [
    dict(batch=0), dict(batch=2049), dict(head_num=0), dict(head_num=257, head_num_kv=1),
    dict(head_num=9), dict(head_num=2), dict(max_pages=0), dict(max_pages=9),
    dict(max_pages=2 ** 27, table_stride=2 ** 27), dict(q_stride=1023), dict(y_stride=100),
    dict(q=P + 1), dict(y=P + 1), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(workspace=P + 4)])
def test_decode_invalid(bad):
    assert call("fa_paged_decode", DECODE, **bad) == fa.FA_ERR_INVALID


def test_decode_workspace():
    out = ctypes.c_size_t(0)

    def size(batch=4, head_num=8, head_num_kv=4, head_dim=128, dtype=2, page_size=16,
             max_pages=4096, pre_tokens=BIG, out=ctypes.byref(out)):
        return fa.lib().fa_paged_decode_workspace_size(batch, head_num, head_num_kv, head_dim,
                                                       dtype, page_size, max_pages, pre_tokens, out)
    long = dict(max_pages=4096, table_stride=4096)
    assert size() == fa.FA_OK and out.value > 0
    assert call("fa_paged_decode", DECODE, workspace_bytes=out.value - 1, **long) == \
        fa.FA_ERR_WORKSPACE
    assert call("fa_paged_decode", DECODE, workspace=None, **long) == fa.FA_ERR_NULLPTR
    # few short requests need none
    assert size(max_pages=8) == fa.FA_OK and out.value == 0
    assert size(pre_tokens=100) == fa.FA_OK and out.value == 0
    assert size(out=None) == fa.FA_ERR_NULLPTR
    for bad in (dict(batch=0), dict(batch=2049), dict(head_num_kv=3), dict(dtype=9),
                dict(page_size=0), dict(max_pages=0), dict(max_pages=2 ** 27)):
        assert size(**bad) == fa.FA_ERR_INVALID
    assert size(head_dim=80) == fa.FA_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors():
    i32, i64 = torch.int32, torch.int64
    kc = torch.zeros(4, 16, 2, 64)
    table, lens = torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.paged_plan(table, lens, lens, torch.zeros(4, dtype=i32), torch.zeros(2, dtype=i64), 16, 3)
    with pytest.raises(ValueError, match="CUDA"):
        fa.paged_write(kc[0, :3], kc[0, :3], torch.zeros(3, dtype=i64), kc, kc)
    with pytest.raises(ValueError, match="CUDA"):
        fa.paged_decode(torch.zeros(3, 2, 64), kc, kc, table, lens, 0.1)


def test_binding_refuses_caches_that_do_not_match():
    a = torch.zeros(4, 16, 2, 64)
    for k, v in ((a, a.half()), (a, a[:2]), (a, a.transpose(1, 2).contiguous().transpose(1, 2)),
                 (a[..., ::2], a[..., ::2]), (a.double(), a.double()), (a[0], a[0])):
        with pytest.raises(ValueError, match="k_pages and v_pages"):
            fa.paged_write(a[0, :3], a[0, :3], torch.zeros(3, dtype=torch.int64), k, v)
