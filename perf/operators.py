"""Measured cases of the paged-cache operators: the plan (block tables and
slot maps from request lengths), the write of new key/value rows, and the
attention of one new token over the cache.

Each has its plain form here in elementary torch operations; with ``own`` set
``run`` makes the calls of ``varlen_flashattention_backward_gb300.binding``.
Request lengths come from the case alone (``lens_seed``), so that the work of
a case is known without its inputs; every value comes from the seed."""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
UNBOUNDED = 2 ** 31 - 1

# Bits of the error word.
EXHAUSTED, ROW_FULL, ROWS, BAD_PAGE, BAD_LENGTH, BAD_POOL = 1, 2, 4, 8, 16, 32


def _plan(name, **kw):
    c = dict(op="plan", batch=64, page=16, max_pages=256, min_len=1, max_len=4096, grow_min=1,
             grow_max=1, grow_share=1.0, release_share=0.0, spare=64, max_tokens=64, lens_seed=1)
    c.update(kw, name=name)
    return c


def _write(name, **kw):
    c = dict(op="write", dtype="bf16", tokens=64, heads_kv=8, dim=128, page=16, num_pages=4096,
             layout="NHD", fused=True, pad=0)
    c.update(kw, name=name)
    return c


def _decode(name, **kw):
    c = dict(op="decode", dtype="bf16", batch=1, heads=32, heads_kv=8, dim=128, page=16,
             min_len=2048, max_len=2048, window=UNBOUNDED, layout="NHD", stats=False, empty=0,
             lens_seed=1)
    c.update(kw, name=name)
    return c


def listed():
    return [
        # One decoding step of a serving batch: every request grows by one
        # token, one in sixteen takes a page.
        _plan("plan-step"),
        # Turnover of a large batch: prompts of up to 4096 tokens come in,
        # a fifth of the requests give all their pages back.
        _plan("plan-turnover", batch=256, page=16, max_pages=1024, max_len=8192, grow_max=4096,
              grow_share=0.5, release_share=0.2, spare=40000, max_tokens=400000, lens_seed=2),
        # The step's new rows, sliced out of a fused q/k/v projection.
        _write("write-step"),
        # The packed prompts of the training benchmark's size (T = 39332).
        _write("write-prompts", tokens=39332, num_pages=4096, layout="HND"),
        # The smallest call: two fp32 heads over one short request.
        _decode("decode-fp32-short", dtype="fp32", heads=2, heads_kv=2, dim=64, min_len=101,
                max_len=101, stats=True),
        # A single user's reply: one request, grouped heads.
        _decode("decode-one"),
        # Long documents, one key head per query head.
        _decode("decode-long", batch=2, heads=8, heads_kv=8, min_len=31111, max_len=32768, page=64),
        # The training benchmark's ragged lengths as a decoding batch.
        _decode("decode-ragged", batch=16, min_len=128, max_len=4096, stats=True, lens_seed=3),
        # A full serving batch: bandwidth counts.
        _decode("decode-serving", batch=128, min_len=1024, max_len=8192, lens_seed=4),
        # Sliding window over long requests.
        _decode("decode-window", batch=4, heads=16, heads_kv=16, min_len=16384, max_len=16384,
                window=4096, page=128),
        # fp16, head dim 64, an odd page size, head-major pages, short
        # requests and a batch padded with empty ones.
        _decode("decode-fp16-short", dtype="fp16", batch=61, heads=32, heads_kv=4, dim=64,
                min_len=1, max_len=1021, page=24, layout="HND", empty=5, stats=True, lens_seed=5),
        # One key head for all query heads, the widest head dim.
        _decode("decode-shared-key", batch=32, heads=32, heads_kv=1, dim=192, min_len=2000,
                max_len=8192, page=64, lens_seed=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "decode", "decode"])
    page = rng.choice([1, 5, 8, 16, 16, 24, 32, 64, 100, 128, 256])
    seed = rng.randrange(1 << 20)
    if op == "plan":
        batch = _log(rng, 1, 2048)
        grow = _log(rng, 1, max(1, min(4096, 200000 // batch)))
        longest = _log(rng, 1, 8192)
        width = min(8192, (longest + grow) // page + 1)
        case = dict(batch=batch, page=page, max_pages=max(1, width), min_len=0,
                    max_len=min(longest, width * page), grow_max=grow,
                    grow_share=rng.choice([0.3, 0.9, 1.0]),
                    release_share=rng.choice([0.0, 0.1, 0.5]),
                    spare=rng.choice([0, 3, batch, batch * (grow // page + 1)]),
                    max_tokens=max(1, int(batch * grow * rng.choice([0.4, 1.0, 1.1]))),
                    lens_seed=seed)
        made = _plan("", **case)
    else:
        dim = rng.choice([32, 64, 64, 96, 128, 128, 128, 192])
        heads_kv = rng.choice([1, 2, 4, 5, 8, 8, 16, 32])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        layout = rng.choice(["NHD", "HND"])
        wide = 4 if dtype == "fp32" else 2
        if op == "write":
            tokens = _log(rng, 1, max(2, min(65536, 39332 * 2048 // (heads_kv * dim * wide))))
            made = _write("", dtype=dtype, tokens=tokens, heads_kv=heads_kv, dim=dim, page=page,
                          num_pages=tokens // page + 1 + rng.randrange(50), layout=layout,
                          fused=rng.random() < 0.5, pad=rng.choice([0, 0, tokens // 3]))
        else:
            group = rng.choice([1, 1, 2, 4, 4, 7, 8, 16, 32])
            group = min(group, 256 // heads_kv)
            batch = _log(rng, 1, 256)
            # Keys in all, so that no draw costs more than the serving batch.
            most = min(65536, 1 << 20, (1 << 30) // (heads_kv * dim * wide * batch))
            longest = _log(rng, 1, max(2, most))
            made = _decode("", dtype=dtype, batch=batch, heads=heads_kv * group, heads_kv=heads_kv,
                           dim=dim, page=page, min_len=rng.choice([1, max(1, longest // 2), longest]),
                           max_len=longest,
                           window=rng.choice([UNBOUNDED, UNBOUNDED, UNBOUNDED, longest // 3]),
                           layout=layout, stats=rng.random() < 0.5,
                           empty=rng.choice([0, 0, 0, batch // 4]), lens_seed=seed)
    del made["name"]
    return made


# ---------------------------------------------------------------------------
# Lengths and work
# ---------------------------------------------------------------------------

def _ceil(a, b):
    return -(-a // b)


def _lens(c):
    r = np.random.RandomState(c["lens_seed"])
    lens = r.randint(c["min_len"], c["max_len"] + 1, c["batch"]).astype(np.int64)
    lens[0] = c["max_len"]
    if c.get("empty"):
        lens[-c["empty"]:] = 0
    return lens


def _deltas(c):
    r = np.random.RandomState(c["lens_seed"] + 7)
    b = c["batch"]
    kind = r.rand(b)
    delta = np.where(kind < c["grow_share"], r.randint(c["grow_min"], c["grow_max"] + 1, b), 0)
    gone = r.rand(b) < c["release_share"]
    # Most of these end (every page back), some drop a few rejected tokens.
    return np.where(gone, np.where(r.rand(b) < 0.8, -(1 << 30), -r.randint(1, 9, b)), delta)


def _keys(c):
    return np.minimum(_lens(c), c["window"] + 1)


def work(c):
    if c["op"] == "plan":
        lens, delta = _lens(c), _deltas(c)
        have = _ceil(lens, c["page"])
        moved = int(np.abs(_ceil(np.maximum(lens + delta, 0), c["page"]) - have).sum())
        return {"bytes": 8 * c["max_tokens"] + 8 * moved + 20 * c["batch"] + 40, "flops": 0}
    wide = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "write":
        return {"bytes": 4 * (c["tokens"] - c["pad"]) * c["heads_kv"] * c["dim"] * wide
                + 8 * c["tokens"], "flops": 0}
    keys = int(_keys(c).sum())
    rows = c["batch"] * c["heads"]
    pages = int(_ceil(_keys(c), c["page"]).sum())
    return {"bytes": 2 * keys * c["heads_kv"] * c["dim"] * wide + 2 * rows * c["dim"] * wide
            + 4 * pages + 4 * c["batch"] + (64 * rows if c["stats"] else 0),
            "flops": 4 * keys * c["heads"] * c["dim"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _cache(g, c, num_pages, dtype):
    """A cache [pages, tokens, heads, dim]; head-major pages are a view."""
    shape = (num_pages, c["page"], c["heads_kv"], c["dim"])
    if c["layout"] == "HND":
        shape = (num_pages, c["heads_kv"], c["page"], c["dim"])
        return _randn(g, shape, dtype).transpose(1, 2)
    return _randn(g, shape, dtype)


def _table(g, pages_of, width, num_pages):
    """Rows of distinct page ids in random order; -1 behind a row's pages."""
    order = torch.randperm(num_pages, generator=g, device=DEV)
    n = torch.from_numpy(np.ascontiguousarray(pages_of)).to(DEV)
    first = n.cumsum(0) - n
    j = torch.arange(width, device=DEV)
    at = (first[:, None] + j).clamp(max=num_pages - 1)
    table = torch.where(j < n[:, None], order[at], -1).to(torch.int32)
    return table, order[int(pages_of.sum()):].to(torch.int32)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    if c["op"] == "plan":
        lens = _lens(c)
        have = _ceil(lens, c["page"])
        num_pages = max(1, int(have.sum()) + c["spare"])
        table, free = _table(g, have, c["max_pages"], num_pages)
        head = int(torch.randint(num_pages, (1,), generator=g, device=DEV))
        ring = torch.full((num_pages,), -1, dtype=torch.int32, device=DEV)
        ring[(head + torch.arange(len(free), device=DEV)) % num_pages] = free
        return {"case": c, "block_table": table,
                "seq_lens": torch.from_numpy(lens).to(DEV, torch.int32),
                "delta": torch.from_numpy(_deltas(c)).to(DEV, torch.int32), "free_pages": ring,
                "free_state": torch.tensor([head, len(free)], dtype=torch.int64, device=DEV),
                "error": torch.zeros(1, dtype=torch.int32, device=DEV)}
    dtype = DTYPES[c["dtype"]]
    if c["op"] == "write":
        n, t = c["num_pages"], c["tokens"]
        kc, vc = _cache(g, c, n, dtype), _cache(g, c, n, dtype)
        h, d = c["heads_kv"], c["dim"]
        if c["fused"]:
            # Rows of a fused projection: 2 h query heads, then keys, then values.
            qkv = _randn(g, (t, 4 * h, d), dtype)
            k, v = qkv[:, 2 * h:3 * h], qkv[:, 3 * h:]
        else:
            k, v = _randn(g, (t, h, d), dtype), _randn(g, (t, h, d), dtype)
        # Whole pages in random order, as a plan hands them out; padding rows
        # of a fixed-size step behind them.
        order = torch.randperm(n, generator=g, device=DEV)[:_ceil(t, c["page"])]
        slots = (order[:, None] * c["page"] + torch.arange(c["page"], device=DEV)).flatten()[:t]
        if c["pad"]:
            slots[t - c["pad"]:] = -1
        return {"case": c, "k": k, "v": v, "slots": slots.contiguous(), "k_pages": kc, "v_pages": vc}
    lens = _lens(c)
    have = _ceil(lens, c["page"])
    num_pages = int(have.sum()) + 3
    table, _ = _table(g, have, max(1, int(have.max())), num_pages)
    return {"case": c, "q": _randn(g, (c["batch"], c["heads"], c["dim"]), dtype),
            "k_pages": _cache(g, c, num_pages, dtype), "v_pages": _cache(g, c, num_pages, dtype),
            "block_table": table, "seq_lens": torch.from_numpy(lens).to(DEV, torch.int32),
            "scale": 1.0 / math.sqrt(c["dim"])}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain_plan(s):
    c = s["case"]
    p, n = c["page"], s["free_pages"].numel()
    lens, delta = s["seq_lens"].long(), s["delta"].long()
    head, count = s["free_state"][0], s["free_state"][1]
    rows = delta.clamp(min=0)
    cu = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    target = (lens + delta).clamp(min=0)
    most = c["max_pages"] * p
    sound = (lens >= 0) & (lens <= most)
    grow = sound & (delta > 0)
    in_row = target <= most
    ask = grow & in_row & (cu[1:] <= c["max_tokens"])
    have, want = (lens + p - 1) // p, (target + p - 1) // p
    need = torch.where(ask, want - have, 0)
    upto = need.cumsum(0)
    granted = ask & ((need == 0) | (upto <= count))
    shrink = sound & (delta < 0)
    give = torch.where(shrink, have - want, 0)
    taken, given = torch.where(granted, need, 0).sum(), give.sum()
    whole = (head >= 0) & (head < n) & (count >= 0) & (count <= n) & (count + given <= n)
    granted, shrink = granted & whole, shrink & whole
    # Pages out of the ring, and back behind its end.
    j = torch.arange(c["max_pages"], device=DEV)
    out = granted[:, None] & (j >= have[:, None]) & (j < want[:, None])
    at = (head + (upto - need)[:, None] + j - have[:, None]) % n
    ring = torch.cat([s["free_pages"], s["free_pages"].new_zeros(1)])
    table = torch.where(out, ring[at.clamp(0, n - 1)], s["block_table"])
    back = shrink[:, None] & (j >= want[:, None]) & (j < have[:, None])
    to = (head + count + (give.cumsum(0) - give)[:, None] + j - want[:, None]) % n
    ring[torch.where(back, to, n)] = table
    s["block_table"].copy_(table)
    s["free_pages"].copy_(ring[:n])
    # Slots of the packed rows.
    t = torch.arange(c["max_tokens"], device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=c["batch"] - 1)
    pos = lens[b] + t - cu[b]
    used = granted[b] & (t < cu[-1])
    page = table[b, (pos // p).clamp(0, c["max_pages"] - 1)].long()
    fine = (page >= 0) & (page < n)
    slots = torch.where(used & fine, page * p + pos % p, -1)
    error = (EXHAUSTED * (ask & (need > 0) & (upto > count)).any() + ROW_FULL * (grow & ~in_row).any()
             + ROWS * (grow & in_row & (cu[1:] > c["max_tokens"])).any()
             + BAD_PAGE * (used & ~fine).any() + BAD_LENGTH * (~sound).any() + BAD_POOL * ~whole)
    s["error"].bitwise_or_(error.to(torch.int32))
    new_lens = torch.where(granted | shrink, target, lens).to(torch.int32)
    state = torch.stack([(head + taken) % n, count - taken + given])
    return (slots, cu, new_lens, torch.where(whole, state, s["free_state"]), s["block_table"],
            s["free_pages"], s["error"])


def _plain_write(s):
    p = s["case"]["page"]
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    s["k_pages"][at // p, at % p] = s["k"][kept]
    s["v_pages"][at // p, at % p] = s["v"][kept]
    return s["k_pages"], s["v_pages"]


def _plain_decode(s):
    c = s["case"]
    b, h, d = c["batch"], c["heads_kv"], c["dim"]
    length = s["block_table"].shape[1] * c["page"]
    lens = s["seq_lens"].long()[:, None]
    j = torch.arange(length, device=DEV)
    allowed = (j < lens) & (j >= lens - 1 - c["window"])
    table = s["block_table"].long().clamp(min=0)
    q = s["q"].float().reshape(b, h, -1, d) * s["scale"]
    k = s["k_pages"][table].float().reshape(b, length, h, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1))
    del k
    score = torch.where(allowed[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    v = torch.where(allowed[:, :, None, None], s["v_pages"][table].float().reshape(b, length, h, d), 0.0)
    y = torch.matmul(e, v.permute(0, 2, 1, 3)) / torch.where(total == 0, 1.0, total)
    y = y.reshape(b, c["heads"], d).to(s["q"].dtype)
    if not c["stats"]:
        return (y,)
    lanes = (b, c["heads"], 8)
    return (y, top.reshape(b, -1, 1).expand(lanes).contiguous(),
            total.reshape(b, -1, 1).expand(lanes).contiguous())


def run(s):
    c = s["case"]
    if not own:
        return {"plan": _plain_plan, "write": _plain_write, "decode": _plain_decode}[c["op"]](s)
    from varlen_flashattention_backward_gb300 import binding as fa
    if c["op"] == "plan":
        slots, cu, lens, state = fa.paged_plan(
            s["block_table"], s["seq_lens"], s["delta"], s["free_pages"], s["free_state"],
            c["page"], c["max_tokens"], error=s["error"])
        return slots, cu, lens, state, s["block_table"], s["free_pages"], s["error"]
    if c["op"] == "write":
        fa.paged_write(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"])
        return s["k_pages"], s["v_pages"]
    y, top, total = fa.paged_decode(s["q"], s["k_pages"], s["v_pages"], s["block_table"],
                                    s["seq_lens"], s["scale"], pre_tokens=c["window"],
                                    stats=c["stats"])
    return (y, top, total) if c["stats"] else (y,)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _exact_plan(s, c):
    """One request after the other, on the host."""
    p, n = c["page"], s["free_pages"].numel()
    table, ring = s["block_table"].cpu().numpy().copy(), s["free_pages"].cpu().numpy().copy()
    lens, delta = s["seq_lens"].tolist(), s["delta"].tolist()
    head, count = s["free_state"].tolist()
    slots, cu, new = np.full(c["max_tokens"], -1, np.int64), [0], list(lens)
    taken = asked = given = error = 0
    for b, (length, d) in enumerate(zip(lens, delta)):
        row = cu[-1]
        cu.append(row + max(d, 0))
        have = _ceil(length, p)
        if d > 0:
            if length + d > c["max_pages"] * p:
                error |= ROW_FULL
            elif cu[-1] > c["max_tokens"]:
                error |= ROWS
            else:
                need = _ceil(length + d, p) - have
                asked += need
                if need and asked > count:
                    error |= EXHAUSTED
                    continue
                for i in range(need):
                    table[b, have + i] = ring[(head + taken + i) % n]
                taken += need
                at = np.arange(length, length + d)
                slots[row:row + d] = table[b, at // p].astype(np.int64) * p + at % p
                new[b] = length + d
        elif d < 0:
            new[b] = max(0, length + d)
            for i in range(_ceil(new[b], p), have):
                ring[(head + count + given) % n] = table[b, i]
                given += 1
    return (slots, np.array(cu), np.array(new, np.int32),
            np.array([(head + taken) % n, count - taken + given]), table, ring,
            np.array([error], np.int32))


def _exact_write(s, c):
    out = []
    slots = s["slots"].cpu().numpy()
    for rows, pages in ((s["k"], s["k_pages"]), (s["v"], s["v_pages"])):
        cache = pages.double().cpu().numpy()
        from_rows = rows.double().cpu().numpy()
        for t, slot in enumerate(slots):
            if slot >= 0:
                cache[slot // c["page"], slot % c["page"]] = from_rows[t]
        out.append(cache)
    return tuple(out)


def _exact_decode(s, c):
    shape = (c["batch"], c["heads"])
    y = torch.zeros(*shape, c["dim"], dtype=torch.float64, device=DEV)
    top = torch.full(shape, -math.inf, dtype=torch.float64, device=DEV)
    total = torch.zeros(shape, dtype=torch.float64, device=DEV)
    group = c["heads"] // c["heads_kv"]
    for b, length in enumerate(_lens(c).tolist()):
        first = max(0, length - 1 - c["window"])
        if first >= length:
            continue
        pos = torch.arange(first, length, device=DEV)
        page = s["block_table"][b, pos // c["page"]].long()
        k = s["k_pages"][page, pos % c["page"]].double().transpose(0, 1)
        v = s["v_pages"][page, pos % c["page"]].double().transpose(0, 1)
        q = s["q"][b].double().reshape(c["heads_kv"], group, c["dim"])
        logits = s["scale"] * torch.bmm(q, k.transpose(1, 2))
        m = logits.max(-1).values
        e = torch.exp(logits - m[..., None])
        top[b], total[b] = m.flatten(), e.sum(-1).flatten()
        y[b] = (torch.bmm(e, v) / e.sum(-1, keepdim=True)).reshape(c["heads"], c["dim"])
    if not c["stats"]:
        return (y,)
    return y, top[..., None].repeat(1, 1, 8), total[..., None].repeat(1, 1, 8)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "plan":
        return _exact_plan(s, c)
    if c["op"] == "write":
        return _exact_write(s, c)
    return _exact_decode(s, c)
