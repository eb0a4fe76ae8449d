"""Measured cases of the paged cache's further operators: attention of a chunk of
new tokens per request over the cache, and the care of its pages: rows forked
and ended, pages copied, and a pool compacted to fewer pages.

Each has its plain form here in elementary torch operations; with ``own`` set
``run`` makes the calls of ``varlen_flashattention_backward_gb300.binding``.
Lengths and sources come from the case alone (``lens_seed``), so that the work of
a case is known without its inputs; every value comes from the seed."""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
UNBOUNDED = 2 ** 31 - 1


def _extend(name, **kw):
    c = dict(op="extend", dtype="bf16", batch=1, heads=32, heads_kv=8, dim=128, page=16, min_new=1,
             max_new=1, min_past=0, max_past=0, cross=False, window=UNBOUNDED, layout="NHD",
             stats=False, pad=0, lens_seed=1)
    c.update(kw, name=name)
    return c


def _copy(name, **kw):
    c = dict(op="copy", dtype="bf16", copies=64, skipped=0.0, num_pages=4096, heads_kv=8, dim=128,
             page=16, layout="NHD")
    c.update(kw, name=name)
    return c


def _fork(name, **kw):
    c = dict(op="fork", groups=16, width=4, beams=True, page=16, min_len=1, max_len=1024,
             tail=64, end_share=0.0, spare=1024, lens_seed=1)
    c.update(kw, name=name)
    return c


def _compact(name, **kw):
    c = dict(op="compact", batch=64, width=4, page=16, min_len=1, max_len=1024, tail=64,
             pool=2.0, keep=1.2, lens_seed=1)
    c.update(kw, name=name)
    return c


def listed():
    return [
        # The smallest call: a few fp32 tokens behind one short request.
        _extend("extend-fp32-short", dtype="fp32", heads=2, heads_kv=2, dim=64, min_new=7, max_new=7,
                min_past=94, max_past=94, stats=True),
        # Checking a draft: a serving batch, five tokens each, lengths as ragged
        # as those of a decoding batch.
        _extend("extend-draft", batch=64, min_new=5, max_new=5, min_past=1024, max_past=8192,
                lens_seed=2),
        # One chunk of a long prompt behind what is cached of it.
        _extend("extend-chunk", min_new=2048, max_new=2048, min_past=30000, max_past=30000, page=64,
                stats=True),
        # Fresh prompts of the training benchmark's size: up to 4096 tokens each,
        # nothing cached.
        _extend("extend-prompts", batch=16, min_new=128, max_new=4096, lens_seed=3),
        # A mixed step: most requests answer with one token, some bring a chunk,
        # under a sliding window; fp16, head dim 64, head-major pages of an odd
        # size, rows of padding behind the last request.
        _extend("extend-mixed", dtype="fp16", batch=61, heads=32, heads_kv=4, dim=64, page=24,
                min_new=1, max_new=512, min_past=0, max_past=16384, window=4096, layout="HND",
                stats=True, pad=100, lens_seed=4),
        # Cross attention: decoder tokens over an encoder's states, one key head
        # per query head, every key seen by every row.
        _extend("extend-cross", batch=8, heads=16, heads_kv=16, dim=96, page=100, min_new=100,
                max_new=500, min_past=1000, max_past=1500, cross=True, lens_seed=5),
        # What a step of beam search copies: half-filled last pages.
        _copy("copy-beams", copies=64, skipped=0.5),
        # What a compaction copies.
        _copy("copy-many", copies=8192, num_pages=20000, layout="HND"),
        # One step of beam search: 16 prompts, four beams each.
        _fork("fork-beams"),
        # 128 long prompts, forked into eight samples each; some are ended.
        _fork("fork-samples", groups=128, width=8, beams=False, min_len=1000, max_len=8192,
              end_share=0.1, spare=4096, lens_seed=2),
        # A small pool cut to three fifths.
        _compact("compact-small"),
        # A serving pool of half a million pages.
        _compact("compact-large", batch=1024, width=1, min_len=1, max_len=8192, tail=8192,
                 lens_seed=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "extend", "extend", "copy", "fork", "compact"])
    page = rng.choice([1, 5, 8, 16, 16, 24, 32, 64, 100, 128, 256])
    seed = rng.randrange(1 << 20)
    dim = rng.choice([32, 64, 64, 96, 128, 128, 128, 192])
    heads_kv = rng.choice([1, 2, 4, 5, 8, 8, 16, 32])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    layout = rng.choice(["NHD", "HND"])
    wide = 4 if dtype == "fp32" else 2
    if op == "extend":
        group = min(rng.choice([1, 1, 2, 4, 4, 7, 8, 16, 32]), 256 // heads_kv)
        heads = heads_kv * group
        cross = rng.random() < 0.2
        # Half of the largest case's products; a tenth of that in fp32.
        flops = 2.5e11 if wide == 2 else 2.5e10
        new = _log(rng, 1, 4096)
        past = _log(rng, 1, 65536)
        most = min(flops / (4.0 * new * (past + new) * heads * dim),
                   float(1 << 30) / ((past + new) * heads_kv * dim * wide))
        if most < 1:
            past = max(1, int(past * most))
            new = max(1, min(new, int(flops / (4.0 * (past + new) * heads * dim))))
            most = 1
        batch = _log(rng, 1, max(1, min(256, int(most))))
        made = _extend("", dtype=dtype, batch=batch, heads=heads, heads_kv=heads_kv, dim=dim, page=page,
                       min_new=rng.choice([0, 1, new]), max_new=new,
                       min_past=rng.choice([0, past // 2, past]), max_past=past, cross=cross,
                       window=UNBOUNDED if cross else rng.choice([UNBOUNDED, UNBOUNDED, past // 3]),
                       layout=layout, stats=rng.random() < 0.5, pad=rng.choice([0, 0, new]),
                       lens_seed=seed)
    elif op == "copy":
        size = page * heads_kv * dim * wide
        copies = _log(rng, 1, max(2, min(65536, (1 << 28) // size)))
        made = _copy("", dtype=dtype, copies=copies, skipped=rng.choice([0.0, 0.5, 0.9]),
                     num_pages=2 * copies + rng.randrange(50), heads_kv=heads_kv, dim=dim, page=page,
                     layout=layout)
    elif op == "fork":
        width = rng.choice([1, 2, 4, 5, 8, 16])
        groups = _log(rng, 1, 1024 // width)
        longest = _log(rng, 1, max(1, min(8192, (1 << 18) * page // (groups * width))))
        made = _fork("", groups=groups, width=width, beams=rng.random() < 0.6, page=page,
                     min_len=rng.choice([0, 1, longest]), max_len=longest, tail=rng.choice([1, 30, 400]),
                     end_share=rng.choice([0.0, 0.1, 0.5]), spare=2 * groups * width + rng.randrange(3),
                     lens_seed=seed)
    else:
        width = rng.choice([1, 1, 4])
        groups = _log(rng, 1, 1024 // width)
        longest = _log(rng, 1, max(1, min(8192, (1 << 18) * page // (groups * width))))
        made = _compact("", batch=groups * width, width=width, page=page,
                        min_len=rng.choice([0, 1, longest]), max_len=longest, tail=rng.choice([1, 30, 400]),
                        pool=rng.choice([1.0, 1.5, 3.0]), keep=rng.choice([1.0, 1.1, 1.4]),
                        lens_seed=seed)
    del made["name"]
    return made


# ---------------------------------------------------------------------------
# Lengths, sources and work
# ---------------------------------------------------------------------------

def _ceil(a, b):
    return -(-a // b)


def _rows(c):
    """(new tokens, length) of each request."""
    r = np.random.RandomState(c["lens_seed"])
    new = r.randint(c["min_new"], c["max_new"] + 1, c["batch"]).astype(np.int64)
    if c["op"] == "extend" and c["window"] != UNBOUNDED and c["batch"] > 8:
        new[r.rand(c["batch"]) < 0.8] = min(1, c["max_new"])     # a mixed step
    new[0] = c["max_new"]
    past = r.randint(c["min_past"], c["max_past"] + 1, c["batch"]).astype(np.int64)
    return new, past if c["cross"] else past + new


def _seen(c):
    """Per request: pairs of query and key, and keys that any row sees."""
    pairs, keys = 0, []
    for n, length in zip(*(x.tolist() for x in _rows(c))):
        if n == 0:
            keys.append(0)
            continue
        if c["cross"]:
            pairs += n * length
            keys.append(length)
            continue
        pos = np.arange(length - n, length, dtype=np.int64)
        first = np.maximum(0, pos - c["window"])
        pairs += int((pos + 1 - first).sum())
        keys.append(int(length - first[0]))
    return pairs, np.array(keys, np.int64)


def _held(c):
    """Rows that share prompts, `width` to a prompt: (length of the shared whole
    pages, length) of each row, in tokens."""
    r = np.random.RandomState(c["lens_seed"])
    width = c["width"]
    groups = c["groups"] if c["op"] == "fork" else c["batch"] // width
    prompt = r.randint(c["min_len"], c["max_len"] + 1, groups).astype(np.int64)
    if width > 1:
        shared = np.repeat(prompt // c["page"] * c["page"], width)
        length = np.repeat(prompt, width) + r.randint(0, c["tail"] + 1, groups * width)
    else:
        shared, length = np.zeros(groups, np.int64), prompt
    if c["op"] == "fork" and not c["beams"]:
        # Only the first row of each group holds anything yet.
        first = np.arange(groups * width) % width == 0
        length = np.where(first, np.repeat(prompt, width), 0)
        shared = np.zeros_like(shared)
    return shared, length


def _sources(c):
    r = np.random.RandomState(c["lens_seed"] + 7)
    rows = c["groups"] * c["width"]
    first = np.arange(rows) // c["width"] * c["width"]
    source = first + (r.randint(0, c["width"], rows) if c["beams"] else 0)
    ended = np.repeat(r.rand(c["groups"]) < c["end_share"], c["width"])
    return np.where(ended, -1, source).astype(np.int32)


def _page_counts(c):
    """Pages in the rows' tables, distinct pages, table width."""
    shared, length = _held(c)
    have = _ceil(length, c["page"])
    own_pages = have - shared // c["page"]
    first = np.arange(len(have)) % c["width"] == 0
    return have, int(own_pages.sum() + (shared // c["page"])[first].sum())


def _pool(c):
    """(num_pages, new_pages) of a compaction."""
    _, used = _page_counts(c)
    new = max(1, int(used * c["keep"]))
    return max(new + 1, int(used * c["pool"] * c["keep"])), new


def work(c):
    if c["op"] == "extend":
        wide = 4 if c["dtype"] == "fp32" else 2
        pairs, keys = _seen(c)
        rows = int(_rows(c)[0].sum()) * c["heads"]
        return {"bytes": 2 * int(keys.sum()) * c["heads_kv"] * c["dim"] * wide
                + 2 * rows * c["dim"] * wide + 4 * int(_ceil(keys, c["page"]).sum())
                + 12 * c["batch"] + (64 * rows if c["stats"] else 0),
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "copy":
        wide = 4 if c["dtype"] == "fp32" else 2
        moved = c["copies"] - int(c["copies"] * c["skipped"])
        return {"bytes": 4 * moved * c["page"] * c["heads_kv"] * c["dim"] * wide + 8 * c["copies"],
                "flops": 0}
    have, _ = _page_counts(c)
    if c["op"] == "fork":
        source = _sources(c)
        rows = np.arange(len(source))
        moved = int(have[source[(source >= 0) & (source != rows)]].sum())
        kept = np.bincount(source[source >= 0], minlength=len(source))
        return {"bytes": 8 * moved + 12 * int(have[kept != 1].sum()) + 20 * len(source) + 32, "flops": 0}
    pages, new = _pool(c)
    return {"bytes": 8 * int(have.sum()) + 4 * c["batch"] + 4 * (pages - int(have.sum())) + 8 * new + 32
            + 8 * min(new, pages - new), "flops": 0}


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


def _shared_table(c, g, num_pages):
    """Rows whose prompts share their whole pages, page ids in random order, -1
    behind a row's pages; how many further rows hold each page; the rest."""
    shared, length = _held(c)
    page, width = c["page"], c["width"]
    have, common = _ceil(length, page), shared // page
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    rows = len(have)
    first = np.arange(rows) // width * width
    # Each group's common pages, then each row's own.
    group_base = np.cumsum(np.where(first == np.arange(rows), common, 0)) - common[first]
    own_base = group_base[-1] + common[-1] + np.cumsum(have - common) - (have - common)
    j = torch.arange(max(1, int(have.max())), device=DEV)
    to = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)[:, None]  # noqa: E731
    at = torch.where(j < to(common), to(group_base) + j, to(own_base) + j - to(common))
    table = torch.where(j < to(have), order[at.clamp(0, num_pages - 1)], -1)
    shares = torch.zeros(num_pages, dtype=torch.int32, device=DEV)
    held = table[table >= 0].long()
    shares.scatter_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    used = int((own_base + have - common)[-1]) if rows else 0
    return (table.contiguous(), torch.from_numpy(length).to(DEV, torch.int32), (shares - 1).clamp(min=0),
            order[used:])


def _ring(g, free, num_pages):
    head = int(torch.randint(num_pages, (1,), generator=g, device=DEV))
    ring = torch.full((num_pages,), -1, dtype=torch.int32, device=DEV)
    ring[(head + torch.arange(len(free), device=DEV)) % num_pages] = free
    return ring, torch.tensor([head, len(free)], dtype=torch.int64, device=DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    error = torch.zeros(1, dtype=torch.int32, device=DEV)
    if c["op"] == "extend":
        dtype = DTYPES[c["dtype"]]
        new, lens = _rows(c)
        have = _ceil(lens, c["page"])
        num_pages = int(have.sum()) + 3
        order = torch.randperm(num_pages, generator=g, device=DEV)
        n = torch.from_numpy(have).to(DEV)
        j = torch.arange(max(1, int(have.max())), device=DEV)
        at = ((n.cumsum(0) - n)[:, None] + j).clamp(max=num_pages - 1)
        rows = int(new.sum()) + c["pad"]
        cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).to(DEV)
        state = {"case": c, "q": _randn(g, (rows, c["heads"], c["dim"]), dtype),
                 "k_pages": _cache(g, c, num_pages, dtype), "v_pages": _cache(g, c, num_pages, dtype),
                 "block_table": torch.where(j < n[:, None], order[at], -1).to(torch.int32),
                 "seq_lens": torch.from_numpy(lens).to(DEV, torch.int32), "cu": cu,
                 "scale": 1.0 / math.sqrt(c["dim"]), "y": torch.zeros(rows, c["heads"], c["dim"],
                                                                       dtype=dtype, device=DEV)}
        if c["stats"]:
            state["max"] = torch.zeros(rows, c["heads"], 8, device=DEV)
            state["sum"] = torch.zeros(rows, c["heads"], 8, device=DEV)
        return state
    if c["op"] == "copy":
        dtype = DTYPES[c["dtype"]]
        n, copies = c["num_pages"], c["copies"]
        order = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        start, end = order[:copies].clone(), order[copies:2 * copies].clone()
        none = torch.randperm(copies, generator=g, device=DEV)[:int(copies * c["skipped"])]
        start[none], end[none] = -1, -1
        return {"case": c, "k_pages": _cache(g, c, n, dtype), "v_pages": _cache(g, c, n, dtype),
                "copy_from": start, "copy_to": end, "error": error}
    num_pages = _page_counts(c)[1] + c["spare"] if c["op"] == "fork" else _pool(c)[0]
    table, lens, shares, free = _shared_table(c, g, max(1, num_pages))
    ring, pool = _ring(g, free, max(1, num_pages))
    state = {"case": c, "block_table": table, "seq_lens": lens, "shares": shares, "free_pages": ring,
             "free_state": pool, "error": error}
    if c["op"] == "fork":
        state["source"] = torch.from_numpy(_sources(c)).to(DEV)
    return state


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain_extend(s):
    c = s["case"]
    h, d, page = c["heads_kv"], c["dim"], c["page"]
    out = [torch.zeros_like(s["y"])]
    if c["stats"]:
        out += [torch.zeros_like(s["max"]), torch.zeros_like(s["sum"])]
    at = 0
    for b, (n, length) in enumerate(zip(*(x.tolist() for x in _rows(c)))):
        if n == 0 or length == 0:
            if c["stats"]:
                out[1][at:at + n] = -math.inf
            at += n
            continue
        q = s["q"][at:at + n].float().reshape(n, h, -1, d).permute(1, 2, 0, 3) * s["scale"]
        table = s["block_table"][b, :_ceil(length, page)].long()
        k = s["k_pages"][table].flatten(0, 1)[:length].float().permute(1, 2, 0)      # [h, d, keys]
        v = s["v_pages"][table].flatten(0, 1)[:length].float().transpose(0, 1)       # [h, keys, d]
        score = torch.matmul(q.reshape(h, -1, d), k).reshape(h, -1, n, length)
        if not c["cross"]:
            pos = torch.arange(length - n, length, device=DEV)[:, None]
            j = torch.arange(length, device=DEV)
            score.masked_fill_((j > pos) | (j < pos - c["window"]), -math.inf)
        top = score.amax(-1, keepdim=True)
        e = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
        total = e.sum(-1, keepdim=True)
        y = torch.matmul(e.reshape(h, -1, length), v).reshape(h, -1, n, d)
        y = y / torch.where(total == 0, 1.0, total)
        out[0][at:at + n] = y.permute(2, 0, 1, 3).reshape(n, -1, d).to(out[0].dtype)
        if c["stats"]:
            out[1][at:at + n] = top.permute(2, 0, 1, 3).reshape(n, -1, 1)
            out[2][at:at + n] = total.permute(2, 0, 1, 3).reshape(n, -1, 1)
        at += n
    return tuple(out)


def _plain_copy(s):
    kept = s["copy_from"] >= 0
    start, end = s["copy_from"][kept].long(), s["copy_to"][kept].long()
    s["k_pages"][end] = s["k_pages"][start]
    s["v_pages"][end] = s["v_pages"][start]
    return s["k_pages"], s["v_pages"]


def _plain_fork(s):
    c = s["case"]
    p, n = c["page"], s["free_pages"].numel()
    table, lens, source = s["block_table"], s["seq_lens"].long(), s["source"].long()
    batch, width = table.shape
    head, count = s["free_state"][0], s["free_state"][1]
    rows = torch.arange(batch, device=DEV)
    there = source >= 0
    safe = source.clamp(min=0)
    kept = torch.zeros_like(lens).scatter_add_(0, safe, there.long())
    have, full = (lens + p - 1) // p, lens // p
    # The row that goes on with a half-filled last page: its owner, or the first
    # of its forks.
    heir = torch.full_like(lens, batch).scatter_reduce_(0, safe, torch.where(there, rows, batch), "amin")
    heir = torch.where(source == rows, rows, heir)
    need = there & (have > full)[safe] & (heir[safe] != rows)
    upto = need.long().cumsum(0)
    taken = upto[-1]
    fine = taken <= count
    need = need & fine
    new_page = s["free_pages"][(head + upto - 1).clamp(min=0) % n]
    # Holders of each page.
    j = torch.arange(width, device=DEV)
    change = torch.where(j < full[:, None], (kept - 1)[:, None],
                         torch.where((j < have[:, None]) & (kept == 0)[:, None], -1, 0))
    change = torch.where(fine, change, 0).to(torch.int32)
    shares = s["shares"].scatter_add(0, table.long().clamp(min=0).flatten(),
                                     torch.where(j < have[:, None], change, 0).flatten())
    gone = shares < 0
    rank = gone.long().cumsum(0) - 1
    ring = torch.cat([s["free_pages"], s["free_pages"].new_zeros(1)])
    ring[torch.where(gone, (head + count + rank) % n, n)] = torch.arange(n, dtype=torch.int32, device=DEV)
    # Tables.
    moves = there & (source != rows) & fine
    new = torch.where(moves[:, None] & (j < have[safe][:, None]), table[safe], table)
    last = torch.gather(table, 1, full[:, None].clamp(max=width - 1))[:, 0]
    new = torch.where(need[:, None] & (j == full[safe][:, None]), new_page[:, None], new)
    s["block_table"].copy_(new)
    s["seq_lens"].copy_(torch.where(fine, torch.where(there, lens[safe], 0), lens))
    s["shares"].copy_(shares.clamp(min=0))
    s["free_pages"].copy_(ring[:n])
    taken = torch.where(fine, taken, 0)
    s["free_state"].copy_(torch.stack([(head + taken) % n, count - taken + gone.sum()]))
    s["error"].bitwise_or_((~fine).to(torch.int32))
    return (torch.where(need, last[safe], -1).to(torch.int32), torch.where(need, new_page, -1),
            s["block_table"], s["seq_lens"], s["shares"], s["free_pages"], s["free_state"], s["error"])


def _plain_compact(s):
    c = s["case"]
    n, new = s["free_pages"].numel(), _pool(c)[1]
    table, lens = s["block_table"], s["seq_lens"].long()
    j = torch.arange(table.shape[1], device=DEV)
    live = j < ((lens + c["page"] - 1) // c["page"])[:, None]
    used = torch.zeros(n + 1, dtype=torch.bool, device=DEV)
    used[torch.where(live, table, n).long().flatten()] = True
    used = used[:n]
    i = torch.arange(n, device=DEV)
    free = torch.zeros(n + 1, dtype=torch.bool, device=DEV)
    free[torch.where((i - s["free_state"][0]) % n < s["free_state"][1], s["free_pages"], n).long()] = True
    low = free[:n] & ~used & (i < new)
    high = used & (i >= new)
    need, room = high.sum(), low.sum()
    limit = min(new, n - new)
    start = torch.full((limit + 1,), -1, dtype=torch.int32, device=DEV)
    end = start.clone()
    start[torch.where(high, high.long().cumsum(0) - 1, limit)] = i.to(torch.int32)
    rank = low.long().cumsum(0) - 1
    end[torch.where(low & (rank < need), rank, limit)] = i.to(torch.int32)
    ring = torch.full((new + 1,), -1, dtype=torch.int32, device=DEV)
    ring[torch.where(low & (rank >= need), rank - need, new)] = i.to(torch.int32)
    start, end, ring = start[:limit], end[:limit], ring[:new]
    where_to = torch.cat([i.to(torch.int32), i.new_zeros(1, dtype=torch.int32)])
    where_to[torch.where(start >= 0, start, n).long()] = end
    shares = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    shares[where_to[:n].long()] = torch.where(used, s["shares"], 0)
    shares[torch.where(start >= 0, end, n).long()] = s["shares"][start.long().clamp(min=0)]
    out = torch.where(live, where_to[table.long().clamp(min=0)], table)
    return start, end, out, ring, torch.stack([need - need, room - need]), shares[:new], s["error"]


def run(s):
    c = s["case"]
    if not own:
        return {"extend": _plain_extend, "copy": _plain_copy, "fork": _plain_fork,
                "compact": _plain_compact}[c["op"]](s)
    from varlen_flashattention_backward_gb300 import binding as fa
    if c["op"] == "extend":
        unseen = UNBOUNDED if c["cross"] else 0
        y, top, total = fa.paged_extend(s["q"], s["k_pages"], s["v_pages"], s["block_table"],
                                        s["seq_lens"], s["cu"], s["scale"], pre_tokens=c["window"],
                                        next_tokens=unseen, y=s["y"], softmax_max=s.get("max"),
                                        softmax_sum=s.get("sum"))
        return (y, top, total) if c["stats"] else (y,)
    if c["op"] == "copy":
        fa.paged_copy(s["k_pages"], s["v_pages"], s["copy_from"], s["copy_to"], error=s["error"])
        return s["k_pages"], s["v_pages"]
    if c["op"] == "fork":
        start, end, _, _ = fa.paged_fork(s["block_table"], s["seq_lens"], s["source"], s["shares"],
                                         s["free_pages"], s["free_state"], c["page"],
                                         seq_lens_out=s["seq_lens"], free_state_out=s["free_state"],
                                         error=s["error"])
        return (start, end, s["block_table"], s["seq_lens"], s["shares"], s["free_pages"],
                s["free_state"], s["error"])
    start, end, table, ring, pool, shares = fa.paged_compact(
        s["block_table"], s["seq_lens"], s["free_pages"], s["free_state"], c["page"], _pool(c)[1],
        shares=s["shares"], error=s["error"])
    return start, end, table, ring, pool, shares, s["error"]


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _exact_extend(s, c):
    shape = (s["q"].shape[0], c["heads"])
    y = torch.zeros(*shape, c["dim"], dtype=torch.float64, device=DEV)
    top = torch.zeros(shape, dtype=torch.float64, device=DEV)
    total = torch.zeros(shape, dtype=torch.float64, device=DEV)
    group = c["heads"] // c["heads_kv"]
    new, lens = _rows(c)
    start = np.concatenate([[0], np.cumsum(new)])
    for b, length in enumerate(lens.tolist()):
        j = torch.arange(length, device=DEV)
        page = s["block_table"][b, j // c["page"]].long()
        for first in range(0, int(new[b]), 512):
            rows = slice(int(start[b]) + first, int(start[b]) + min(first + 512, int(new[b])))
            pos = length - int(new[b]) + first + torch.arange(rows.stop - rows.start, device=DEV)[:, None]
            seen = torch.ones_like(pos, dtype=torch.bool) if c["cross"] else j <= pos
            if not c["cross"] and c["window"] < length:
                seen = seen & (pos - j <= c["window"])
            for n in range(c["heads"]):
                if n % group == 0:
                    k = s["k_pages"][page, j % c["page"], n // group].double()
                    v = s["v_pages"][page, j % c["page"], n // group].double()
                if length == 0:
                    top[rows, n] = -math.inf
                    continue
                logits = s["scale"] * (s["q"][rows, n].double() @ k.T)
                logits = torch.where(seen, logits, -math.inf)
                m = logits.max(-1).values
                e = torch.exp(logits - m[:, None])
                top[rows, n], total[rows, n] = m, e.sum(-1)
                y[rows, n] = (e @ v) / e.sum(-1, keepdim=True)
    if not c["stats"]:
        return (y,)
    return y, top[..., None].repeat(1, 1, 8), total[..., None].repeat(1, 1, 8)


def _exact_copy(s, c):
    out = []
    pairs = [(a, b) for a, b in zip(s["copy_from"].tolist(), s["copy_to"].tolist()) if a >= 0]
    for pages in (s["k_pages"], s["v_pages"]):
        cache = pages.double().contiguous()
        for a, b in pairs:
            cache[b].copy_(pages[a])
        out.append(cache)
    return tuple(out)


def _exact_fork(s, c):
    """One row after the other, on the host."""
    p = c["page"]
    table, ring = s["block_table"].cpu().numpy().copy(), s["free_pages"].cpu().numpy().copy()
    lens, source = s["seq_lens"].tolist(), s["source"].tolist()
    head, count = s["free_state"].tolist()
    n, batch = len(ring), len(lens)
    holders = {}
    held = [list(table[b, :_ceil(lens[b], p)]) for b in range(batch)]
    after, copies, taken = [], [], 0
    went_on = {b for b in range(batch) if source[b] == b}
    for b in range(batch):
        if source[b] < 0:
            after.append([])
            continue
        row = list(held[source[b]])
        if source[b] != b and lens[source[b]] % p:
            if source[b] in went_on:
                copies.append((b, row[-1], ring[(head + taken) % n]))
                row[-1] = copies[-1][2]
                taken += 1
            else:
                went_on.add(source[b])
        after.append(row)
    start, end = np.full(batch, -1, np.int32), np.full(batch, -1, np.int32)
    shares = s["shares"].cpu().numpy().copy()
    if taken > count:
        return (start, end, table, np.array(lens, np.int32), shares, ring, np.array([head, count]),
                np.array([1], np.int32))
    for b, a, z in copies:
        start[b], end[b] = a, z
    for row in after:
        for page in row:
            holders[page] = holders.get(page, 0) + 1
    before = {page for row in held for page in row}
    for page in before | set(holders):
        shares[page] = max(0, holders.get(page, 0) - 1)
    given = sorted(page for page in before if page not in holders)
    for i, page in enumerate(given):
        ring[(head + count + i) % n] = page
    for b, row in enumerate(after):
        table[b, :len(row)] = row
    return (start, end, table, np.array([lens[x] if x >= 0 else 0 for x in source], np.int32), shares,
            ring, np.array([(head + taken) % n, count - taken + len(given)]), np.array([0], np.int32))


def _exact_compact(s, c):
    n, new = s["free_pages"].numel(), _pool(c)[1]
    table, ring = s["block_table"].cpu().numpy(), s["free_pages"].cpu().numpy()
    head, count = s["free_state"].tolist()
    shares = s["shares"].cpu().numpy()
    have = [_ceil(x, c["page"]) for x in s["seq_lens"].tolist()]
    used = sorted({int(x) for b, k in enumerate(have) for x in table[b, :k]})
    free = sorted(int(ring[(head + i) % n]) for i in range(count))
    low = [x for x in free if x < new]
    moved = [x for x in used if x >= new]
    to = dict(zip(moved, low))
    limit = min(new, n - new)
    start, end = np.full(limit, -1, np.int32), np.full(limit, -1, np.int32)
    start[:len(moved)], end[:len(moved)] = moved, low[:len(moved)]
    out = table.copy()
    for b, k in enumerate(have):
        out[b, :k] = [to.get(int(x), int(x)) for x in table[b, :k]]
    pages, held = np.full(new, -1, np.int32), np.zeros(new, np.int32)
    left = low[len(moved):]
    pages[:len(left)] = left
    for x in used:
        held[to.get(x, x)] = shares[x]
    return start, end, out, pages, np.array([0, len(left)]), held, np.array([0], np.int32)


def exact(c, seed):
    s = prepare(c, seed)
    return {"extend": _exact_extend, "copy": _exact_copy, "fork": _exact_fork,
            "compact": _exact_compact}[c["op"]](s, c)
