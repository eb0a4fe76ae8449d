"""The paged-cache operators in numpy, one request after the other: the plan
in whole numbers, the write as copies, single-token attention in float64.
Definitions: the comments of ``fa_paged_*`` in ``include/fa_varlen.h``.
"""

from __future__ import annotations

import numpy as np

EXHAUSTED, ROW_FULL, ROWS, BAD_PAGE, BAD_LENGTH, BAD_POOL, BAD_SLOT = 1, 2, 4, 8, 16, 32, 64


def _pages(tokens, page_size):
    return -(-int(tokens) // page_size)


def paged_plan(block_table, seq_lens, delta, free_pages, free_state, page_size, max_tokens):
    """dict of slots, cu, seq_lens, free_state, block_table, free_pages and
    error after one plan; the arguments are left as they were."""
    table, ring = np.array(block_table), np.array(free_pages)
    batch, width = table.shape
    n = len(ring)
    most = width * page_size
    head, count = (int(x) for x in free_state)
    lens = [int(x) for x in seq_lens]
    delta = [int(x) for x in delta]
    cu = np.concatenate([[0], np.cumsum([max(d, 0) for d in delta])]).astype(np.int64)
    slots = np.full(max_tokens, -1, np.int64)
    error = 0
    # What each request gives back or asks for, before anything changes.
    give = [0] * batch
    need = [None] * batch          # None: not asking
    for b, (length, d) in enumerate(zip(lens, delta)):
        if not 0 <= length <= most:
            error |= BAD_LENGTH
        elif d < 0:
            give[b] = _pages(length, page_size) - _pages(max(0, length + d), page_size)
        elif d > 0 and length + d > most:
            error |= ROW_FULL
        elif d > 0 and cu[b + 1] > max_tokens:
            error |= ROWS
        elif d > 0:
            need[b] = _pages(length + d, page_size) - _pages(length, page_size)
    whole = 0 <= head < n and 0 <= count <= n and count + sum(give) <= n
    out = dict(slots=slots, cu=cu, seq_lens=np.array(lens, np.int32),
               free_state=np.array([head, count], np.int64), block_table=table, free_pages=ring)
    asked = taken = 0
    before = ring.copy()
    for b in range(batch):
        if need[b] is None:
            continue
        asked += need[b]
        if need[b] and asked > count:
            error |= EXHAUSTED
            continue
        if not whole:
            continue
        have = _pages(lens[b], page_size)
        for i in range(need[b]):
            table[b, have + i] = before[(head + taken + i) % n]
        taken += need[b]
        for i in range(delta[b]):
            pos = lens[b] + i
            page = int(table[b, pos // page_size])
            if 0 <= page < n:
                slots[cu[b] + i] = page * page_size + pos % page_size
            else:
                error |= BAD_PAGE
        out["seq_lens"][b] = lens[b] + delta[b]
    if whole:
        given = 0
        for b in range(batch):
            if not 0 <= lens[b] <= most or delta[b] >= 0:
                continue
            target = max(0, lens[b] + delta[b])
            for i in range(give[b]):
                ring[(head + count + given) % n] = block_table[b][_pages(target, page_size) + i]
                given += 1
            out["seq_lens"][b] = target
        out["free_state"][:] = ((head + taken) % n, count - taken + given)
    else:
        error |= BAD_POOL
    out["error"] = error
    return out


def paged_write(k, v, slots, k_pages, v_pages):
    """(k_pages, v_pages, error) after the write; caches [pages, tokens, heads,
    dim]."""
    kc, vc = np.array(k_pages), np.array(v_pages)
    page_size, error = kc.shape[1], 0
    for t, slot in enumerate(int(s) for s in slots):
        if slot >= kc.shape[0] * page_size:
            error |= BAD_SLOT
        elif slot >= 0:
            kc[slot // page_size, slot % page_size] = k[t]
            vc[slot // page_size, slot % page_size] = v[t]
    return kc, vc, error


def paged_decode(q, k_pages, v_pages, block_table, seq_lens, scale, pre_tokens=2 ** 31 - 1):
    """dict of y [batch, heads, dim], max and sum [batch, heads] in float64,
    error, and `weight`: [batch, heads] the largest sum of |q_d k_d| * |scale|
    over a row's keys (the size of what cancels in its scores)."""
    q = np.asarray(q, np.float64)
    batch, heads, dim = q.shape
    num_pages, page_size, heads_kv, _ = k_pages.shape
    group = heads // heads_kv
    most = block_table.shape[1] * page_size
    y = np.zeros((batch, heads, dim))
    top, total = np.full((batch, heads), -np.inf), np.zeros((batch, heads))
    weight, error = np.zeros((batch, heads)), 0
    for b in range(batch):
        length = int(seq_lens[b])
        if not 0 <= length <= most:
            error |= BAD_LENGTH
            length = min(max(length, 0), most)
        pos = np.arange(max(0, length - 1 - pre_tokens), max(length, 0))
        pages = np.asarray(block_table[b], np.int64)[pos // page_size]
        fine = (pages >= 0) & (pages < num_pages)
        if not fine.all():
            error |= BAD_PAGE
        pos, pages = pos[fine], pages[fine]
        if len(pos) == 0:
            continue
        k = np.asarray(k_pages[pages, pos % page_size], np.float64)    # [keys, heads_kv, dim]
        v = np.asarray(v_pages[pages, pos % page_size], np.float64)
        for n in range(heads):
            kn, vn = k[:, n // group], v[:, n // group]
            s = scale * (kn @ q[b, n])
            m = s.max()
            weight[b, n] = abs(scale) * (np.abs(kn) @ np.abs(q[b, n])).max()
            if m == -np.inf:
                continue
            e = np.exp(s - m)
            top[b, n], total[b, n] = m, e.sum()
            y[b, n] = (e @ vn) / e.sum()
    return dict(y=y, max=top, sum=total, error=error, weight=weight)


def paged_extend(q, k_pages, v_pages, block_table, seq_lens, cu_tokens, scale,
                 pre_tokens=2 ** 31 - 1, next_tokens=0):
    """dict of y [tokens, heads, dim], max and sum [tokens, heads] in float64, error;
    `weight`: [tokens, heads] the largest sum of |q_d k_d| * |scale| over a row's
    keys, `spread`: [tokens, heads, dim] the weighted mean of |v|, `keys`: [tokens] how
    many keys a row sees; `owned`: [tokens] whether a request owns the row (others are
    left as they were, and 0 here)."""
    q = np.asarray(q, np.float64)
    tokens, heads, dim = q.shape
    num_pages, page_size, heads_kv, _ = k_pages.shape
    group = heads // heads_kv
    most = block_table.shape[1] * page_size
    y, spread = np.zeros((tokens, heads, dim)), np.zeros((tokens, heads, dim))
    top, total = np.full((tokens, heads), -np.inf), np.zeros((tokens, heads))
    weight, seen = np.zeros((tokens, heads)), np.zeros(tokens, np.int64)
    owned, error = np.zeros(tokens, bool), 0
    descends = (np.diff(cu_tokens) < 0).any()      # requests could share rows: nothing is done
    for b in range(len(seq_lens)):
        start = min(max(int(cu_tokens[b]), 0), tokens)
        end = min(max(int(cu_tokens[b + 1]), start), tokens)
        if (start, end) != (int(cu_tokens[b]), int(cu_tokens[b + 1])):
            error |= ROWS
        length = int(seq_lens[b])
        if not 0 <= length <= most:
            error |= BAD_LENGTH
            length = min(max(length, 0), most)
        if descends:
            continue
        n = end - start
        owned[start:end] = True
        if n == 0:
            continue
        pos = length - n + np.arange(n)
        lo = np.clip(pos - pre_tokens, 0, length)
        hi = np.maximum(np.clip(pos + next_tokens + 1, 0, length), lo)
        first, last = int(lo.min()), int(hi.max())
        j = np.arange(first, max(first, last))
        j = j[((j >= lo[:, None]) & (j < hi[:, None])).any(0)]      # (none between empty windows)
        pages = np.asarray(block_table[b], np.int64)[j // page_size]
        fine = (pages >= 0) & (pages < num_pages)
        if not fine.all():
            error |= BAD_PAGE
        j, pages = j[fine], pages[fine]
        k = np.asarray(k_pages[pages, j % page_size], np.float64)      # [keys, heads_kv, dim]
        v = np.asarray(v_pages[pages, j % page_size], np.float64)
        allowed = (j >= lo[:, None]) & (j < hi[:, None])
        seen[start:end] = allowed.sum(1)
        for h in range(heads if len(j) else 0):
            kn, vn, qn = k[:, h // group], v[:, h // group], q[start:end, h]
            with np.errstate(invalid="ignore", over="ignore"):
                s = np.where(allowed, scale * (qn @ kn.T), -np.inf)
                m = s.max(1)
                e = np.where(allowed, np.exp(s - np.where(m == -np.inf, 0, m)[:, None]), 0)
                weight[start:end, h] = abs(scale) * np.where(allowed, np.abs(qn) @ np.abs(kn).T, 0).max(1)
                # What a row does not see counts as 0, also where it is not finite.
                use = e.any(1)
                sums = np.where(use, e.sum(1), 1)[:, None]
                for row in range(n):
                    if use[row] or np.isnan(e[row]).any():
                        y[start + row, h] = e[row, allowed[row]] @ vn[allowed[row]] / sums[row]
                        spread[start + row, h] = e[row, allowed[row]] @ np.abs(vn[allowed[row]]) / sums[row]
                top[start:end, h], total[start:end, h] = m, e.sum(1)
    return dict(y=y, max=top, sum=total, error=error, weight=weight, spread=spread, keys=seen, owned=owned)
