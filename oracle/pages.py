"""Page operations of a paged cache, one entry after the other, on the host.

A pool is a list of arrays [num_blocks, page_size, ...]; tables as
block_table [B, max_blocks] (a negative entry holds no page), ctx_lens [B] and
refcount [num_blocks] (0 or less: free). Every function changes its arrays in
place and returns the set of error names it would flag. Test infrastructure:
it shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def _free_pages(refcount):
    return [int(p) for p in np.flatnonzero(np.asarray(refcount) <= 0)]


def copy_pages(pool, src, dst):
    blocks = pool[0].shape[0]
    errors, pairs = set(), []
    for i, (s, d) in enumerate(zip(src, dst)):
        if s < 0 or d < 0:
            continue
        if s >= blocks or d >= blocks:
            errors.add("BLOCK")
        elif s != d:
            pairs.append((i, int(s), int(d)))
    before = [c.copy() for c in pool]
    for i, s, d in pairs:
        if any(d == d2 for j, _, d2 in pairs if j < i) or any(d == s2 for _, s2, _ in pairs):
            errors.add("ALIAS")
            continue
        for c, old in zip(pool, before):
            c[d] = old[s]
    return errors


def fork(pool, page, block_table, ctx_lens, refcount, parents, children):
    B, M = block_table.shape
    blocks = len(refcount)
    free = _free_pages(refcount)
    errors, named, full_pool = set(), set(), False
    old_bt, old_ctx = block_table.copy(), ctx_lens.copy()
    for p, c in zip(parents, children):
        if p < 0 or c < 0:
            continue
        if p >= B or c >= B:
            errors.add("ROW")
            continue
        bad = set()
        if c in named or old_ctx[c] != 0 or old_bt[c, 0] >= 0:
            bad.add("ALIAS")
        named.add(c)
        ctx = int(old_ctx[p])
        if ctx < 0 or ctx > M * page:
            bad.add("CTX")
        if not bad:
            held = old_bt[p, :-(-ctx // page)]
            if ((held < 0) | (held >= blocks)).any():
                bad.add("BLOCK")
        errors |= bad
        if bad or ctx == 0:
            continue
        full, part = divmod(ctx, page)
        if part and (full_pool or not free):
            full_pool = True
            errors.add("PAGES")
            continue
        row = np.full(M, -1, block_table.dtype)
        row[:full] = old_bt[p, :full]
        for x in row[:full]:
            refcount[x] += 1
        if part:
            new = free.pop(0)
            row[full] = new
            refcount[new] = 1
            for a in pool:
                a[new, :part] = a[old_bt[p, full], :part]
        block_table[c] = row
        ctx_lens[c] = ctx
    return errors


def reserve(page, block_table, refcount, rows, tokens):
    B, M = block_table.shape
    free = _free_pages(refcount)
    errors, named, shut = set(), set(), False
    for r, n in zip(rows, tokens):
        if r < 0:
            continue
        if r >= B:
            errors.add("ROW")
            continue
        again = r in named
        named.add(r)
        if again:
            errors.add("ALIAS")
            continue
        if n < 0 or n > M * page:
            errors.add("CTX")
            continue
        empty = [j for j in range(-(-int(n) // page)) if block_table[r, j] < 0]
        if not empty:
            continue
        if shut or len(empty) > len(free):
            shut = True
            errors.add("PAGES")
            continue
        for j in empty:
            block_table[r, j] = free.pop(0)
            refcount[block_table[r, j]] = 1
    return errors


def free(block_table, ctx_lens, refcount, rows):
    errors = set()
    for r in rows:
        if r < 0:
            continue
        if r >= block_table.shape[0]:
            errors.add("ROW")
            continue
        for j, p in enumerate(block_table[r]):
            if p < 0:
                continue
            block_table[r, j] = -1
            if p >= len(refcount) or refcount[p] <= 0:
                errors.add("BLOCK")
            else:
                refcount[p] -= 1
        ctx_lens[r] = 0
    return errors


def compact(pool, block_table, refcount):
    """Returns (errors, live pages)."""
    errors = set()
    blocks = len(refcount)
    live = int((refcount > 0).sum())
    holes = [p for p in range(live) if refcount[p] <= 0]
    movers = [p for p in range(live, blocks) if refcount[p] > 0]
    to = dict(zip(movers, holes))
    for s, d in to.items():
        for a in pool:
            a[d] = a[s]
        refcount[d], refcount[s] = refcount[s], 0
    for r in range(block_table.shape[0]):
        for j, p in enumerate(block_table[r]):
            if p >= live:
                if int(p) in to:
                    block_table[r, j] = to[int(p)]
                else:
                    errors.add("BLOCK")
    return errors, live
