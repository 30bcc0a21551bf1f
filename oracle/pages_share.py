"""Shared pages in plain Python: giving blocks up, forking, compacting, copying.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code
with the library.  Works on copies; flags have the library's meaning.
"""
from __future__ import annotations

import numpy as np

BAD_POS, BAD_SEQ, BAD_BLOCK, FREE_FULL, NO_BLOCKS = 1, 2, 4, 32, 64


def free(table, bs, refs, seqs, free_ids, count, keep_lo=None, keep_hi=None):
    """(table, refs, free_ids, count, flags) after the sequences gave up their blocks outside [keep_lo, keep_hi)."""
    table, refs, ids, flags = table.copy(), refs.copy(), list(free_ids), 0
    S, mb = table.shape
    for i, s in enumerate(seqs):
        if not 0 <= s < S:
            flags |= BAD_SEQ
            continue
        a = 0 if keep_lo is None else int(keep_lo[i])
        b = 0 if keep_hi is None else int(keep_hi[i])
        for bi in range(mb):
            if max(bi * bs, a) < min(bi * bs + bs, b):  # a position of the block is kept
                continue
            x = int(table[s, bi])
            if x < 0:
                continue
            if x >= len(refs):
                flags |= BAD_BLOCK
                continue
            table[s, bi] = -1
            refs[x] -= 1
    dead = [b for b in range(len(refs)) if refs[b] < 0]
    if dead and (count < 0 or count + len(dead) > len(ids)):
        return table, refs, ids, count, flags | FREE_FULL
    for j, b in enumerate(dead):
        ids[count + j] = b
        refs[b] = 0
    return table, refs, ids, count + len(dead), flags


def fork(table, bs, refs, src, dst, lens, free_ids, count):
    """(table, refs, pairs, count, flags); pairs [(from, to)]."""
    old_table, old_refs = table, refs
    table, refs, flags, pairs = table.copy(), refs.copy(), 0, []
    S, mb = table.shape
    nb = len(refs)
    taken = 0
    for s, d, n in zip(src, dst, lens):
        n = int(n)
        if not (0 <= s < S and 0 <= d < S) or s == d:
            flags |= BAD_SEQ
            continue
        if not 0 <= n <= mb * bs:
            flags |= BAD_POS
            continue
        taken += n % bs > 0
    if count < 0 or count > len(free_ids) or taken > count:
        return old_table.copy(), old_refs.copy(), [], count, flags | NO_BLOCKS
    for s, d, n in zip(src, dst, lens):
        n = int(n)
        if not (0 <= s < S and 0 <= d < S) or s == d or not 0 <= n <= mb * bs:
            continue
        for bi in range(n // bs):
            x = int(old_table[s, bi])
            if not 0 <= x < nb:
                flags |= BAD_BLOCK
                x = -1
            else:
                refs[x] += 1
            table[d, bi] = x
        if n % bs:
            x, y = int(old_table[s, n // bs]), int(free_ids[count - 1 - len(pairs)])
            okx, oky = 0 <= x < nb, 0 <= y < nb
            if not okx or not oky:
                flags |= BAD_BLOCK
            table[d, n // bs] = y if oky else -1
            pairs.append((x if okx and oky else -1, -1 if not okx or not oky else y))
    return table, refs, pairs, count - taken, flags


def compact(table, refs, free_ids, count, limit=0):
    """(table, refs, free list up to count, pairs, flags)."""
    nb = len(refs)
    ids = [int(x) for x in free_ids[:max(count, 0)]]
    if count < 0 or count > len(free_ids) or len(set(ids)) != count or any(not 0 <= x < nb for x in ids):
        return table.copy(), refs.copy(), ids, [], BAD_BLOCK
    gone = set(ids)
    used = [b for b in range(nb) if b not in gone]
    limit = min(limit, nb) if limit > 0 else len(used)
    if limit < len(used):
        return table.copy(), refs.copy(), ids, [], NO_BLOCKS
    holes = [b for b in range(limit) if b in gone]
    pairs = list(zip([b for b in used if b >= limit], holes))
    new = {b: b for b in used}
    new.update(pairs)
    out = np.zeros_like(refs)
    for b in used:
        out[new[b]] = refs[b]
    t = table.copy()
    for e in np.ndindex(*t.shape):
        if 0 <= t[e] < nb:
            t[e] = new.get(int(t[e]), -1)
    left = sorted(set(range(nb)) - set(new.values()), reverse=True)
    return t, out, left, pairs, 0
