"""Sequences that share pages, and sequences cut back (oracle): plain loops over a `chunk.Pool` with
`refs`, the holders of each page beside the first.  Paging: "长程 agent 把显存撑爆以后", section
"四、为什么进不了 vLLM 一类的引擎".
"""
import numpy as np

from .chunk import BAD_LENGTH, CAPACITY, PAGE

BAD_INDEX = 1


def _consistent(pool, ctx, held):
    maxp = pool.block_table.shape[1]
    return 0 <= ctx <= maxp * PAGE and -(-ctx // PAGE) <= held <= maxp


def fork(pool, refs, src):
    """(from_seq, from_page, flags); the pool and refs change."""
    B = len(src)
    from_seq, from_page = np.full((2, B), -1, dtype=np.int64)
    flags, asked, free0 = 0, 0, len(pool.free)
    for b in range(B):
        s = int(src[b])
        if s < 0:
            continue
        if s >= B or src[s] >= 0:
            flags |= BAD_INDEX
            continue
        n = int(pool.ctx[s])
        if pool.n_pages[b] != 0 or not _consistent(pool, n, pool.n_pages[s]):
            flags |= BAD_LENGTH
            continue
        full = n // PAGE
        if n % PAGE:
            if not 0 <= pool.block_table[s, full] < pool.num_pages:
                flags |= BAD_INDEX
                continue
            asked += 1
            if asked > free0:
                flags |= CAPACITY
                continue
            pool.block_table[b, full] = pool.free.pop()
            from_page[b] = pool.block_table[s, full]
        for p in range(full):
            pool.block_table[b, p] = pool.block_table[s, p]
            refs[pool.block_table[s, p]] += 1
        from_seq[b] = s
        pool.n_pages[b] = -(-n // PAGE)
        pool.ctx[b] = n
    return from_seq, from_page, flags


def truncate(pool, refs, keep):
    """(from_seq, from_page, flags); refs may be None (no shared pages)."""
    B = len(keep)
    from_page = np.full(B, -1, dtype=np.int64)
    flags, asked, free0 = 0, 0, len(pool.free)
    before = None if refs is None else list(refs)          # what is shared as the call begins
    let_go = []                                            # pages in order of (sequence, logical page)
    for b in range(B):
        if keep[b] < 0:
            continue
        if not _consistent(pool, int(pool.ctx[b]), int(pool.n_pages[b])):
            flags |= BAD_LENGTH
            continue
        n = min(int(keep[b]), int(pool.ctx[b]))
        after, held = -(-n // PAGE), int(pool.n_pages[b])
        if n % PAGE:
            last = int(pool.block_table[b, after - 1])
            if not 0 <= last < pool.num_pages:
                flags |= BAD_INDEX
                continue
            own = refs is not None and before[last] > 0
            if own:
                asked += 1
                if asked > free0:
                    flags |= CAPACITY
                    continue
                let_go.append(last)
                pool.block_table[b, after - 1] = pool.free.pop()
            if own or n < pool.ctx[b]:
                from_page[b] = last
        let_go += [int(p) for p in pool.block_table[b, after:held]]
        pool.ctx[b], pool.n_pages[b] = n, after
    freed = []
    for i, page in enumerate(let_go):
        if not 0 <= page < pool.num_pages:
            flags |= BAD_INDEX
        elif refs is None:
            freed.append(page)
        else:
            refs[page] -= 1
            if refs[page] < 0:                             # its last holder, and the last of this call
                refs[page] = 0
                freed.append(page)
    pool.free += freed[::-1]
    return np.full(B, -1), from_page, flags


def carry(pool, k, v, meta, from_seq, from_page):
    """One layer's k, v [pages][Hkv][16][D] and meta [B][maxp][Hkv][2][D] (or None) follow."""
    for b in range(len(from_seq)):
        full, rows = divmod(int(pool.ctx[b]), PAGE)
        if from_seq[b] >= 0 and meta is not None:
            meta[b, :full] = meta[from_seq[b], :full]
        if from_page[b] >= 0 and rows:
            to, old = pool.block_table[b, full], from_page[b]
            k[to, :, :rows], v[to, :, :rows] = k[old, :, :rows], v[old, :, :rows]
            if meta is not None:
                meta[b, full, :, 0] = k[to, :, :rows].min(1)
                meta[b, full, :, 1] = k[to, :, :rows].max(1)
