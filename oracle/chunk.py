"""Chunks of new tokens over a paged cache (oracle): the pages and rows they
get, their append with page summaries, and their attention.

Pages of 16 tokens with a token->page table follow "长程 agent 把显存撑爆以后", section
"四、为什么进不了 vLLM 一类的引擎".  The definitions are plain loops, sequence by sequence
and token by token, in float64 where numbers are computed.
"""
import numpy as np

from .attention import attend

PAGE = 16
CAPACITY, BAD_LENGTH = 2, 4


class Pool:
    """Free pages (a stack: the last is the top), each sequence's pages and length."""

    def __init__(self, num_pages, batch, max_pages):
        self.num_pages = num_pages
        self.free = list(range(num_pages - 1, -1, -1))
        self.block_table = np.full((batch, max_pages), -1, dtype=np.int64)
        self.n_pages = np.zeros(batch, dtype=np.int64)
        self.ctx = np.zeros(batch, dtype=np.int64)


def plan(pool, new_len, max_tokens):
    """(start, seq, pos, slot, flags); the pool's table, counts and stack change."""
    B, maxp = pool.block_table.shape
    start = np.zeros(B + 1, dtype=np.int64)
    seq, pos, slot = np.full((3, max_tokens), -1, dtype=np.int64)
    flags, row, asked, free0 = 0, 0, 0, len(pool.free)
    for b in range(B):
        n, ctx, held = int(new_len[b]), int(pool.ctx[b]), int(pool.n_pages[b])
        first, row = row, row + max(0, n)
        start[b], start[b + 1] = min(first, max_tokens), min(row, max_tokens)
        seq[start[b]:start[b + 1]] = b
        if n < 0 or not 0 <= ctx <= maxp * PAGE or not -(-ctx // PAGE) <= held <= maxp:
            flags |= BAD_LENGTH
            continue
        if ctx + n > maxp * PAGE or row > max_tokens:
            flags |= CAPACITY
            continue
        need = max(0, -(-(ctx + n) // PAGE) - held)
        asked += need
        if need and asked > free0:
            flags |= CAPACITY
            continue
        for p in range(held, held + need):
            pool.block_table[b, p] = pool.free.pop()
        pool.n_pages[b] += need
        for i in range(n):
            p = ctx + i
            pos[first + i] = p
            slot[first + i] = pool.block_table[b, p // PAGE] * PAGE + p % PAGE
    return start, seq, pos, slot, flags


def release(pool, done):
    """Pages of the flagged sequences back on the stack, the first on top."""
    pages = []
    for b in np.flatnonzero(done):
        pages += list(pool.block_table[b, :pool.n_pages[b]])
        pool.n_pages[b] = pool.ctx[b] = 0
    pool.free += pages[::-1]


def append(pool, k, v, meta, k_new, v_new, start, seq, pos, slot):
    """Rows into k, v [pages][Hkv][16][D] token by token; meta [B][maxp][Hkv][2][D] or None."""
    for t in range(len(slot)):
        if slot[t] < 0:
            continue
        b, p = seq[t], pos[t]
        k[slot[t] // PAGE, :, slot[t] % PAGE] = k_new[t]
        v[slot[t] // PAGE, :, slot[t] % PAGE] = v_new[t]
        if meta is not None:
            m = meta[b, p // PAGE]
            if p % PAGE == 0:
                m[:, 0] = m[:, 1] = k_new[t]
            else:
                m[:, 0] = np.minimum(m[:, 0], k_new[t])
                m[:, 1] = np.maximum(m[:, 1], k_new[t])
        pool.ctx[b] = p + 1


def chunk_attend(q, k, v, pos0, scale, window=0, sink=0, absent=()):
    """Rows q [n][G][D] at positions pos0 + i (pos0 -1: refused, they see nothing) over the
    held k, v [L][D]; keys listed in `absent` are left out.  Returns (out [n][G][D], lse [n][G])."""
    n, G, D = np.shape(q)
    out, lse = np.zeros((n, G, D)), np.full((n, G), -np.inf)
    L = len(k)
    there = np.ones(L, dtype=bool)
    there[list(absent)] = False
    for i in range(n):
        p = pos0 + i if pos0 >= 0 else -1
        see = [j for j in range(min(L, p + 1))
               if there[j] and (window == 0 or j > p - window or j < sink)]
        if see:
            out[i], lse[i] = attend(q[i], np.asarray(k)[see], np.asarray(v)[see], scale)
    return out, lse
