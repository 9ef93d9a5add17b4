"""Appends of chunks some of whose rows have no slot or are dropped, between rows that have
one: lengths, rows and page summaries are the oracle's, every time."""
import numpy as np
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se
from oracle import chunk as oc
from tests.test_gpu_chunk import BAD_INDEX, PAGE, Cache, bf16, f64, i32, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


def append_rows(c, start, seq, pos, slot, status=0, kept=None):
    """Appends the rows on both sides; `kept`: the slots that the oracle writes."""
    kn, vn = normal(c.g, len(slot), c.H, c.D), normal(c.g, len(slot), c.H, c.D)
    lengths = c.pool.ctx_len.clone()
    oc.append(c.o, c.k, c.v, c.meta, kn, vn, start, seq, pos, slot if kept is None else kept)
    chunk = se.Chunk(i32(start), i32(seq), i32(pos), i32(slot))
    meta = None if c.meta is None else c.kv.meta.clone()
    for _ in range(8):
        c.pool.ctx_len.copy_(lengths)
        if meta is not None:
            c.kv.meta.copy_(meta)
        se.se_kv_append_chunk(c.kv, bf16(kn), bf16(vn), chunk, c.B, c.ws)
        assert se.status_word(c.ws) == status
        c.check()
    c.ws[:4] = 0


def planned(c, new, pad=0):
    """start, seq, pos, slot of `new` tokens per sequence, pages taken on both sides."""
    rows = int(sum(new)) + pad
    start, seq, pos, slot, flags = oc.plan(c.o, new, rows)
    assert flags == 0
    c.pool.block_table.copy_(i32(c.o.block_table))
    c.pool.n_pages.copy_(i32(c.o.n_pages))
    c.pool.n_free.fill_(len(c.o.free))
    return start, seq, pos, slot


# (tokens held, new tokens, holes as (sequence, first page of its new tokens, pages)):
# one page, many, the first, the last, up to the next sequence, all of a sequence
PAGE_HOLES = [
    ([0], [48], [(0, 1, 1)]), ([0], [33], [(0, 1, 1)]), ([5], [100], [(0, 1, 2), (0, 5, 1)]),
    ([0, 3], [700, 20], [(0, 1, 40), (1, 0, 1)]), ([16, 0], [64, 16], [(0, 3, 1), (1, 0, 1)]),
    ([0, 7, 9], [32, 90, 5], [(0, 0, 2), (1, 1, 3), (2, 0, 1)]),
    ([1, 1], [47, 47], [(0, 2, 1), (1, 0, 1)]),
]


@pytest.mark.parametrize("pad", [0, 3, 200])
@pytest.mark.parametrize("held,new,holes", PAGE_HOLES)
def test_pages_that_were_not_found(held, new, holes, pad):
    """Rows of whole pages have no slot: the last row that has one sets the length."""
    g = np.random.default_rng([31, len(new), new[0], pad])
    c = Cache(g, len(new), 2, 64, 48, 120)
    if any(held):
        c.add(held)
    start, seq, pos, slot = planned(c, new, pad)
    for b, first, pages in holes:
        at = held[b] // PAGE + first
        slot[(seq == b) & (pos >= at * PAGE) & (pos < (at + pages) * PAGE)] = -1
    assert (slot[:start[-1]] == -1).any()
    append_rows(c, start, seq, pos, slot)


@pytest.mark.parametrize("what", ["seq", "slot", "pos"])
def test_dropped_rows_in_the_middle(what):
    """Rows dropped for a bad seq, slot or pos are no end of their sequence."""
    g = np.random.default_rng([32])
    c = Cache(g, 2, 2, 64, 40, 80)
    start, seq, pos, slot = planned(c, [200, 50], 5)
    kept = slot.copy()
    for a, z in ((16, 32), (48, 128), (200 + 16, 200 + 32)):
        kept[a:z] = -1
        (seq if what == "seq" else slot if what == "slot" else pos)[a:z] = \
            {"seq": 2, "slot": 80 * PAGE, "pos": 40 * PAGE}[what]
    append_rows(c, start, seq, pos, slot, BAD_INDEX, kept)


def test_plan_with_bad_pages_then_append():
    """Pages outside the cache met on the stack: se_chunk_plan's rows of them have no slot, and the
    append behind it commits the length of the last row that has one."""
    g = np.random.default_rng([33])
    c = Cache(g, 2, 2, 64, 8, 16, summaries=False)
    c.pool.free_pages[13:15] = i32([16, -5])             # second and third page handed out
    chunk = se.Chunk.empty(2, 90)
    se.se_chunk_plan(c.pool, i32([70, 18]), 2, chunk, c.ws_pool)
    assert se.status_word(c.ws_pool) == BAD_INDEX
    start, seq, pos, slot = (getattr(chunk, x).cpu().numpy() for x in ("start", "seq", "pos", "slot"))
    assert (slot[16:48] == -1).all() and (slot[:16] >= 0).all() and (slot[48:88] >= 0).all()
    c.o.n_pages[:] = c.pool.n_pages.tolist()
    c.o.block_table[:] = c.pool.block_table.cpu().numpy()
    append_rows(c, start, seq, pos, slot)
    assert c.pool.ctx_len.tolist() == [70, 18]


# rows of one sequence that have no slot: inside a page, at its first or last token, across the
# 16-row groups that the kernel's blocks look at
ROW_HOLES = [
    ([0], [16], [5]), ([0], [16], [0]), ([0], [32], [15, 16]), ([3], [40], [7, 8, 9]),
    ([9], [100], [6, 22, 38, 54, 70]), ([0, 11], [7, 90], [3, 7 + 1, 7 + 5, 7 + 20, 7 + 21, 7 + 36]),
    ([5, 2], [15, 15], [*range(1, 10), *range(16, 29)]), ([0], [64], [*range(1, 64, 2)]),
    ([14], [70], [*range(3, 17), *range(20, 33)]),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("held,new,rows", ROW_HOLES)
def test_rows_without_a_slot_inside_pages(held, new, rows, D):
    """The rows of a page around a hole are folded into its summary by one warp."""
    g = np.random.default_rng([34, len(new), new[0], len(rows)])
    c = Cache(g, len(new), 3, D, 16, 40)
    c.meta[:] = c.g.choice([-0.25, 0.25, 1.0], c.meta.shape)      # what earlier users left
    c.kv.meta.copy_(bf16(c.meta))
    if any(held):
        c.add(held)
    start, seq, pos, slot = planned(c, new, 2)
    slot[rows] = -1
    append_rows(c, start, seq, pos, slot)
    # the same holes by rows that name no position, in the next tokens
    start, seq, pos, slot = planned(c, new, 1)
    slot[rows] = pos[rows] = -1
    append_rows(c, start, seq, pos, slot)


@pytest.mark.parametrize("what", ["seq", "slot", "offset"])
def test_dropped_rows_inside_pages(what):
    g = np.random.default_rng([35])
    c = Cache(g, 2, 4, 64, 20, 40)
    c.add([21, 0])
    start, seq, pos, slot = planned(c, [60, 33])
    kept = slot.copy()
    at = np.array([2, 3, 14, 30, 60 + 4, 60 + 15, 60 + 16])
    kept[at] = -1
    if what == "seq":
        seq[at] = [2, -3, 7, 2, 2, -9, 2]
    elif what == "slot":
        slot[at] = 40 * PAGE + 3
    else:
        slot[at] ^= 1                                        # another row of the page than pos says
    append_rows(c, start, seq, pos, slot, BAD_INDEX, kept)


def test_holes_between_other_sequences_rows():
    """Single tokens in the middle of a page behind a request that found no page."""
    g = np.random.default_rng([36])
    c = Cache(g, 40, 2, 64, 3, 70)
    held = [int(x) for x in g.integers(0, 30, 40)]
    c.add(held)
    start, seq, pos, slot = planned(c, [1, 3] * 20, 4)
    for b in range(1, 40, 4):
        pos[seq == b] = slot[seq == b] = -1
    append_rows(c, start, seq, pos, slot)


@pytest.mark.parametrize("D", [64, 128])
def test_keys_that_are_no_numbers_fold_as_one_by_one(D):
    """NaN and infinite keys give the summaries that se_kv_append gives token by token: a NaN
    is passed over unless the page holds nothing else in that channel."""
    g = np.random.default_rng([37, D])
    n = 40
    c = Cache(g, 2, 2, D, 6, 12)
    other = se.PagedKV(c.kv.k.clone(), c.kv.v.clone(), c.kv.meta.clone(), c.kv.block_table,
                       c.kv.ctx_len.clone())
    k = normal(g, 2 * n, 2, D)
    k[g.random(k.shape) < 0.5] = np.nan
    k[:16, 0, :8] = k[n:n + 3, 1] = np.nan
    k[5, 1, 3], k[6, 1, 4] = np.inf, -np.inf
    k, v = bf16(k), bf16(normal(g, 2 * n, 2, D))
    at = [0, 0]
    for new in ([1, 3], [20, 1], [19, 36]):
        start, seq, pos, slot = planned(c, new)
        rows = np.concatenate([np.arange(b * n + at[b], b * n + at[b] + new[b]) for b in range(2)])
        se.se_kv_append_chunk(c.kv, k[rows], v[rows], se.Chunk(i32(start), i32(seq), i32(pos), i32(slot)),
                              2, c.ws)
        at = [a + x for a, x in zip(at, new)]
        c.o.ctx[:] = at
    for b in range(2):                                        # one token of one sequence a call
        one = se.PagedKV(other.k, other.v, other.meta[b:], other.block_table[b:], other.ctx_len[b:])
        for i in range(n):
            se.se_kv_append(one, k[b * n + i:b * n + i + 1], v[b * n + i:b * n + i + 1], 1, c.ws)
    assert se.status_word(c.ws) == 0 and c.kv.ctx_len.tolist() == other.ctx_len.tolist() == [n, n]
    assert np.array_equal(f64(c.kv.k), f64(other.k), equal_nan=True)
    assert np.isnan(f64(other.meta[0, 0, 0, :, :8])).all() and np.isinf(f64(other.meta)).any()
    assert np.array_equal(f64(c.kv.meta), f64(other.meta), equal_nan=True)


@pytest.mark.parametrize("whole_page", [False, True])
def test_dropped_rows_that_name_no_sequence(whole_page):
    """A seq of -1 beside a slot is a dropped row like any other, not the end of the rows."""
    g = np.random.default_rng([38])
    c = Cache(g, 2, 2, 64, 10, 20)
    c.add([3, 0])
    start, seq, pos, slot = planned(c, [90, 40], 6)
    kept = slot.copy()
    at = np.r_[13:29, 45:61] if whole_page else np.array([5, 20, 21, 44, 90 + 1, 90 + 30])
    kept[at] = -1
    seq[at] = -1
    append_rows(c, start, seq, pos, slot, BAD_INDEX, kept)
