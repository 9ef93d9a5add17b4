"""GPU parity of forks, truncations and what the caches take over, against the oracle: every table, count
and stored row equal."""
import numpy as np
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se
from oracle import chunk as oc
from oracle import forks as of
from tests.test_gpu_chunk import both_pools, i32, plan_both, same_pool

pytestmark = pytest.mark.gpu
BAD_INDEX, CAPACITY, BAD_LENGTH = 1, 2, 4


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


class Both:
    """The oracle's pool and the GPU's, with counts of shared pages."""

    def __init__(self, pages, batch, maxp, g=None, shared=True):
        self.o, self.p = both_pools(pages, batch, maxp)
        if g is not None:
            order = g.permutation(pages).tolist()
            self.o.free = list(order)
            self.p.free_pages.copy_(i32(order))
        self.batch = batch
        self.o_refs = [0] * pages if shared else None
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda") if shared else None
        self.carry = se.Carry.empty(batch)
        self.ws = se.workspace(se.se_pages_truncate_workspace(batch, pages))

    def grow(self, new):
        rows = int(np.sum(new))
        chunk = plan_both(self.o, self.p, new, rows, self.ws)
        pos, seq = chunk.pos.cpu().numpy(), chunk.seq.cpu().numpy()
        for b in range(self.batch):
            mine = pos[seq == b]
            if len(mine) and mine[-1] >= 0:
                self.o.ctx[b] = mine[-1] + 1
        self.p.ctx_len.copy_(i32(self.o.ctx))
        return chunk

    def same(self, got):
        from_seq, from_page, flags = got
        assert self.carry.from_seq.tolist() == list(from_seq)
        assert self.carry.from_page.tolist() == list(from_page)
        assert se.status_word(self.ws) == flags
        assert not self.ws[4:].any()                               # all zero past the status word
        self.ws[:4] = 0
        same_pool(self.o, self.p)
        if self.refs is not None:
            assert self.refs.tolist() == list(self.o_refs)
        return flags

    def fork(self, src):
        self.carry.from_page.fill_(-7)
        se.se_pages_fork(self.p, self.refs, i32(src), self.batch, self.carry, self.ws)
        return self.same(of.fork(self.o, self.o_refs, src))

    def cut(self, keep):
        self.carry.from_seq.fill_(-7)
        se.se_pages_truncate(self.p, self.refs, i32(keep), self.batch, self.carry, self.ws)
        return self.same(of.truncate(self.o, self.o_refs, keep))


def random_src(g, b, share):
    src = np.full(b.batch, -1)
    full, empty = np.flatnonzero(b.o.n_pages > 0), np.flatnonzero(b.o.n_pages == 0)
    if len(full):
        for x in empty:
            if g.random() < share:
                src[x] = g.choice(full)
    return src


def random_keep(g, b, share):
    keep = np.where(g.random(b.batch) < share, (b.o.ctx * g.random(b.batch) * 1.1).astype(int), -1)
    keep[g.random(b.batch) < 0.2] = 0
    whole = g.random(b.batch) < 0.1
    keep[whole] = keep[whole] // 16 * 16
    return keep


# up to 4096 entries: one block; more: a cluster, of 256, 512 or 1024 threads a block; sequences per
# thread one and several
@pytest.mark.parametrize("batch,hi,pages,maxp", [
    (1, 40, 6, 5), (4, 50, 20, 9), (16, 100, 120, 20), (300, 60, 1500, 30), (257, 90, 9000, 40),
    (1025, 40, 20000, 17), (2500, 60, 9001, 12), (3, 40000, 12000, 8200),
    (40, 6000, 30000, 1000), (70, 6000, 60000, 1000)])
def test_many_steps(batch, hi, pages, maxp):
    g = np.random.default_rng([31, batch, pages])
    b = Both(pages, batch, maxp, g)
    seen = 0
    for step in range(8):
        new = g.integers(0, hi + 1, batch) * (g.random(batch) < 0.6)
        new = np.where(b.o.ctx + new > maxp * 16, 0, new)
        b.grow(new)
        b.fork(random_src(g, b, 0.7))
        seen = max(seen, max(b.o_refs))
        b.cut(random_keep(g, b, 0.5))
    assert batch < 16 or seen >= 1
    b.cut([0] * batch)
    assert sorted(b.o.free) == list(range(pages)) and max(b.o_refs) == 0


@pytest.mark.parametrize("batch,hi,pages,maxp", [(5, 60, 40, 9), (600, 300, 12000, 20)])
def test_truncation_without_shared_pages(batch, hi, pages, maxp):
    g = np.random.default_rng([32, batch])
    b = Both(pages, batch, maxp, g, shared=False)
    for step in range(4):
        new = g.integers(0, hi + 1, batch)
        b.grow(np.where(b.o.ctx + new > maxp * 16, 0, new))
        b.cut(random_keep(g, b, 0.6))
    b.cut([0] * batch)
    assert sorted(b.o.free) == list(range(pages))


def test_truncation_to_nothing_is_a_release():
    for pages, batch in ((40, 3), (20000, 700)):
        a = Both(pages, batch, 30)
        c = Both(pages, batch, 30)
        new = [7 + 13 * i % 300 for i in range(batch)]
        for x in (a, c):
            x.grow(new)
        done = np.arange(batch) % 3 != 1
        a.cut(np.where(done, 0, -1))
        se.se_pages_release(c.p, i32(done), batch, c.ws)
        n = int(a.p.n_free)
        assert int(c.p.n_free) == n and c.p.free_pages[:n].equal(a.p.free_pages[:n])
        assert c.p.n_pages.equal(a.p.n_pages) and c.p.ctx_len.equal(a.p.ctx_len)


def test_planned_tokens_are_taken_back():
    """A plan whose tokens are never appended: the cut returns its pages, and the next plan finds them."""
    b = Both(30, 2, 12)
    b.grow([20, 5])
    chunk = plan_both(b.o, b.p, [40, 60], 100, b.ws)
    assert b.o.n_pages.tolist() == [4, 5]
    b.cut([1 << 30, 5])
    assert b.o.n_pages.tolist() == [2, 1] and b.o.ctx.tolist() == [20, 5]
    again = plan_both(b.o, b.p, [40, 60], 100, b.ws)
    assert again.slot.equal(chunk.slot)


def test_two_holders_cut_inside_the_page_they_share():
    """Both take a page of their own, the shared one goes back, and its rows are still read from it."""
    b = Both(12, 3, 6)
    b.grow([40, 0, 0])
    b.fork([-1, 0, 0])
    assert max(b.o_refs) == 2
    b.cut([20, 21, -1])                                            # page 1 is still the third's
    assert b.carry.from_page.tolist()[0] == b.carry.from_page.tolist()[1] >= 0
    b.cut([5, 6, 7])                                               # page 0 nobody holds any more
    assert max(b.o_refs) == 0


def test_no_page_left():
    b = Both(4, 3, 6)
    b.grow([40, 0, 0])
    assert b.fork([-1, 0, 0]) == CAPACITY                          # one page was left: the first fork has it
    assert b.o.n_pages.tolist() == [3, 3, 0]
    assert b.cut([20, -1, -1]) == CAPACITY                         # needs a page of its own: stays as it was
    assert b.o.ctx.tolist() == [40, 40, 0]
    assert b.cut([32, -1, -1]) == 0
    # a fork that needs no page is served all the same
    assert b.cut([-1, 0, -1]) == 0
    b.grow([0, 0, 0])
    b.cut([16, -1, -1])
    assert b.fork([-1, 0, -1]) == 0
    b.o.free, b.p.n_free[0] = [], 0
    assert b.fork([-1, -1, 0]) == 0 and b.o.n_pages.tolist() == [1, 1, 1]


def test_inconsistent_requests_stay_as_they_were():
    g = np.random.default_rng(33)
    b = Both(60, 8, 6, g)
    b.grow([40, 20, 0, 0, 0, 0, 0, 0])
    assert b.fork([1, -1, 8, 2, 7, -1, 0, 0]) & (BAD_INDEX | BAD_LENGTH)
    # lengths that make no sense
    for field, bad in (("ctx", -3), ("ctx", 97), ("held", 7), ("held", -1), ("held", 0)):
        b = Both(60, 3, 6)
        b.grow([40, 20, 0])
        if field == "ctx":
            b.o.ctx[1] = bad
            b.p.ctx_len[1] = bad
        else:
            b.o.n_pages[1] = bad
            b.p.n_pages[1] = bad
        n = b.p.n_pages.tolist()
        se.se_pages_fork(b.p, b.refs, i32([-1, -1, 1]), 3, b.carry, b.ws)
        se.se_pages_truncate(b.p, b.refs, i32([-1, 3, -1]), 3, b.carry, b.ws)
        assert se.status_word(b.ws) == BAD_LENGTH and b.p.n_pages.tolist() == n
        assert int(b.p.n_free) == len(b.o.free) and not b.refs.any()


def test_pages_outside_the_pool():
    """A table or stack with pages that do not exist: flagged, never counted, never on the stack."""
    for batch, pages, maxp in ((3, 40, 8), (900, 12000, 12)):
        b = Both(pages, batch, maxp)
        b.grow([70, 35, 0] + [70] * (batch - 3))
        b.p.block_table[0, 2] = pages
        b.p.block_table[0, 3] = -5
        se.se_pages_truncate(b.p, b.refs, i32([20] + [-1] * (batch - 1)), batch, b.carry, b.ws)
        assert se.status_word(b.ws) == BAD_INDEX
        assert b.p.ctx_len[0] == 20 and int(b.p.n_free) == len(b.o.free) + 1
        assert not b.ws[4:].any() and not b.refs.any()
        b.ws[:4] = 0
        b.p.block_table[1, 0] = -1                                 # the page that would be the last
        se.se_pages_truncate(b.p, b.refs, i32([-1, 7] + [-1] * (batch - 2)), batch, b.carry, b.ws)
        assert se.status_word(b.ws) == BAD_INDEX and b.p.ctx_len[1] == 35
        b.ws[:4] = 0
        se.se_pages_fork(b.p, b.refs, i32([-1, -1, 1] + [-1] * (batch - 3)), batch, b.carry, b.ws)
        assert se.status_word(b.ws) == BAD_INDEX
        b.ws[:4] = 0
        third = i32([-1, -1, 0] + [-1] * (batch - 3))
        se.se_pages_truncate(b.p, b.refs, third, batch, b.carry, b.ws)
        assert se.status_word(b.ws) == BAD_INDEX and b.p.n_pages[2] == 0   # (the bad page it shared)
        b.ws[:4] = 0
        b.p.free_pages[int(b.p.n_free) - 1] = pages + 3            # the next page to be taken
        se.se_pages_fork(b.p, b.refs, third, batch, b.carry, b.ws)
        assert se.status_word(b.ws) == BAD_INDEX and b.p.n_pages[2] == 0


def test_a_stack_that_would_pass_its_end():
    """Pages let go twice: nothing changes, also on the next calls' workspace."""
    for batch, pages, maxp in ((3, 20, 8), (700, 9000, 12)):
        b = Both(pages, batch, maxp)
        b.grow([30] * batch)
        b.p.n_free.fill_(pages)
        keep = [0] * batch
        state = [x.clone() for x in (b.p.free_pages, b.p.n_pages, b.p.ctx_len, b.p.block_table)]
        se.se_pages_truncate(b.p, b.refs, i32(keep), batch, b.carry, b.ws)
        assert se.status_word(b.ws) == CAPACITY and int(b.p.n_free) == pages
        for x, y in zip(state, (b.p.free_pages, b.p.n_pages, b.p.ctx_len, b.p.block_table)):
            assert x.equal(y)
        assert not b.ws[4:].any() and not b.refs.any()
        b.ws[:4] = 0
        b.p.n_free.fill_(len(b.o.free))
        b.cut(keep)


# ---------------------------------------------------------------------------
# the caches
# ---------------------------------------------------------------------------

class Cache:
    """A layer on both sides, filled token by token by the oracle."""

    def __init__(self, b, heads, dim, g, summaries=True):
        pages, maxp = b.o.num_pages, b.o.block_table.shape[1]
        self.g, self.heads, self.dim = g, heads, dim
        self.k, self.v = np.zeros((2, pages, heads, 16, dim))
        self.meta = np.zeros((b.batch, maxp, heads, 2, dim)) if summaries else None
        z = lambda x: torch.zeros(x.shape, dtype=torch.bfloat16, device="cuda")          # noqa: E731
        self.kv = se.PagedKV(z(self.k), z(self.v), z(self.meta) if summaries else None, b.p.block_table,
                             b.p.ctx_len)

    def append(self, b, chunk):
        n = chunk.slot.numel()
        x = [torch.from_numpy(self.g.standard_normal((n, self.heads, self.dim))).bfloat16().cuda()
             for _ in range(2)]
        ctx = b.o.ctx.copy()
        words = [y.cpu().numpy() for y in (chunk.start, chunk.seq, chunk.pos, chunk.slot)]
        oc.append(b.o, self.k, self.v, self.meta, *[y.double().cpu().numpy() for y in x], *words)
        assert np.array_equal(b.o.ctx, ctx)
        se.se_kv_append_chunk(self.kv, *x, chunk, b.batch, b.ws)

    def follow(self, b):
        fs, fp = b.carry.from_seq.tolist(), b.carry.from_page.tolist()
        of.carry(b.o, self.k, self.v, self.meta, fs, fp)
        se.se_pages_carry(self.kv, b.carry, b.batch, b.ws)
        assert se.status_word(b.ws) == 0
        self.same(b)

    def same(self, b):
        for x, y in ((self.kv.k, self.k), (self.kv.v, self.v)):
            assert np.array_equal(x.double().cpu().numpy(), y)
        if self.meta is not None:
            got = self.kv.meta.double().cpu().numpy()
            for s in range(b.batch):
                n = -(-int(b.o.ctx[s]) // 16)
                assert np.array_equal(got[s, :n], self.meta[s, :n]), s


@pytest.mark.parametrize("batch,hi,pages,maxp,heads,dim", [
    (4, 50, 30, 9, 1, 64), (6, 120, 90, 20, 4, 128), (5, 90, 70, 14, 2, 64), (40, 60, 300, 12, 8, 128),
    (3, 3000, 1500, 600, 4, 128)])
def test_caches_follow(batch, hi, pages, maxp, heads, dim):
    """Random growth, forks and cuts; two layers, one without summaries.  The summaries are those of the rows
    that are held, whatever was taken back."""
    g = np.random.default_rng([34, batch, hi])
    b = Both(pages, batch, maxp, g)
    layers = [Cache(b, heads, dim, g), Cache(b, heads, dim, g, summaries=False)]
    for step in range(6):
        new = g.integers(0, hi + 1, batch) * (g.random(batch) < 0.7)
        chunk = b.grow(np.where(b.o.ctx + new > maxp * 16, 0, new))
        for x in layers:
            x.append(b, chunk)
        for change in (lambda: b.fork(random_src(g, b, 0.8)), lambda: b.cut(random_keep(g, b, 0.5))):
            change()
            for x in layers:
                x.follow(b)
    ref = layers[0].kv.meta.clone()
    se.se_page_meta_build(layers[0].kv, batch, b.ws)               # made anew from all rows: the same
    for s in range(batch):
        n = -(-int(b.o.ctx[s]) // 16)
        assert layers[0].kv.meta[s, :n].equal(ref[s, :n])


def test_carry_with_bad_words_skips_them():
    g = np.random.default_rng(35)
    b = Both(30, 4, 6, g)
    x = Cache(b, 2, 64, g)
    x.append(b, b.grow([40, 20, 7, 0]))
    before = [y.clone() for y in (x.kv.k, x.kv.v, x.kv.meta)]
    for seqs, pages, flags in (([4, -1, -1, -1], [-1] * 4, BAD_INDEX), ([-1] * 4, [30, -1, -1, -1], BAD_INDEX),
                               ([-1, -1, 99, -1], [-1, 1 << 30, -1, -1], BAD_INDEX)):
        c = se.Carry(i32(seqs), i32(pages))
        se.se_pages_carry(x.kv, c, 4, b.ws)
        assert se.status_word(b.ws) == flags
        b.ws[:4] = 0
    ok = se.Carry(i32([-1, 0, -1, -1]), i32([-1, -1, 0, -1]))
    for bad in (-1, 97):
        b.p.ctx_len[1], b.p.ctx_len[2] = bad, bad
        se.se_pages_carry(x.kv, ok, 4, b.ws)
        assert se.status_word(b.ws) == BAD_LENGTH
        b.ws[:4] = 0
    b.p.ctx_len.copy_(i32([40, 20, 7, 0]))
    b.p.block_table[2, 0] = 30                                     # the page that the rows go to
    se.se_pages_carry(x.kv, se.Carry(i32([-1] * 4), i32([-1, -1, 0, -1])), 4, b.ws)
    assert se.status_word(b.ws) == BAD_INDEX
    for y, z in zip(before, (x.kv.k, x.kv.v, x.kv.meta)):
        assert y.equal(z)


def test_replayed_from_a_graph():
    """One captured turn of samples (cut, fork, carry) replayed as the prompt grows."""
    g = np.random.default_rng(36)
    b = Both(60, 5, 10, g)
    x = Cache(b, 2, 128, g)
    src, none = [-1, 0, 0, 0, 0], [-1, 0, 0, 0, 0]
    isrc, inone, second = i32(src), i32(none), se.Carry.empty(5)

    def turn():
        se.se_pages_truncate(b.p, b.refs, inone, 5, second, b.ws)
        se.se_pages_fork(b.p, b.refs, isrc, 5, b.carry, b.ws)
        se.se_pages_carry(x.kv, b.carry, 5, b.ws)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    x.append(b, b.grow([19, 0, 0, 0, 0]))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        turn()
    for n in (30, 1, 14, 40):
        graph.replay()
        of.truncate(b.o, b.o_refs, none)
        b.same(of.fork(b.o, b.o_refs, src))
        fs, fp = b.carry.from_seq.tolist(), b.carry.from_page.tolist()
        of.carry(b.o, x.k, x.v, x.meta, fs, fp)
        x.same(b)
        x.append(b, b.grow([n, 0, 0, 0, 0]))


def test_more_entries_than_the_cluster_holds_at_once():
    """Hundreds of samples of one long prompt let go together, and all but one of them: the pages that
    come back, their order and the counts."""
    g = np.random.default_rng(37)
    pages, batch, maxp = 5000, 420, 2010
    b = Both(pages, batch, maxp, g)
    b.grow([2003 * 16 + 5] + [0] * (batch - 1))
    src = np.full(batch, -1)
    src[1:] = 0
    for keep in (0, 1000 * 16 + 3):
        assert b.fork(src) == 0 and max(b.o_refs) == batch - 1
        some = np.full(batch, keep)
        some[[0, 17]] = -1, -1
        if keep:
            some[5:200] = 0                                      # others keep a part, in pages of their own
        assert b.cut(some) == 0
        assert b.cut(np.where(np.arange(batch) == 0, -1, 0)) == 0 and max(b.o_refs) == 0
    assert b.cut([0] * batch) == 0 and sorted(b.o.free) == list(range(pages))


FIRST_CALL = """
import torch
from kv_cache_decode_quest_gb300 import binding as se
B, pages, maxp = 20, 20000, 900
pool = se.PagePool.empty(B, pages, maxp)
refs, carry = torch.zeros(pages, dtype=torch.int32, device="cuda"), se.Carry.empty(B)
ws = se.workspace(se.se_pages_truncate_workspace(B, pages))
keep = torch.zeros(B, dtype=torch.int32, device="cuda")
src = torch.tensor([-1] + [0] * (B - 1), dtype=torch.int32, device="cuda")
new = torch.tensor([14000] + [0] * (B - 1), dtype=torch.int32, device="cuda")
chunk = se.Chunk.empty(B, 14000)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    se.se_chunk_plan(pool, new, B, chunk, ws)
    pool.ctx_len[:1] = 14000
    se.se_pages_fork(pool, refs, src, B, carry, ws)
    se.se_pages_truncate(pool, refs, keep, B, carry, ws)
for _ in range(2):
    graph.replay()
    torch.cuda.synchronize()
    assert se.status_word(ws) == 0 and int(pool.n_free) == pages and not refs.any()
    assert not ws[4:].any() and pool.free_pages.flip(0).equal(torch.arange(pages, device="cuda").int())
"""


def test_the_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True,
                       timeout=250)
    assert r.returncode == 0, r.stderr[-2000:]


def test_a_source_whose_last_page_does_not_exist_takes_no_page():
    """A fork of it asks for none: the stack keeps its pages, the forks behind it get theirs."""
    for batch, pages, maxp in ((6, 12, 6), (900, 3000, 12)):
        b = Both(pages, batch, maxp)
        b.grow([40, 20] + [0] * (batch - 2))
        src = np.full(batch, -1)
        src[2:6] = [1, 0, 1, 0]
        for bad in (pages, -1):
            b.o.block_table[1, 1] = bad
            b.p.block_table[1, 1] = bad
            before = len(b.o.free)
            assert b.fork(src) == BAD_INDEX
            assert b.o.n_pages[2:6].tolist() == [0, 3, 0, 3] and len(b.o.free) == before - 2
            assert b.cut(np.where(np.isin(np.arange(batch), (3, 5)), 0, -1)) == 0
            assert len(b.o.free) == before
        # the last page of the stack goes to the fork that can be served
        b.o.free = b.o.free[:1]
        b.p.n_free.fill_(1)
        src[5] = -1
        assert b.fork(src) == BAD_INDEX and b.o.n_pages[2:6].tolist() == [0, 3, 0, 0]
