"""GPU parity of the append with rotation where it has rows enough for one block to take 16 of them alone
(heads side by side, rows beside them, passes dealt out by what each warp's keys take): the bits of
the two calls it stands for."""
import numpy as np
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se
from tests.test_gpu_chunk import i32
from tests.test_gpu_rope import append_both, make, marked, small_ws

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


def enough_rows():
    """Above this number of rows a block has its 16 for itself."""
    return 16 * 2 * torch.cuda.get_device_properties(0).multi_processor_count


def lengths(kind, g, extra):
    """New rows of every sequence: a step to begin with (pages are then begun), and the large one."""
    need = enough_rows() + extra
    if kind == "one":                                  # one prompt
        return [3], [need]
    if kind == "few":                                  # prompts of unequal length, some none
        return [5, 0, 16, 33, 7], [need // 2 + 1, 1, 0, need // 3, need // 4]
    if kind == "ragged":
        n = 150
        return g.integers(0, 40, n).tolist(), g.integers(0, 2 * need // n + 30, n).tolist()
    n = need + 37                                      # single tokens
    return g.integers(0, 18, n).tolist(), [1] * n


# (kind, query heads, KV heads, channels, rotated, layout, norm, summaries)
CASES = [("one", 4, 1, 64, 64, 0, 1, True), ("one", 2, 3, 128, 96, 1, 0, True), ("few", 5, 2, 64, 48, 1, 0, True),
         ("few", 8, 5, 128, 128, 0, 1, False), ("few", 3, 8, 64, 16, 0, 1, True), ("few", 1, 9, 64, 64, 1, 1, True),
         ("ragged", 6, 3, 64, 32, 0, 0, True), ("ragged", 4, 4, 128, 128, 1, 1, True), ("ragged", 7, 1, 128, 64, 0, 1, False),
         ("single", 2, 2, 64, 64, 0, 1, True), ("single", 1, 36, 64, 64, 1, 0, True),     # (more than 64 jobs a block)
         ("single", 4, 5, 128, 128, 0, 1, True)]


@pytest.mark.parametrize("kind,hq,hk,dim,rot,layout,norm,summaries", CASES)
def test_append_of_many_rows_is_rotation_then_append(kind, hq, hk, dim, rot, layout, norm, summaries):
    g = np.random.default_rng([61, hq, hk, dim])
    torch.manual_seed(61 + hq)
    steps = lengths(kind, g, 5 + hq)
    batch = len(steps[0])
    rows = [int(np.sum(s)) + 3 * i for i, s in enumerate(steps)]           # (rows behind the last sequence)
    assert rows[1] - 3 > enough_rows()
    held = np.sum(steps, 0)
    maxp, pages = int(held.max()) // 16 + 1, int((held // 16 + 1).sum())
    pool = se.PagePool.empty(batch, pages, maxp)
    pool.free_pages.copy_(i32(g.permutation(pages)))
    ws = se.workspace(se.se_page_pool_workspace(batch))
    rope = make(g, rot, dim, layout, (norm, norm))
    kv = se.PagedKV(marked(pages, hk, 16, dim), marked(pages, hk, 16, dim),
                    marked(batch, maxp, hk, 2, dim) if summaries else None, pool.block_table, pool.ctx_len)
    for step, (new, n) in enumerate(zip(steps, rows)):
        chunk = se.Chunk.empty(batch, n)
        se.se_chunk_plan(pool, i32(new), batch, chunk, ws)
        assert se.status_word(ws) == 0
        if step == 1:                                                      # holes, as of pages not found
            hole = torch.from_numpy(g.choice(n - 3, 40, replace=False))
            chunk.slot[hole] = -1
        x = torch.randn(n, hq + 2 * hk, dim, device="cuda").bfloat16()
        append_both(kv, rope, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], chunk, batch)
    # keys alone, and the queries over themselves
    two = se.PagedKV(kv.k.clone(), kv.v.clone(), None, kv.block_table, kv.ctx_len)
    se.se_rope_append_chunk(two, rope, None, x[:, hq:hq + hk], x[:, hq + hk:], None, chunk, batch, small_ws())
    assert two.k.equal(kv.k) and two.v.equal(kv.v)
    want = marked(rows[1], hq, dim)
    se.se_qk_rope(rope, chunk.pos, x[:, :hq], None, want, None, small_ws())
    live = chunk.pos >= 0
    before = x.clone()
    se.se_rope_append_chunk(kv, rope, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], x[:, :hq], chunk, batch, small_ws())
    assert x[live][:, :hq].equal(want[live]) and x[~live].equal(before[~live])
    assert x[:, hq:].equal(before[:, hq:])
