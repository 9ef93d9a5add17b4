"""Page tables of pools so large that se_pages_release runs on several blocks, against the oracle."""
import numpy as np
import pytest

from kv_cache_decode_quest_gb300 import binding as se
from oracle import chunk as oc
from tests.test_gpu_chunk import both_pools, i32, plan_both, same_pool

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


# the grid is a block for every 4096 entries of the smaller of table and pool
@pytest.mark.parametrize("batch,hi,pages,maxp", [
    (3, 70000, 9001, 4400), (200, 900, 8192, 60), (1024, 500, 20000, 33), (1025, 400, 16500, 27),
    (2500, 200, 33000, 14)])
def test_release_on_several_blocks(batch, hi, pages, maxp):
    """Plan, release of some and then of all sequences, and the plan behind each on the same
    workspace: stack, tables and counts are the oracle's."""
    assert min(batch * maxp, pages) // 4096 >= 2
    g = np.random.default_rng([41, batch])
    o, p = both_pools(pages, batch, maxp)
    order = g.permutation(pages)
    o.free = order.tolist()
    p.free_pages.copy_(i32(order))
    ws = se.workspace(se.se_page_pool_workspace(batch))
    for share in (0.5, 1.0, 0.9, 1.0):
        new = g.integers(1, hi + 1, batch)
        plan_both(o, p, new, int(new.sum()) + 3, ws)
        assert o.n_pages.sum() > pages // 3
        o.ctx[:] = np.minimum(o.ctx + new, o.n_pages * 16)
        p.ctx_len.copy_(i32(o.ctx))
        done = g.random(batch) < share
        se.se_pages_release(p, i32(done), batch, ws)
        oc.release(o, done)
        assert se.status_word(ws) == 0
        same_pool(o, p)
    assert o.n_pages.sum() == 0 and sorted(o.free) == list(range(pages))


def test_refused_release_on_several_blocks_leaves_the_counter_at_zero():
    """Pages released twice: nothing moves, and the next calls on the workspace are right."""
    batch, pages, maxp = 600, 12000, 20
    o, p = both_pools(pages, batch, maxp)
    ws = se.workspace(se.se_page_pool_workspace(batch))
    plan_both(o, p, [300] * batch, 300 * batch, ws)
    p.n_free.fill_(pages)
    stack = p.free_pages.clone()
    se.se_pages_release(p, i32([1] * batch), batch, ws)
    assert se.status_word(ws) == 2 and int(p.n_free) == pages                    # SE_DEV_CAPACITY
    assert p.n_pages.tolist() == o.n_pages.tolist() and p.free_pages.equal(stack)
    ws[:4] = 0
    p.n_free.fill_(len(o.free))
    done = np.arange(batch) % 3 != 0
    se.se_pages_release(p, i32(done), batch, ws)
    oc.release(o, done)
    assert se.status_word(ws) == 0
    same_pool(o, p)
    plan_both(o, p, [17] * batch, 17 * batch, ws)
