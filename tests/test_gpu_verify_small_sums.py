"""GPU tests of draws from rows that weigh little: the first token whose running sum passes u times the whole,
to a part in 2^22 of the whole (of rows that weigh 2^-16 or more: to 2^-38), and never one without weight."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import verify as V
from tests.test_gpu_verify import Case

pytestmark = pytest.mark.gpu
# one block a sequence, a cluster of several, several that meet over a counter
VOCABS = [700, 5000, 20000, 131072]


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


def check(weights, u, token):
    """weights: whole numbers of units of 2^-149."""
    total, u = sum(weights), Fraction(float(min(max(u, 0.0), V.BELOW_ONE)))
    assert 0 <= token < len(weights) and weights[token] > 0
    room = Fraction(total, 1 << 22) if total < 1 << (149 - 16) else Fraction(1 << (149 - 38))
    before = sum(weights[:token])
    assert before - room <= u * total < before + weights[token] + room


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_weights(vocab, dtype):
    """Equal powers of two add up exactly at any size: the oracle's token."""
    g = np.random.default_rng([51, vocab])
    c = Case(g, [1] * 6, vocab, dtype, drafter=False)
    c.sample_u.copy_(torch.tensor([0.0, 0.1, 0.5, 0.7, 0.99, 1 - 2.0 ** -24]))
    for power in (-59, -60, -75, -100, -126, -133):
        c.p.zero_()
        c.p[:, 3:vocab - 40] = 2.0 ** power
        got, status = c.run()
        assert status == 0 and got == c.want(), power
    if dtype is torch.float32:
        c.p.zero_()
        c.p[:, 9:vocab - 40:5] = 2.0 ** -149
        got, status = c.run()
        assert status == 0 and got == c.want()


@pytest.mark.parametrize("vocab", VOCABS)
def test_a_refused_draft_beside_tiny_weights(vocab):
    """The refused token had nearly all the weight: the next one comes from what little is left."""
    g = np.random.default_rng([52, vocab])
    for drafter in (True, False):
        c = Case(g, [2] * 5, vocab, drafter=drafter)
        c.tokens.fill_(vocab - 1)
        c.accept_u.fill_(0.99)
        for power in (-60, -90):
            c.p.zero_()
            c.p[:, 1:vocab // 2:2] = 2.0 ** power
            c.p[:, vocab - 1] = 0.5
            if drafter:
                c.q.zero_()
                c.q[:, vocab - 1] = 0.75
            got, status = c.run()
            want = c.want()
            assert status == 0 and got == want and want[0] == [0] * 5
            assert all(t % 2 == 1 and t < vocab // 2 for t in got[1])


@pytest.mark.parametrize("vocab", VOCABS[:3])
def test_weights_of_all_sizes(vocab):
    """p a little above q by amounts between 2^-40 and 2^-140, some of them none."""
    g = np.random.default_rng([53, vocab])
    c = Case(g, [2] * 8, vocab)
    c.tokens.fill_(0)
    c.accept_u.fill_(0.99)
    for low, high in ((-140, -40), (-70, -45), (-30, -18)):
        d = np.exp2(g.uniform(low, high, (16, vocab))).astype(np.float32) * (g.random((16, vocab)) < 0.6)
        q = np.where(g.random((16, vocab)) < 0.5, d * np.float32(7), np.float32(0))
        p = (q + d).astype(np.float32)
        p[:, 0], q[:, 0] = 0.25, 0.5
        c.p.copy_(torch.from_numpy(p))
        c.q.copy_(torch.from_numpy(q.astype(np.float32)))
        (stay, token, _), status = c.run()
        assert status == 0 and stay == [0] * 8
        for b in range(8):
            w = [max(0, x - y) for x, y in zip(V._whole(p[2 * b]), V._whole(q[2 * b]))]
            check(w, float(c.sample_u[b]), token[b])


def test_a_tile_of_tiny_weights_between_large_ones():
    """Half the weight before and half behind: a draw that falls between takes one that has weight."""
    for power in (-60, -80):
        c = Case(np.random.default_rng(54), [1, 1, 1], 4100, drafter=False)
        c.p.zero_()
        c.p[:, 5] = c.p[:, 4000] = 0.5
        c.p[:, 1030:1800] = 2.0 ** power
        c.sample_u.copy_(torch.tensor([0.5, 0.5 - 2.0 ** -25, 0.75]))
        (_, token, _), status = c.run()
        w = V._whole(c.p[0].cpu().numpy())
        assert status == 0 and token[1:] == [5, 4000]
        check(w, 0.5, token[0])


@pytest.mark.parametrize("vocab", VOCABS)
def test_no_weight_at_all_and_then_another_call(vocab):
    """Rows that weigh nothing, and nothing left beside q, in every way that sums meet; the workspace
    serves the next call."""
    from kv_cache_decode_quest_gb300 import binding as se
    g = np.random.default_rng([55, vocab])
    ws = se.workspace(se.se_draft_verify_workspace(3, vocab))
    c = Case(g, [3, 0, 2], vocab)
    p = c.p.clone()
    want = c.want()
    assert c.run(ws) == (want, 0)
    c.q.copy_((p * 1.5).clamp(max=1))
    c.accept_u.fill_(0.99)
    got, status = c.run(ws)
    assert status == 0 and got == c.want() and got[0] == [0, 0, 0]
    c.p.zero_()
    got, status = c.run(ws)
    assert status == 16 and got == [[0, 0, 0], [-1, -1, -1], [c.first[0] + 1, -1, c.first[2] + 1]]
    ws[:4] = 0
    c.p.copy_(p)
    got, status = c.run(ws)
    assert status == 0 and got == c.want()
    assert not ws[256:256 + 8192 * 4].any()
