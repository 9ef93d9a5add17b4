"""GPU: a cache that prompts in chunks left, under the methods other than two-call Quest: what each
gives over it is, bit for bit, what it gives over the cache that the host laid out."""
import numpy as np
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se
from kv_cache_decode_quest_gb300 import synth
from kv_cache_decode_quest_gb300.workloads import PromptRun, QuestRun
from tests.test_gpu_chunk import Attn, held

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


def both(name):
    w = synth.QuestWorkload(name, batch=3, num_q_heads=16, num_kv_heads=2, head_dim=128,
                            ctx=(700, 130, 333), budget=(128, 64, 64), steps=3, outliers=True)
    inputs = synth.quest_inputs(w)
    run = PromptRun(w, inputs, synth.prompt_queries(w), 150)
    for _ in run.prefill():
        pass
    ref = QuestRun(w, inputs, mode="step")
    assert run.status() == 0
    return w, run, ref


def queries(*shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(61),
                       device="cuda").bfloat16()


def test_one_kernel_step():
    w, run, ref = both("prompt_step")
    B, H, Hq, D, maxp = w.batch, run.Hkv, run.Hq, run.D, run.kv.block_table.shape[1]
    ws = se.workspace(se.se_quest_step_workspace(B, H, Hq, D, maxp))
    for s in range(w.steps):
        ref.step(s)
        se.se_chunk_plan(run.pool, torch.ones_like(run.pool.n_pages), B, run.one, run.ws_pool)
        se.se_quest_step(run.kv, ref.k_new[s], ref.v_new[s], ref.q[s], B, Hq, run.budget, run.scale,
                         run.sel, run.n_sel, run.view, run.out, run.lse, ws)
        assert se.status_word(ws) == 0 and ref.status() == 0
        assert torch.equal(run.n_sel, ref.n_sel)
        for u in range(B * H):
            k = int(ref.n_sel[u])
            assert torch.equal(run.sel[u, :k], ref.sel[u, :k])
        assert torch.equal(run.out, ref.out) and torch.equal(run.lse, ref.lse)
    assert run.kv.ctx_len.tolist() == [c + w.steps for c in w.ctx] and run.status() == 0


def test_sink_and_recent_pages():
    w, run, ref = both("prompt_sink")
    B, H, Hq, D = w.batch, run.Hkv, run.Hq, run.D
    q, got = queries(B, Hq, D), []
    for kv in (run.kv, ref.kv):
        view = se.View.empty(B * H, kv.block_table.shape[1])
        ws, ws_dec = se.workspace(se.se_small_workspace()), se.workspace(
            se.se_sparse_decode_workspace(B * H, Hq // H, D))
        out, lse = torch.zeros_like(run.out), torch.zeros_like(run.lse)
        se.se_view_sink_recent(kv, B, 2, 5, view, ws)
        se.se_sparse_decode(kv.k, kv.v, view, q, B, Hq, H, D, run.scale, out, lse, ws_dec)
        assert se.status_word(ws) == 0 and se.status_word(ws_dec) == 0
        got.append((view.n_tokens, out, lse))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and bool(torch.isfinite(got[0][2]).all())


def test_snapkv_compaction():
    w, run, ref = both("prompt_snap")
    B, H, Hq, D, window, keep = w.batch, run.Hkv, run.Hq, run.D, 16, 40
    q, got = queries(B, window, Hq, D), []
    for kv in (run.kv, ref.kv):
        cache = se.VarlenKV.empty(B, H, keep + window + 8, D)
        ws = se.workspace(se.se_snapkv_workspace(B, H, Hq, window, max(w.ctx)))
        se.se_snapkv_compact(kv, q, B, Hq, window, 5, keep, window, run.scale, cache, ws)
        assert se.status_word(ws) == 0
        got.append([getattr(cache, x) for x in ("k", "v", "pos", "seg_len", "seq_len")])
    assert all(torch.equal(a, b) for a, b in zip(*got)) and int(got[0][3].min()) == keep + window


def test_last_2048_tokens_of_32k():
    """32 query heads over 4 KV heads of 128: sampled rows, bf16 and fp32 output."""
    g = np.random.default_rng([62])
    c = held(g, 1, 4, 128, [30720], [2048])
    chunk = c.add([2048])
    for f32 in (False, True):
        a = Attn(c, 8, f32)
        a.run(chunk)
        a.check(chunk, rows=5)
