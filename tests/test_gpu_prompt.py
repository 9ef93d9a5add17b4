"""GPU: prompts taken into the paged cache in chunks (page tables, append,
attention), then Quest decode over what they left, against the oracle and
against the cache that is laid out by the host."""
import math

import numpy as np
import pytest
import torch

import oracle
from kv_cache_decode_quest_gb300 import synth
from kv_cache_decode_quest_gb300.workloads import PromptRun, QuestRun
from tests.parity import TOL_BF16, TOL_F32, max_abs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


def case(D, G, H, name):
    return synth.QuestWorkload(name, batch=4, num_q_heads=H * G, num_kv_heads=H, head_dim=D,
                               ctx=(700, 16, 333, 1), budget=(128, 64, 64, 64), steps=20,
                               outliers=True)


def logical(run, b, what, L):
    """[Hkv][L][D] of sequence b."""
    bt = run.kv.block_table[b, :-(-L // 16)].long()
    x = getattr(run.kv, what)[bt]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :L]


@pytest.mark.parametrize("D,G,H,chunk,out_dtype,window", [
    (128, 8, 2, 700, 0, 0), (128, 8, 2, 129, 1, 0), (64, 4, 1, 16, 0, 0), (64, 1, 4, 250, 1, 100)])
def test_prompt_in_chunks_then_quest(D, G, H, chunk, out_dtype, window):
    w = case(D, G, H, f"prompt_{D}_{G}_{chunk}")
    inputs, pq = synth.quest_inputs(w), synth.prompt_queries(w)
    run = PromptRun(w, inputs, pq, chunk, out_dtype=out_dtype, window=window)
    tol = TOL_F32 if out_dtype else TOL_BF16
    for first, new in run.prefill():
        out, lse = run.out_rows.double().cpu().numpy(), run.lse_rows.cpu().numpy()
        at = 0
        for b in range(w.batch):
            n = int(new[b])
            pick = sorted({0, n // 2, n - 1} & set(range(n)))
            for h in range(H):
                T = int(first[b]) + n
                K, V = (oracle.widen(inputs[x][b][h, :T]) for x in ("k", "v"))
                for i in pick:
                    q = oracle.widen(pq[b][first[b] + i, h * G:(h + 1) * G])[None]
                    o, z = oracle.chunk_attend(q, K, V, int(first[b]) + i, run.scale, window)
                    assert max_abs(out[at + i, h * G:(h + 1) * G], o[0]) <= tol
                    assert max_abs(lse[at + i, h * G:(h + 1) * G], z[0]) <= 1e-3
            at += n
    assert run.status() == 0
    # the cache is the one the host would have laid out
    ref = QuestRun(w, inputs, mode="fused", out_dtype=out_dtype)
    assert run.kv.ctx_len.tolist() == list(w.ctx)
    for b, L in enumerate(w.ctx):
        for what in ("k", "v"):
            assert torch.equal(logical(run, b, what, L), logical(ref, b, what, L))
        n = -(-L // 16)
        assert torch.equal(run.kv.meta[b, :n], ref.kv.meta[b, :n])
    for s in range(w.steps):
        run.step(s)
        ref.step(s)
        torch.cuda.synchronize()
        assert torch.equal(run.n_sel, ref.n_sel)
        for u in range(w.batch * H):
            k = int(ref.n_sel[u])
            assert torch.equal(run.sel[u, :k], ref.sel[u, :k])
        assert torch.equal(run.out, ref.out) and torch.equal(run.lse, ref.lse)
    assert run.status() == 0
    held = run.pool.n_pages.tolist()
    assert held == [-(-(c + w.steps) // 16) for c in w.ctx]
    run.release(torch.tensor([1, 0, 1, 0], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert int(run.pool.n_free) == held[0] + held[2] and run.pool.ctx_len[0] == 0
    assert run.status() == 0


def test_prompt_prefill_at_full_size_sampled():
    """One sequence of the 32K workload: its last 2048-token chunk, sampled rows."""
    w = synth.scaled(synth.workloads()["quest_32k"], name="prompt_32k", batch=1, ctx=(32768,),
                     budget=(2048,), steps=1)
    inputs, pq = synth.quest_inputs(w), synth.prompt_queries(w)
    run = PromptRun(w, inputs, pq, 8192)
    G, H = run.Hq // run.Hkv, run.Hkv
    for first, new in run.prefill():
        rows = [0, 1, 4000, 8191]
        out = run.out_rows[rows].double().cpu().numpy()
        for h in range(H):
            K, V = (oracle.widen(inputs[x][0][h]) for x in ("k", "v"))
            for i, r in enumerate(rows):
                t = int(first[0]) + r
                o, _ = oracle.attend(oracle.widen(pq[0][t, h * G:(h + 1) * G]), K[:t + 1], V[:t + 1],
                                     1 / math.sqrt(w.head_dim))
                assert max_abs(out[i, h * G:(h + 1) * G], o) <= TOL_BF16
    assert run.status() == 0
