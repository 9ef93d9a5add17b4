"""Cases of the operators around the paged cache that a serving loop needs beside the chunk
calls: rotary positions with per-head norms, the append that applies them, the check of drafted
tokens, forked sequences, and sequences cut back.

Five kinds of case ("op"):
  "rope"      se_qk_rope: queries and keys normalised per head and rotated to their positions.
  "append"    se_rope_append_chunk: the same, with the keys and values of a chunk of new tokens
              written into their pages, page summaries folded, lengths committed.
  "verify"    se_draft_verify: which drafted tokens stay, and the token behind them.
  "fork"      se_pages_truncate of the earlier samples to nothing, se_pages_fork of new ones from
              their prompts, se_pages_carry of one layer: the turnover of parallel samples.
              The pages let go come back in the order they were taken, so the same pass on
              the same state gives the same tables.
  "rollback"  a step whose drafts are partly refused: se_chunk_plan, se_rope_append_chunk,
              se_pages_truncate to the kept lengths, se_pages_carry of one layer.  From the second
              pass on a state begins and ends at the kept lengths.

Where `own` is false the same results come from elementary torch operations in 32 bits (64 for
angles and for sums that decide which token is drawn).  Lengths are a function of the case (its
"lens" number), values of the seed.
"""
import math
import random

import torch

own = False

PAGE = 16
DEV = "cuda"
EPS = 1e-6


def listed():
    return [
        # one token of 64 decoding sequences ahead of a sparse decode call: call latency
        dict(name="rope_decode_64", op="rope", rows=64, heads=32, kv=4, dim=128, rot=128, pair=False,
             norm=True, scaling="none", far=32768, pad=0),
        # 16K packed prompt rows of a long-context layer, interleaved pairs on half of each head
        dict(name="rope_far_16k", op="rope", rows=16384, heads=8, kv=8, dim=64, rot=32, pair=True,
             norm=False, scaling="yarn", far=1 << 20, pad=0),
        # 64 decoding sequences, one token each: call latency
        dict(name="append_decode_64", op="append", batch=64, heads=32, kv=4, dim=128, rot=128,
             pair=False, norm=True, scaling="none", decodes=64, new_lo=1, new_hi=1, ctx_lo=0,
             ctx_hi=2000, summaries=True, pad=0, lens=1),
        # ragged chunks beside decoding sequences, part of each head rotated, padded rows
        dict(name="append_ragged_d64", op="append", batch=9, heads=8, kv=8, dim=64, rot=48,
             pair=True, norm=False, scaling="bands", decodes=3, new_lo=5, new_hi=700, ctx_lo=0,
             ctx_hi=999, summaries=False, pad=11, lens=2),
        # eight prompts of 8192 tokens: memory bound, the largest
        dict(name="append_8x8k", op="append", batch=8, heads=32, kv=4, dim=128, rot=128, pair=False,
             norm=True, scaling="none", decodes=0, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0,
             summaries=True, pad=0, lens=3),
        # one sequence, four drafted tokens: call latency
        dict(name="verify_one", op="verify", batch=1, new_lo=5, new_hi=5, vocab=32000, drafter=True,
             half=False, lens=4),
        # an odd batch whose drafts were looked up, not drawn: no draft probabilities; odd rows
        dict(name="verify_lookup_37", op="verify", batch=37, new_lo=1, new_hi=9, vocab=50001,
             drafter=False, half=True, lens=5),
        # 256 sequences with five drafts each over a large vocabulary: memory bound
        dict(name="verify_256", op="verify", batch=256, new_lo=6, new_hi=6, vocab=131072,
             drafter=True, half=False, lens=6),
        # four samples of one prompt of about 2K tokens: call latency
        dict(name="fork_4", op="fork", prompts=1, samples=4, ctx_lo=1999, ctx_hi=1999, room=100,
             kv=1, dim=64, lens=7),
        # 64 samples of a prompt of about 32K tokens: page summaries, memory bound
        dict(name="fork_64x32k", op="fork", prompts=1, samples=64, ctx_lo=32761, ctx_hi=32761,
             room=100, kv=4, dim=128, lens=8),
        # 16 sequences of up to 32K tokens, 8 drafts each, some kept
        dict(name="rollback_16", op="rollback", batch=16, heads=32, kv=4, dim=128, rot=128,
             pair=False, norm=True, scaling="none", decodes=0, new_lo=8, new_hi=8, ctx_lo=100,
             ctx_hi=32000, summaries=True, pad=0, lens=9),
        # 256 sequences with up to 65 new tokens each, cut back anywhere in them
        dict(name="rollback_256", op="rollback", batch=256, heads=8, kv=4, dim=128, rot=64,
             pair=False, norm=True, scaling="linear", decodes=20, new_lo=1, new_hi=65, ctx_lo=0,
             ctx_hi=3000, summaries=True, pad=7, lens=10),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["rope", "append", "append", "verify", "verify", "fork", "rollback"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 8])
    lens = rng.randrange(1 << 30)
    turn = dict(rot=rng.choice([dim, dim, 16 * rng.randint(1, dim // 16)]), pair=rng.random() < 0.4,
                norm=rng.random() < 0.6,
                scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]))
    if op == "rope":
        return dict(op=op, rows=_spread(rng, 1, (1 << 19) // (heads + kv) * 64 // dim), heads=heads,
                    kv=kv, dim=dim, far=_spread(rng, 16, 1 << 20), pad=rng.choice([0, 3]), **turn)
    if op == "verify":
        batch = _spread(rng, 1, 256)
        hi = _spread(rng, 1, 12)
        vocab = _spread(rng, 100, 131072 if batch * hi <= 1536 else 131072 * 1536 // (batch * hi))
        return dict(op=op, batch=batch, new_lo=rng.randint(1, hi), new_hi=hi, vocab=vocab,
                    drafter=rng.random() < 0.7, half=rng.random() < 0.4, lens=lens)
    if op == "fork":
        prompts = _spread(rng, 1, 16)
        samples = _spread(rng, prompts, 128)
        hi = _spread(rng, 1, min(32768, (1 << 30) // (kv * dim * (samples + prompts))))
        return dict(op=op, prompts=prompts, samples=samples, ctx_lo=max(1, hi // 2), ctx_hi=hi,
                    room=rng.choice([100, 100, 60]), kv=kv, dim=dim, lens=lens)
    batch = _spread(rng, 1, 256)
    rows = 65536 * 40 * 128 // ((heads + 2 * kv) * dim)
    hi = _spread(rng, 1, min(65536, rows) // batch if op == "append" else 200)
    return dict(op=op, batch=batch, heads=heads, kv=kv, dim=dim, decodes=rng.randint(0, batch),
                new_lo=rng.randint(1, hi), new_hi=hi, ctx_lo=0, ctx_hi=_spread(rng, 1, 4000),
                summaries=rng.random() < 0.7, pad=rng.choice([0, 5]), lens=lens, **turn)


# ---------------------------------------------------------------------------
# a case's lengths
# ---------------------------------------------------------------------------

def _lengths(case):
    """(tokens held, new tokens) of each sequence: the case's, whatever the seed."""
    r = random.Random(case["lens"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    for b in r.sample(range(case["batch"]), case["decodes"]):
        new[b] = 1
    return ctx, new


def _kept(case):
    """Of each sequence's new tokens: those that a rollback keeps."""
    r = random.Random(case["lens"] + 1)
    return [r.randint(0, n) for n in _lengths(case)[1]]


def _drafts(case):
    """Rows of each sequence: the last token that stands, then the drafts."""
    r = random.Random(case["lens"])
    return [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]


def _forks(case):
    """(prompt lengths, source of each sample); the prompts are sequences 0.., the samples behind."""
    r = random.Random(case["lens"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["prompts"])]
    src = [r.randrange(case["prompts"]) for _ in range(case["samples"])]
    return ctx, src


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).bfloat16()


class State:
    pass


# ---------------------------------------------------------------------------
# rotary frequencies
# ---------------------------------------------------------------------------

BASE = {"none": 1e4, "linear": 1e4, "ntk": 1e4, "yarn": 1e6, "bands": 5e5}
FACTOR, BEFORE = 8.0, 4096.0           # a context eight times the 4096 positions there were


def _frequencies(case):
    """(radians a position of each pair, factor on cos and sin), for the scaling of the case."""
    kind, R = case["scaling"], case["rot"]
    base = BASE[kind]
    if kind == "ntk":
        base *= FACTOR ** (R / (R - 2))
    f = torch.tensor([base ** (-2 * i / R) for i in range(R // 2)], dtype=torch.float64)
    if kind == "linear":
        return f / FACTOR, 1.0
    if kind == "yarn":
        at = [R * math.log(BEFORE / (beta * 2 * math.pi)) / (2 * math.log(base)) for beta in (32, 1)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
        ramp = ((torch.arange(R // 2).double() - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / FACTOR * ramp, 0.1 * math.log(FACTOR) + 1
    if kind == "bands":
        smooth = ((BEFORE * f / (2 * math.pi) - 1) / (4 - 1)).clamp(0, 1)
        return f / FACTOR * (1 - smooth) + f * smooth, 1.0
    return f, 1.0


def _rope_handle(s):
    case = s.case
    D = case["dim"]
    s.freq, s.amp = _frequencies(case)
    s.freq = s.freq.to(DEV)
    s.qw = s.kw = None
    if case["norm"]:
        s.qw, s.kw = ((1 + 0.3 * torch.randn(D, generator=s.gen, device=DEV)).bfloat16()
                      for _ in range(2))
    if own:
        from kv_cache_decode_quest_gb300 import binding as se
        kind = {"none": se.SE_ROPE_PLAIN, "linear": se.SE_ROPE_LINEAR, "ntk": se.SE_ROPE_NTK,
                "yarn": se.SE_ROPE_YARN, "bands": se.SE_ROPE_BANDS}[case["scaling"]]
        low, high = (1.0, 32.0) if case["scaling"] == "yarn" else (1.0, 4.0)
        s.rope = se.Rope.make(case["rot"], base=BASE[case["scaling"]], scaling=kind, factor=FACTOR,
                              original_len=BEFORE, low=low, high=high,
                              layout=se.SE_ROPE_PAIRS if case["pair"] else se.SE_ROPE_HALVES,
                              q_weight=s.qw, k_weight=s.kw, eps=EPS)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _keys(g, rows, kv, dim):
    """Keys with four channels eight times as large in every head."""
    scale = torch.ones(kv, dim, device=DEV)
    at = torch.rand(kv, dim, generator=g, device=DEV).argsort(1)[:, :4]
    scale.scatter_(1, at, 8.0)
    return (torch.randn(rows, kv, dim, generator=g, device=DEV) * scale).bfloat16()


def _projection(s, rows):
    """Packed q | k | v rows, as a fused projection leaves them."""
    H, Hq, D = s.case["kv"], s.case["heads"], s.case["dim"]
    qkv = _bf16(s.gen, rows, Hq + 2 * H, D)
    qkv[:, Hq:Hq + H] = _keys(s.gen, rows, H, D)
    s.q, s.k_new, s.v_new = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]


def _packed(s, new, first, rows):
    """start, seq, pos of packed rows, `first` the first position of each sequence."""
    B, total = len(new), sum(new)
    s.start = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    s.start[1:] = torch.cumsum(_ints(new), 0)
    b = torch.repeat_interleave(torch.arange(B, device=DEV), _ints(new).long(), output_size=total)
    pos = _ints(first)[b] + torch.arange(total, device=DEV) - s.start[b]
    tail = torch.full((rows - total,), -1, dtype=torch.int32, device=DEV)
    s.seq, s.pos = (torch.cat([x.int(), tail]) for x in (b, pos))
    return b, pos


def _cache(s, num_pages, batch, held):
    """K, V pages and, where kept, the summaries of what is held."""
    H, D, g = s.case["kv"], s.case["dim"], s.gen
    s.k = _keys(g, num_pages * PAGE, H, D).view(num_pages, PAGE, H, D).transpose(1, 2).contiguous()
    s.v = _bf16(g, num_pages, H, PAGE, D)
    s.meta = None
    if s.case.get("summaries", True):
        s.meta = torch.zeros(batch, s.maxp, H, 2, D, dtype=torch.bfloat16, device=DEV)
        for b, n in enumerate(held):                    # pages without a held token have none yet
            if n:
                p = -(-n // PAGE)
                k = s.k[s.block_table[b, :p].long()].float()
                live = torch.arange(p * PAGE, device=DEV).view(p, 1, PAGE, 1) < n
                s.meta[b, :p, :, 0] = torch.where(live, k, math.inf).amin(2).bfloat16()
                s.meta[b, :p, :, 1] = torch.where(live, k, -math.inf).amax(2).bfloat16()


def _pool(s, held, num_pages, batch):
    """A pool whose first sequences hold the pages of `held` tokens, the rest on the stack."""
    pages = [-(-n // PAGE) for n in held]
    perm = torch.randperm(num_pages, generator=s.gen, device=DEV).int()
    s.num_pages, s.free_pages = num_pages, perm.clone()
    s.n_free = _ints([num_pages - sum(pages)])
    s.n_pages = _ints(pages + [0] * (batch - len(held)))
    s.ctx_len = _ints(list(held) + [0] * (batch - len(held)))
    first = torch.cumsum(s.n_pages, 0) - s.n_pages
    p = torch.arange(s.maxp, device=DEV)[None, :]
    where = (num_pages - 1 - first[:, None] - p).clamp(min=0)
    s.block_table = torch.where(p < s.n_pages[:, None], perm[where.long()], -1).int().contiguous()
    s.refs = torch.zeros(num_pages, dtype=torch.int32, device=DEV)
    s.from_seq, s.from_page = (torch.full((batch,), -1, dtype=torch.int32, device=DEV)
                               for _ in range(2))


def prepare(case, seed):
    s = State()
    s.case = case
    s.gen = torch.Generator(device=DEV)
    s.gen.manual_seed(int(seed))
    globals()["_prepare_" + case["op"]](s, case)
    del s.gen
    return s


def _prepare_rope(s, case):
    rows = case["rows"] + case["pad"]
    _rope_handle(s)
    _projection(s, rows)
    s.pos = torch.randint(0, case["far"], (rows,), generator=s.gen, device=DEV, dtype=torch.int32)
    s.pos[case["rows"]:] = -1                           # rows of no token
    s.q_out, s.k_out = (torch.zeros(rows, h, case["dim"], dtype=torch.bfloat16, device=DEV)
                        for h in (case["heads"], case["kv"]))
    if own:
        from kv_cache_decode_quest_gb300 import binding as se
        s.ws = se.workspace(se.se_small_workspace())


def _prepare_append(s, case):
    ctx, new = _lengths(case)
    _rope_handle(s)
    pages = [-(-(c + n) // PAGE) for c, n in zip(ctx, new)]
    s.maxp = max(pages) + 2
    _pool(s, [c + n for c, n in zip(ctx, new)], sum(pages) + 3, len(ctx))
    s.ctx_len = _ints(ctx)
    rows = sum(new) + case["pad"]
    b, pos = _packed(s, new, ctx, rows)
    s.slot = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    s.slot[:len(b)] = (s.block_table[b, pos // PAGE] * PAGE + pos % PAGE).int()
    _projection(s, rows)
    _cache(s, s.num_pages, len(ctx), ctx)
    s.q_out = torch.zeros(rows, case["heads"], case["dim"], dtype=torch.bfloat16, device=DEV)
    if own:
        from kv_cache_decode_quest_gb300 import binding as se
        s.kv = se.PagedKV(s.k, s.v, s.meta, s.block_table, s.ctx_len)
        s.chunk = se.Chunk(s.start, s.seq, s.pos, s.slot)
        s.ws = se.workspace(se.se_small_workspace())


def _prepare_verify(s, case):
    new, V, g = _drafts(case), case["vocab"], s.gen
    rows = sum(new)
    _packed(s, new, [100 + 3 * b for b in range(len(new))], rows)
    s.slot = torch.zeros_like(s.seq)                    # not looked at
    t = torch.float32 if not case["half"] else torch.bfloat16
    s.p = torch.empty(rows, V, dtype=t, device=DEV)
    s.draft = torch.empty(rows, V, dtype=t, device=DEV) if case["drafter"] else None
    s.tokens = torch.zeros(rows, dtype=torch.int32, device=DEV)
    for lo in range(0, rows, 256):                      # few rows at once: the vocabulary is large
        hi = min(rows, lo + 256)
        x = torch.randn(hi - lo, V, generator=g, device=DEV) * 3
        s.p[lo:hi] = torch.softmax(x, 1).to(t)
        x += 0.4 * torch.randn(hi - lo, V, generator=g, device=DEV)
        y = torch.softmax(x, 1)
        if s.draft is not None:
            s.draft[lo:hi] = y.to(t)
        e = torch.empty_like(y).exponential_(generator=g)
        tok = (y / e).argmax(1).int()                   # drawn from y; row t's is the token of row t + 1
        s.tokens[lo + 1:hi + 1] = tok[:len(s.tokens[lo + 1:hi + 1])]
    s.accept_u = torch.rand(rows, generator=g, device=DEV)
    s.sample_u = torch.rand(len(new), generator=g, device=DEV)
    s.n_accepted, s.next_token, s.keep = (torch.zeros(len(new), dtype=torch.int32, device=DEV)
                                          for _ in range(3))
    if own:
        from kv_cache_decode_quest_gb300 import binding as se
        s.chunk = se.Chunk(s.start, s.seq, s.pos, s.slot)
        s.ws = se.workspace(se.se_draft_verify_workspace(len(new), V))


def _prepare_fork(s, case):
    ctx, src = _forks(case)
    N = len(ctx) + len(src)
    pages = [-(-c // PAGE) for c in ctx]
    last = sum(1 for x in src if ctx[x] % PAGE)
    s.maxp = max(pages) + 1
    _pool(s, ctx, sum(pages) + last * case["room"] // 100 + (3 if case["room"] == 100 else 0), N)
    s.src = _ints([-1] * len(ctx) + src)
    s.none = _ints([-1] * len(ctx) + [0] * len(src))    # lengths that the earlier samples are cut to
    _cache(s, s.num_pages, N, ctx)
    if own:
        from kv_cache_decode_quest_gb300 import binding as se
        s.kv = se.PagedKV(s.k, s.v, s.meta, s.block_table, s.ctx_len)
        s.pool = se.PagePool(s.free_pages, s.n_free, s.n_pages, s.block_table, s.ctx_len)
        s.carry = se.Carry(s.from_seq, s.from_page)
        s.ws = se.workspace(se.se_pages_truncate_workspace(N, s.num_pages))


def _prepare_rollback(s, case):
    ctx, new = _lengths(case)
    _rope_handle(s)
    after = [-(-(c + 2 * n) // PAGE) for c, n in zip(ctx, new)]
    s.maxp = max(after) + 1
    _pool(s, ctx, sum(after) + 2, len(ctx))
    s.new_len = _ints(new)
    s.keep = _ints([c + k for c, k in zip(ctx, _kept(case))])
    rows = sum(new) + case["pad"]
    _projection(s, rows)
    _cache(s, s.num_pages, len(ctx), ctx)
    s.q_out = torch.zeros(rows, case["heads"], case["dim"], dtype=torch.bfloat16, device=DEV)
    s.start = torch.zeros(len(ctx) + 1, dtype=torch.int32, device=DEV)
    s.seq, s.pos, s.slot = (torch.zeros(rows, dtype=torch.int32, device=DEV) for _ in range(3))
    if own:
        from kv_cache_decode_quest_gb300 import binding as se
        s.kv = se.PagedKV(s.k, s.v, s.meta, s.block_table, s.ctx_len)
        s.pool = se.PagePool(s.free_pages, s.n_free, s.n_pages, s.block_table, s.ctx_len)
        s.chunk = se.Chunk(s.start, s.seq, s.pos, s.slot)
        s.carry = se.Carry(s.from_seq, s.from_page)
        s.ws = se.workspace(se.se_pages_truncate_workspace(len(ctx), s.num_pages))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case, op = s.case, s.case["op"]
    if own:
        from kv_cache_decode_quest_gb300 import binding as se
        if op == "rope":
            se.se_qk_rope(s.rope, s.pos, s.q, s.k_new, s.q_out, s.k_out, s.ws)
        elif op == "append":
            se.se_rope_append_chunk(s.kv, s.rope, s.q, s.k_new, s.v_new, s.q_out, s.chunk,
                                    case["batch"], s.ws)
        elif op == "verify":
            se.se_draft_verify(s.p, s.draft, s.tokens, s.accept_u, s.sample_u, s.chunk,
                               case["batch"], s.n_accepted, s.next_token, s.keep, s.ws)
        elif op == "fork":
            B = case["prompts"] + case["samples"]
            se.se_pages_truncate(s.pool, s.refs, s.none, B, s.carry, s.ws)
            se.se_pages_fork(s.pool, s.refs, s.src, B, s.carry, s.ws)
            se.se_pages_carry(s.kv, s.carry, B, s.ws)
        else:
            B = case["batch"]
            se.se_chunk_plan(s.pool, s.new_len, B, s.chunk, s.ws)
            se.se_rope_append_chunk(s.kv, s.rope, s.q, s.k_new, s.v_new, s.q_out, s.chunk, B, s.ws)
            se.se_pages_truncate(s.pool, s.refs, s.keep, B, s.carry, s.ws)
            se.se_pages_carry(s.kv, s.carry, B, s.ws)
    elif op == "rope":
        live = (s.pos >= 0)[:, None, None]
        s.q_out.copy_(torch.where(live, _turned_plain(s, s.q, s.qw), s.q_out.float()))
        s.k_out.copy_(torch.where(live, _turned_plain(s, s.k_new, s.kw), s.k_out.float()))
    elif op == "append":
        _append_plain(s)
    elif op == "verify":
        _verify_plain(s)
    elif op == "fork":
        _truncate_plain(s, s.none)
        _fork_plain(s)
        _carry_plain(s)
    else:
        _plan_plain(s)
        _append_plain(s)
        _truncate_plain(s, s.keep)
        _carry_plain(s)
    if op == "rope":
        return dict(q_out=s.q_out, k_out=s.k_out)
    if op == "verify":
        return dict(n_accepted=s.n_accepted, next_token=s.next_token, keep=s.keep)
    out = dict(k=s.k, v=s.v, meta=s.meta, ctx_len=s.ctx_len)
    if op != "fork":
        out["q_out"] = s.q_out
    if op != "append":
        out.update(free_pages=s.free_pages, n_free=s.n_free, n_pages=s.n_pages, refs=s.refs,
                   block_table=s.block_table, from_seq=s.from_seq, from_page=s.from_page)
    return out


def _turned_plain(s, x, w):
    R = s.case["rot"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    angle = s.pos.double()[:, None] * s.freq                       # 64 bits: positions are far
    cos, sin = ((s.amp * y).float()[:, None, :] for y in (torch.cos(angle), torch.sin(angle)))
    if s.case["pair"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., R:]], -1)


def _append_plain(s):
    """Rows past the last sequence have no slot; they go to a page of their own, which is dropped."""
    q, k = _turned_plain(s, s.q, s.qw), _turned_plain(s, s.k_new, s.kw).bfloat16()
    ok = s.slot >= 0
    s.q_out.copy_(torch.where(ok[:, None, None], q, s.q_out.float()))
    page = torch.where(ok, s.slot // PAGE, s.num_pages).long()
    off = torch.where(ok, s.slot % PAGE, 0).long()
    for cache, rows in ((s.k, k), (s.v, s.v_new)):
        wide = torch.cat([cache, cache[:1]])
        wide[page, :, off] = rows
        cache.copy_(wide[:-1])
    B = s.case["batch"]
    if s.meta is not None:
        H, D, n = s.case["kv"], s.case["dim"], B * s.maxp
        at = torch.where(ok, s.seq * s.maxp + s.pos // PAGE, n).long()
        begins = torch.zeros(n + 1, device=DEV)
        begins.scatter_reduce_(0, at, (ok & (s.pos % PAGE == 0)).float(), "amax")
        begins = begins.view(-1, 1, 1) > 0                         # pages that begin here
        old = torch.cat([s.meta.view(n, H, 2, D), s.meta.view(n, H, 2, D)[:1]]).float()
        lo = torch.where(begins, math.inf, old[:, :, 0])
        hi = torch.where(begins, -math.inf, old[:, :, 1])
        rows = at.view(-1, 1, 1).expand(-1, H, D)
        lo.scatter_reduce_(0, rows, k.float(), "amin")
        hi.scatter_reduce_(0, rows, k.float(), "amax")
        s.meta.copy_(torch.stack([lo, hi], 2)[:-1].view(B, s.maxp, H, 2, D))
    length = torch.cat([s.ctx_len, s.ctx_len[:1]])
    length.scatter_reduce_(0, torch.where(ok, s.seq, B).long(), s.pos + 1, "amax")
    s.ctx_len.copy_(length[:-1])


def _verify_plain(s):
    B, n = s.case["batch"], s.case["new_hi"]
    first, rows = s.start[:-1].long(), s.start[1:].long() - s.start[:-1].long()
    i = torch.arange(n - 1, device=DEV)
    t = (first[:, None] + i).clamp(max=len(s.tokens) - 1)           # the row that a draft follows
    d = (t + 1).clamp(max=len(s.tokens) - 1)
    tok = s.tokens[d].long()
    q = 1.0 if s.draft is None else s.draft[t, tok].double()
    ok = (s.accept_u[d].double() * q < s.p[t, tok].double()) & (i < rows[:, None] - 1)
    n_ok = torch.cumprod(ok.int(), 1).sum(1)
    r = first + n_ok
    p = s.p[r].double()
    refused = (n_ok < rows - 1)[:, None]
    if s.draft is None:
        at = s.tokens[(r + 1).clamp(max=len(s.tokens) - 1)].long()[:, None]
        rest = p.scatter(1, at, 0.0)
    else:
        rest = (p - s.draft[r].double()).clamp(min=0)
    rest = torch.where(refused, rest, p)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p)
    upto = torch.cumsum(rest, 1)                                    # 64 bits: it decides a token
    s.next_token.copy_((upto <= s.sample_u.double()[:, None] * upto[:, -1:]).sum(1))
    s.n_accepted.copy_(n_ok)
    s.keep.copy_(s.pos[first] + 1 + n_ok)


def _plan_plain(s):
    B, ctx, new, held = s.case["batch"], s.ctx_len, s.new_len, s.n_pages
    need = ((ctx + new + PAGE - 1) // PAGE - held).clamp(min=0)
    upto = torch.cumsum(need, 0)
    p = torch.arange(s.maxp, device=DEV)[None, :]
    fresh = (p >= held[:, None]) & (p < (held + need)[:, None])
    at = s.n_free - 1 - ((upto - need - held)[:, None] + p)
    s.block_table.copy_(torch.where(fresh, s.free_pages[at.clamp(0, s.num_pages - 1).long()],
                                    s.block_table))
    s.start[1:] = torch.cumsum(new, 0)
    t = torch.arange(len(s.seq), device=DEV)
    b = torch.searchsorted(s.start[1:].contiguous(), t.int(), right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    pos = ctx[b] + t - s.start[b]
    slot = s.block_table[b, (pos // PAGE).clamp(max=s.maxp - 1)] * PAGE + pos % PAGE
    s.seq.copy_(torch.where(live, b, -1))
    s.pos.copy_(torch.where(live, pos, -1))
    s.slot.copy_(torch.where(live, slot, -1))
    s.n_pages += need
    s.n_free -= upto[-1]


def _truncate_plain(s, keep):
    ctx, held, maxp, P = s.ctx_len, s.n_pages, s.maxp, s.num_pages
    n = torch.minimum(keep, ctx)
    after = (n + PAGE - 1) // PAGE
    part = (keep >= 0) & (n % PAGE != 0)
    last = s.block_table.gather(1, (after - 1).clamp(min=0)[:, None].long())[:, 0]
    copy = part & (s.refs[last.clamp(min=0).long()] > 0)             # the page is shared: take one
    upto = torch.cumsum(copy.int(), 0)
    act = (keep >= 0) & (~copy | (upto <= s.n_free))
    copy &= act
    fresh = s.free_pages[(s.n_free - upto).clamp(min=0).long()]
    taken = copy.sum()
    p = torch.arange(maxp, device=DEV)[None, :]
    go = act[:, None] & (p < held[:, None]) & (p >= (after - copy.int())[:, None])
    go &= (p >= after[:, None]) | copy[:, None]
    page = torch.where(go, s.block_table, P).long()
    b = torch.arange(1, len(ctx) + 1, device=DEV)[:, None].expand_as(page)
    holders = torch.zeros(P + 1, dtype=torch.int32, device=DEV)
    holders.scatter_add_(0, page.reshape(-1), torch.ones_like(page.reshape(-1)).int())
    who = torch.zeros(P + 1, dtype=torch.int64, device=DEV)
    who.scatter_reduce_(0, page.reshape(-1), b.reshape(-1), "amax")   # its last sequence in this call
    left = torch.cat([s.refs, s.refs[:1]]) - holders
    freed = go & (left[page] < 0) & (who[page] == b)
    rank = torch.cumsum(freed.reshape(-1), 0).view_as(page)
    total = rank[-1, -1]
    at = torch.where(freed, s.n_free - taken + total - rank, P)       # one word past the stack: dropped
    stack = torch.cat([s.free_pages, s.free_pages[:1]])
    stack.scatter_(0, at.reshape(-1).long(), page.reshape(-1).int())
    s.free_pages.copy_(stack[:-1])
    s.refs.copy_(left[:-1].clamp(min=0))
    s.n_free += total - taken
    s.block_table.copy_(torch.where(copy[:, None] & (p == after[:, None] - 1), fresh[:, None],
                                    s.block_table))
    s.from_page.copy_(torch.where(act & part & (copy | (n < ctx)), last, -1))
    s.from_seq.fill_(-1)
    s.n_pages.copy_(torch.where(act, after, held))
    s.ctx_len.copy_(torch.where(act, n, ctx))


def _fork_plain(s):
    want, maxp, P = s.src >= 0, s.maxp, s.num_pages
    src = s.src.clamp(min=0).long()
    ctx = s.ctx_len[src]
    pages, full = (ctx + PAGE - 1) // PAGE, ctx // PAGE
    need = want & (ctx % PAGE != 0)
    upto = torch.cumsum(need.int(), 0)
    ok = want & (~need | (upto <= s.n_free))
    take = ok & need
    fresh = s.free_pages[(s.n_free - upto).clamp(min=0).long()]
    p = torch.arange(maxp, device=DEV)[None, :]
    theirs = s.block_table[src]
    share = ok[:, None] & (p < full[:, None])
    refs = torch.cat([s.refs, s.refs[:1]])
    at = torch.where(share, theirs, P).reshape(-1).long()
    refs.scatter_add_(0, at, torch.ones_like(at).int())
    s.refs.copy_(refs[:-1])
    last = theirs.gather(1, (pages - 1).clamp(min=0)[:, None].long())[:, 0]
    table = torch.where(share, theirs, s.block_table)
    s.block_table.copy_(torch.where(take[:, None] & (p == full[:, None]), fresh[:, None], table))
    s.from_seq.copy_(torch.where(ok, s.src, -1))
    s.from_page.copy_(torch.where(take, last, -1))
    s.n_pages.copy_(torch.where(ok, pages, s.n_pages))
    s.ctx_len.copy_(torch.where(ok, ctx, s.ctx_len))
    s.n_free -= take.sum()


def _carry_plain(s):
    n = s.ctx_len
    part = s.from_page >= 0
    last = s.block_table.gather(1, (n // PAGE).clamp(max=s.maxp - 1)[:, None].long())[:, 0]
    row = torch.arange(PAGE, device=DEV)[None, :] < (n % PAGE)[:, None]
    here = (part[:, None] & row)[:, None, :, None]                    # rows of the last page that are held
    old = s.from_page.clamp(min=0).long()
    to = torch.where(part, last, s.num_pages).long()
    for cache in (s.k, s.v):
        wide = torch.cat([cache, cache[:1]])
        wide[to] = torch.where(here, cache[old], wide[to])
        cache.copy_(wide[:-1])
    if s.meta is not None:
        p = torch.arange(s.maxp, device=DEV)[None, :]
        whole = ((s.from_seq >= 0)[:, None] & (p < (n // PAGE)[:, None]))[:, :, None, None, None]
        s.meta.copy_(torch.where(whole, s.meta[s.from_seq.clamp(min=0).long()], s.meta))
        k = s.k[old].float()
        fold = torch.stack([torch.where(here, k, math.inf).amin(2),
                            torch.where(here, k, -math.inf).amax(2)], 2).bfloat16()
        at = (part[:, None] & (p == (n // PAGE)[:, None]))[:, :, None, None, None]
        s.meta.copy_(torch.where(at, fold[:, None], s.meta))


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# ---------------------------------------------------------------------------

def _append_work(case, ctx, new):
    H, Hq, D, total = case["kv"], case["heads"], case["dim"], sum(new)
    pages = sum(-(-(c + n) // PAGE) - c // PAGE for c, n in zip(ctx, new))
    meta = pages * H * 2 * D * 2 if case["summaries"] else 0
    return dict(bytes=2 * total * (Hq + 2 * H) * D * 2 + meta + 12 * total,
                flops=total * (Hq + H) * (3 * case["rot"] + (4 * D if case["norm"] else 0)))


def work(case):
    op = case["op"]
    if op == "rope":
        rows, heads, D = case["rows"], case["heads"] + case["kv"], case["dim"]
        return dict(bytes=2 * rows * heads * D * 2 + 4 * rows,
                    flops=rows * heads * (3 * case["rot"] + (4 * D if case["norm"] else 0)))
    if op == "append":
        return _append_work(case, *_lengths(case))
    if op == "verify":
        # the row that the last token is drawn from, and the drafter's where a draft is refused: with
        # the logits of prepare a draft stays with probability 0.84
        size, V = 2 if case["half"] else 4, case["vocab"]
        two = sum(1 - 0.84 ** (n - 1) for n in _drafts(case)) if case["drafter"] else 0
        return dict(bytes=int(size * V * (case["batch"] + two)) + 16 * case["batch"], flops=0)
    if op == "fork":
        # per fork its table, the holders of its pages, its summaries and a page of keys and values
        H, D = case["kv"], case["dim"]
        ctx, src = _forks(case)
        some = sum(ctx[x] // PAGE for x in src)
        rows = sum(ctx[x] % PAGE for x in src)
        read = sum(ctx[x] // PAGE for x in set(src))
        last = sum(1 for x in src if ctx[x] % PAGE)
        return dict(bytes=some * (8 + H * 4 * D) + read * (4 + H * 4 * D) + rows * H * D * 8 +
                    last * H * 4 * D, flops=0)
    ctx, new = _lengths(case)
    kept = [c + k for c, k in zip(ctx, _kept(case))]
    w = _append_work(case, kept, new)
    rows = sum(k % PAGE for k in kept)
    if case["summaries"]:
        w["bytes"] += rows * case["kv"] * case["dim"] * 2 + len(ctx) * case["kv"] * 4 * case["dim"]
    w["bytes"] += 32 * len(ctx)
    return w


def _turned_exact(s, x, w):
    """The same turn as a product of complex numbers in 64 bits."""
    R, x = s.case["rot"], x.double()
    if w is not None:
        x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS)
        x = x * w.double()
    turn = torch.polar(torch.full((1,), float(s.amp), dtype=torch.float64, device=DEV).expand(
        len(s.pos), R // 2), torch.outer(s.pos.double(), s.freq))[:, None, :]
    y = x.clone()
    if s.case["pair"]:
        z = torch.complex(x[..., 0:R:2], x[..., 1:R:2]) * turn
        y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :R // 2], x[..., R // 2:R]) * turn
        y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
    return y


def _appended(s, k, v, meta, q_out, slot, seq, pos):
    """Rows into k, v (64 bits) page by page; the summaries of the pages that got any."""
    live = slot >= 0
    t = torch.nonzero(live)[:, 0]
    kr = _turned_exact(s, s.k_new, s.kw)[t]
    q_out[t] = _turned_exact(s, s.q, s.qw)[t]
    page, off = (slot[t] // PAGE).long(), (slot[t] % PAGE).long()
    k[page, :, off] = kr
    v[page, :, off] = s.v_new[t].double()
    if meta is None:
        return
    for b, lp in sorted(set(zip(seq[t].tolist(), (pos[t] // PAGE).tolist()))):
        rows = [i for i in _rows_of(s, t, b, lp)]
        lo, hi = kr[rows].amin(0), kr[rows].amax(0)
        if int(pos[t[rows[0]]]) % PAGE:
            lo, hi = torch.minimum(lo, meta[b, lp, :, 0]), torch.maximum(hi, meta[b, lp, :, 1])
        meta[b, lp, :, 0], meta[b, lp, :, 1] = lo, hi


def _rows_of(s, t, b, lp):
    """Rows (of the live ones) of sequence b in its logical page lp."""
    if getattr(s, "_index", None) is None:
        s._index = {}
        for i, key in enumerate(zip(s.seq[t].tolist(), (s.pos[t] // PAGE).tolist())):
            s._index.setdefault(key, []).append(i)
    return s._index[(b, lp)]


def exact(case, seed):
    op = case["op"]
    if op == "verify":
        return None                                      # whole numbers throughout
    if op in ("append", "rollback") and sum(_lengths(case)[1]) > 100000:
        return None
    s = prepare(case, seed)
    if op == "rope":
        live = (s.pos >= 0)[:, None, None]
        return {name: torch.where(live, _turned_exact(s, x, w), y.double()) for name, x, w, y in
                (("q_out", s.q, s.qw, s.q_out), ("k_out", s.k_new, s.kw, s.k_out))}
    k, v = s.k.double(), s.v.double()
    meta = None if s.meta is None else s.meta.double()
    out = dict(k=k, v=v, meta=meta, ctx_len=None)
    whole = ("free_pages", "n_free", "n_pages", "refs", "block_table", "from_seq", "from_page")
    if op == "append":
        out["q_out"] = s.q_out.double()
        _appended(s, k, v, meta, out["q_out"], s.slot, s.seq, s.pos)
        return out
    out.update({name: None for name in whole})
    if op == "fork":
        ctx, src = _forks(case)
        free, at = s.free_pages.tolist(), int(s.n_free)
        for i, x in enumerate(src):
            b, full, rows = len(ctx) + i, ctx[x] // PAGE, ctx[x] % PAGE
            if rows:
                if at == 0:
                    continue                             # no page was left for this one
                at -= 1
                page, old = free[at], int(s.block_table[x, full])
                k[page, :, :rows], v[page, :, :rows] = k[old, :, :rows], v[old, :, :rows]
                meta[b, full, :, 0] = k[old, :, :rows].amin(1)
                meta[b, full, :, 1] = k[old, :, :rows].amax(1)
            meta[b, :full] = meta[x, :full]
        return out
    ctx, new = _lengths(case)
    kept = [c + n for c, n in zip(ctx, _kept(case))]
    rows, at = [], int(s.n_free)
    free, table = s.free_pages.tolist(), s.block_table.tolist()
    for b, (c, n) in enumerate(zip(ctx, new)):
        for lp in range(-(-c // PAGE), -(-(c + n) // PAGE)):
            at -= 1
            table[b][lp] = free[at]
        rows += [(b, p, table[b][p // PAGE] * PAGE + p % PAGE) for p in range(c, c + n)]
    rows += [(-1, -1, -1)] * case["pad"]
    s.seq, s.pos, slot = (_ints(x) for x in zip(*rows))
    out["q_out"] = s.q_out.double()
    _appended(s, k, v, meta, out["q_out"], slot, s.seq, s.pos)
    for b, n in enumerate(kept):
        if meta is not None and n % PAGE and n < ctx[b] + new[b]:
            page = k[table[b][n // PAGE], :, :n % PAGE]
            meta[b, n // PAGE, :, 0], meta[b, n // PAGE, :, 1] = page.amin(1), page.amax(1)
    return out
