"""Cases of the paged-prefill operators: page tables from request lengths, the
append of a chunk of new tokens, and the attention of a chunk over the cache.

Three kinds of case ("op"):
  "tables"  se_pages_release of the finished sequences, then se_chunk_plan of
            the next requests: the turnover of a serving batch.  Releasing puts
            pages back in the order the plan took them, so the same call on
            the same state finds the same free list and gives the same tables.
  "append"  se_kv_append_chunk: new K/V rows into their pages by the slot map,
            page summaries folded, lengths committed.
  "attn"    se_chunk_attn: each new token's causal attention over its sequence.

Where `own` is false the same results come from elementary torch operations in
32 bits.  Sequence lengths are a function of the case (its "lens" number), the
values of the seed.
"""
import math
import random

import torch

own = False

PAGE = 16
DEV = "cuda"


def listed():
    return [
        # one query of the small 4/1-head, 64-wide layer over 2048 tokens: call latency
        dict(name="attn_one_2k_d64", op="attn", batch=1, heads=4, kv=1, dim=64, decodes=1, new_lo=1,
             new_hi=1, ctx_lo=2047, ctx_hi=2047, window=0, sink=0, fp32=False, pad=0, lens=1),
        # 16 sequences of 32K tokens checking 8 drafted tokens each: memory bound
        dict(name="attn_draft8_16x32k", op="attn", batch=16, heads=32, kv=4, dim=128, decodes=0,
             new_lo=8, new_hi=8, ctx_lo=32760, ctx_hi=32760, window=0, sink=0, fp32=False, pad=0,
             lens=2),
        # a mixed serving batch: two odd chunks beside fourteen decoding sequences, padded rows
        dict(name="attn_mixed_16", op="attn", batch=16, heads=32, kv=4, dim=128, decodes=14,
             new_lo=300, new_hi=511, ctx_lo=900, ctx_hi=8000, window=0, sink=0, fp32=False, pad=13,
             lens=3),
        # a whole prompt of 8192 tokens in one chunk: tensor bound, half the square masked
        dict(name="attn_prompt_8k", op="attn", batch=1, heads=32, kv=4, dim=128, decodes=0,
             new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0, window=0, sink=0, fp32=False, pad=0,
             lens=4),
        # the last 2048-token chunk of a 32K prompt: tensor bound, the largest
        dict(name="attn_chunk2k_at_32k", op="attn", batch=1, heads=32, kv=4, dim=128, decodes=0,
             new_lo=2048, new_hi=2048, ctx_lo=30720, ctx_hi=30720, window=0, sink=0, fp32=False,
             pad=0, lens=5),
        # ragged chunks under a sliding window with sink tokens, one head per KV head, fp32 output
        dict(name="attn_window_fp32", op="attn", batch=5, heads=8, kv=8, dim=64, decodes=1,
             new_lo=17, new_hi=1001, ctx_lo=0, ctx_hi=4099, window=1000, sink=4, fp32=True, pad=0,
             lens=6),
        # 64 decoding sequences, one token each: call latency
        dict(name="append_decode_64", op="append", batch=64, heads=32, kv=4, dim=128, decodes=64,
             new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=2000, summaries=True, packed=False, lens=7),
        # ragged chunks out of a packed q/k/v projection, a layer without page summaries
        dict(name="append_ragged_d64", op="append", batch=9, heads=8, kv=8, dim=64, decodes=3,
             new_lo=5, new_hi=700, ctx_lo=0, ctx_hi=999, summaries=False, packed=True, lens=8),
        # eight prompts of 8192 tokens: memory bound
        dict(name="append_8x8k", op="append", batch=8, heads=32, kv=4, dim=128, decodes=0,
             new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0, summaries=True, packed=True, lens=9),
        # a decode step's tables: 16 sequences, one token each, none finished
        dict(name="tables_decode_16", op="tables", batch=16, decodes=16, new_lo=1, new_hi=1,
             ctx_lo=1, ctx_hi=32768, done=0, room=100, pad=0, lens=10),
        # an odd batch with chunks, finished sequences and too few pages for the last requests
        dict(name="tables_short_257", op="tables", batch=257, decodes=200, new_lo=3, new_hi=700,
             ctx_lo=0, ctx_hi=4000, done=60, room=80, pad=31, lens=11),
        # every sequence of a batch of 1024 replaced by a prompt
        dict(name="tables_turnover_1024", op="tables", batch=1024, decodes=0, new_lo=1, new_hi=511,
             ctx_lo=1, ctx_hi=2000, done=1024, room=100, pad=0, lens=12),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm (0 counts as 1/2)."""
    a, b = math.log(max(lo, 0.5)), math.log(max(hi, 0.5))
    return max(lo, min(hi, int(round(math.exp(rng.uniform(a, b)) - (0.5 if lo == 0 else 0)))))


def draw(rng):
    """One more case of the listed ranges; the cost of an attention case is bounded by
    the padded score array that the plain form builds."""
    op = rng.choice(["attn", "attn", "attn", "append", "append", "tables"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8, 16])
    group = min(group, 64 // kv)
    lens = rng.randrange(1 << 30)
    if op == "tables":
        batch = _spread(rng, 1, 1024)
        hi = _spread(rng, 1, 1024)
        return dict(op=op, batch=batch, decodes=rng.randint(0, batch), new_lo=rng.randint(1, hi),
                    new_hi=hi, ctx_lo=rng.choice([0, 1]), ctx_hi=_spread(rng, 1, 4096),
                    done=rng.choice([0, batch // 3, batch]), room=rng.choice([100, 100, 70]),
                    pad=rng.choice([0, 7]), lens=lens)
    if op == "append":
        batch = _spread(rng, 1, 64)
        hi = _spread(rng, 1, 65536 // batch)
        return dict(op=op, batch=batch, heads=kv * group, kv=kv, dim=dim,
                    decodes=rng.randint(0, batch), new_lo=max(1, hi // 3), new_hi=hi, ctx_lo=0,
                    ctx_hi=_spread(rng, 1, 2000), summaries=rng.random() < 0.7,
                    packed=rng.random() < 0.5, lens=lens)
    batch = _spread(rng, 1, 16)
    hi = _spread(rng, 1, 4096)
    ctx = _spread(rng, 1, 32768)
    while batch * kv * group * hi * (ctx + hi) > 1 << 30:
        if hi >= ctx:
            hi = max(1, hi // 2 + 1) if hi > 3 else 1
        else:
            ctx = ctx // 2 + 1
    window = rng.choice([0, 0, _spread(rng, 1, 4096)])
    return dict(op=op, batch=batch, heads=kv * group, kv=kv, dim=dim,
                decodes=rng.randint(0, batch), new_lo=max(1, hi // 4), new_hi=hi,
                ctx_lo=rng.choice([0, ctx // 2]), ctx_hi=ctx, window=window,
                sink=rng.choice([0, 4, 100]) if window else 0, fp32=rng.random() < 0.3,
                pad=rng.choice([0, 5]), lens=lens)


def _lengths(case):
    """(tokens held, new tokens) of each sequence: the case's, whatever the seed."""
    r = random.Random(case["lens"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    for b in r.sample(range(case["batch"]), case["decodes"]):
        new[b] = 1
    return ctx, new


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class State:
    pass


def _chunk_rows(s, ctx, new, pad):
    """The packed rows of the new tokens (what a plan of them gives) and the paging."""
    g = s.gen
    B = len(ctx)
    s.total = sum(new)
    s.rows = s.total + pad
    pages = [-(-(c + n) // PAGE) for c, n in zip(ctx, new)]
    s.maxp = max(pages) + 2
    s.num_pages = sum(pages) + 3
    perm = torch.randperm(s.num_pages, generator=g, device=DEV).int()
    held = _ints(pages)
    first = torch.cumsum(held, 0) - held
    p = torch.arange(s.maxp, device=DEV)[None, :]
    s.block_table = torch.where(p < held[:, None], perm[(first[:, None] + p).clamp(max=s.num_pages - 1)],
                                -1).int().contiguous()
    n, c = _ints(new), _ints(ctx)
    s.start = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    s.start[1:] = torch.cumsum(n, 0)
    b = torch.repeat_interleave(torch.arange(B, device=DEV), n.long())
    pos = c[b] + torch.arange(s.total, device=DEV) - s.start[b]
    slot = s.block_table[b, pos // PAGE] * PAGE + pos % PAGE
    tail = torch.full((pad,), -1, dtype=torch.int32, device=DEV)
    s.seq, s.pos, s.slot = (torch.cat([x.int(), tail]) for x in (b, pos, slot))
    return c, n


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).bfloat16()


def _keys(g, rows, kv, dim):
    """Keys with four channels eight times as large in every head."""
    scale = torch.ones(kv, dim, device=DEV)
    at = torch.rand(kv, dim, generator=g, device=DEV).argsort(1)[:, :4]
    scale.scatter_(1, at, 8.0)
    return (torch.randn(rows, kv, dim, generator=g, device=DEV) * scale).bfloat16()


def prepare(case, seed):
    s = State()
    s.case = case
    s.gen = torch.Generator(device=DEV)
    s.gen.manual_seed(int(seed))
    op = case["op"]
    ctx, new = _lengths(case)
    if op == "tables":
        _prepare_tables(s, case, ctx, new)
    else:
        H, D, Hq = case["kv"], case["dim"], case["heads"]
        s.c, s.n = _chunk_rows(s, ctx, new, case.get("pad", 0))
        P = s.num_pages
        s.k = _keys(s.gen, P * PAGE, H, D).view(P, PAGE, H, D).transpose(1, 2).contiguous()
        s.v = _bf16(s.gen, P, H, PAGE, D)
        if op == "attn":
            s.q = _bf16(s.gen, s.rows, Hq, D)
            s.ctx_len = (s.c + s.n).int()
            s.scale = 1.0 / math.sqrt(D)
            s.out = torch.zeros(s.rows, Hq, D, dtype=torch.float32 if case["fp32"] else torch.bfloat16,
                                device=DEV)
            s.lse = torch.zeros(s.rows, Hq, dtype=torch.float32, device=DEV)
            s.meta = None
        else:
            s.ctx_len = s.c.clone()
            if case["packed"]:
                qkv = _bf16(s.gen, s.rows, Hq + 2 * H, D)
                qkv[:, Hq:Hq + H] = _keys(s.gen, s.rows, H, D)
                s.k_new, s.v_new = qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
            else:
                s.k_new, s.v_new = _keys(s.gen, s.rows, H, D), _bf16(s.gen, s.rows, H, D)
            s.meta = None
            if case["summaries"]:
                # summaries of what is held: pages without a held token have none yet
                k = s.k[s.block_table.clamp(min=0).long()].float()          # [B][maxp][H][16][D]
                tok = torch.arange(s.maxp * PAGE, device=DEV).view(1, s.maxp, 1, PAGE, 1)
                live = tok < s.c.view(-1, 1, 1, 1, 1)
                lo = torch.where(live, k, math.inf).amin(3)
                hi = torch.where(live, k, -math.inf).amax(3)
                s.meta = torch.stack([lo, hi], 3)
                s.meta = torch.where(s.meta.isinf(), 0.0, s.meta).bfloat16().contiguous()
    del s.gen
    if op != "tables":
        _handles(s)
    return s


def _prepare_tables(s, case, ctx, new):
    """A pool some of whose sequences are finished.  The held pages come from the top of
    a full stack in sequence order, finished sequences last, as a plan would take them."""
    B = case["batch"]
    r = random.Random(case["lens"] + 1)
    done = [0] * B
    for b in r.sample(range(B), case["done"]):
        done[b] = 1
    held = [-(-c // PAGE) for c in ctx]
    after = [-(-((0 if d else c) + n) // PAGE) for c, n, d in zip(ctx, new, done)]
    kept = sum(h for h, d in zip(held, done) if not d)
    gone = sum(h for h, d in zip(held, done) if d)
    need = sum(a if d else max(0, a - h) for a, h, d in zip(after, held, done))
    s.num_pages = kept + max(gone, -(-need * case["room"] // 100)) + (5 if case["room"] == 100 else 0)
    s.maxp = max(max(held), max(after)) + 1
    perm = torch.randperm(s.num_pages, generator=s.gen, device=DEV).int()
    s.free_pages = perm.clone()
    s.n_pages = _ints(held)
    order = [b for b in range(B) if not done[b]] + [b for b in range(B) if done[b]]
    first, at = [0] * B, 0
    for b in order:
        first[b] = at
        at += held[b]
    p = torch.arange(s.maxp, device=DEV)[None, :]
    where = (s.num_pages - 1 - _ints(first)[:, None] - p).clamp(min=0)
    s.block_table = torch.where(p < s.n_pages[:, None], perm[where.long()], -1).int().contiguous()
    s.n_free = _ints([s.num_pages - at])
    s.ctx_len, s.new_len, s.done = _ints(ctx), _ints(new), _ints(done)
    s.rows = sum(new) + case["pad"]
    s.start = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    s.seq, s.pos, s.slot = (torch.zeros(s.rows, dtype=torch.int32, device=DEV) for _ in range(3))
    if own:
        from kv_cache_decode_quest_gb300 import binding as se
        s.pool = se.PagePool(s.free_pages, s.n_free, s.n_pages, s.block_table, s.ctx_len)
        s.chunk = se.Chunk(s.start, s.seq, s.pos, s.slot)
        s.ws = se.workspace(se.se_page_pool_workspace(B))


def _handles(s):
    if own:
        from kv_cache_decode_quest_gb300 import binding as se
        case = s.case
        B = case["batch"]
        s.kv = se.PagedKV(s.k, s.v, s.meta, s.block_table, s.ctx_len)
        s.chunk = se.Chunk(s.start, s.seq, s.pos, s.slot)
        if case["op"] == "attn":
            s.ws = se.workspace(se.se_chunk_attn_workspace(B, s.rows, case["kv"], case["heads"],
                                                           case["dim"]))
        else:
            s.ws = se.workspace(se.se_small_workspace())


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case = s.case
    op, B = case["op"], case["batch"]
    if own:
        from kv_cache_decode_quest_gb300 import binding as se
        if op == "tables":
            se.se_pages_release(s.pool, s.done, B, s.ws)
            se.se_chunk_plan(s.pool, s.new_len, B, s.chunk, s.ws)
        elif op == "append":
            se.se_kv_append_chunk(s.kv, s.k_new, s.v_new, s.chunk, B, s.ws)
        else:
            se.se_chunk_attn(s.kv, s.q, s.chunk, B, case["heads"], s.scale, s.out, s.lse, s.ws,
                             out_dtype=int(case["fp32"]), window=case["window"], sink=case["sink"])
    elif op == "tables":
        _release_plain(s)
        _plan_plain(s)
    elif op == "append":
        _append_plain(s)
    else:
        _attn_plain(s)
    if op == "tables":
        return dict(free_pages=s.free_pages, n_free=s.n_free, n_pages=s.n_pages,
                    block_table=s.block_table, ctx_len=s.ctx_len, start=s.start, seq=s.seq,
                    pos=s.pos, slot=s.slot)
    if op == "append":
        return dict(k=s.k, v=s.v, meta=s.meta, ctx_len=s.ctx_len)
    return dict(out=s.out, lse=s.lse)


def _release_plain(s):
    held = torch.where(s.done != 0, s.n_pages, 0)
    upto = torch.cumsum(held, 0)
    count = upto[-1]
    p = torch.arange(s.maxp, device=DEV)[None, :]
    at = s.n_free + count - 1 - ((upto - held)[:, None] + p)
    at = torch.where(p < held[:, None], at, s.num_pages)              # one word past the stack: dropped
    stack = torch.cat([s.free_pages, s.free_pages[:1]])
    stack.scatter_(0, at.reshape(-1).long(), s.block_table.reshape(-1))
    s.free_pages.copy_(stack[:-1])
    s.n_free += count
    s.n_pages.mul_(s.done == 0)
    s.ctx_len.mul_(s.done == 0)


def _plan_plain(s):
    B = s.case["batch"]
    ctx, new, held = s.ctx_len, s.new_len, s.n_pages
    after = (ctx + new + PAGE - 1) // PAGE
    room = ctx + new <= s.maxp * PAGE
    need = torch.where(room, (after - held).clamp(min=0), 0)
    upto = torch.cumsum(need, 0)
    granted = room & (new > 0) & ((need == 0) | (upto <= s.n_free))
    take = torch.where(granted, need, 0)
    p = torch.arange(s.maxp, device=DEV)[None, :]
    fresh = (p >= held[:, None]) & (p < (held + take)[:, None])
    at = s.n_free - 1 - ((upto - need - held)[:, None] + p)
    page = s.free_pages[at.clamp(0, s.num_pages - 1).long()]
    s.block_table.copy_(torch.where(fresh, page, s.block_table))
    s.start[1:] = torch.cumsum(new, 0).clamp(max=s.rows)
    t = torch.arange(s.rows, device=DEV)
    b = torch.searchsorted(s.start[1:].contiguous(), t.int(), right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    ok = live & granted[b]
    pos = ctx[b] + t - s.start[b]
    slot = s.block_table[b, (pos // PAGE).clamp(0, s.maxp - 1)] * PAGE + pos % PAGE
    s.seq.copy_(torch.where(live, b, -1))
    s.pos.copy_(torch.where(ok, pos, -1))
    s.slot.copy_(torch.where(ok, slot, -1))
    s.n_pages += take
    s.n_free -= take.sum()


def _append_plain(s):
    page, off = (s.slot // PAGE).long(), (s.slot % PAGE).long()
    s.k[page, :, off] = s.k_new
    s.v[page, :, off] = s.v_new
    if s.meta is not None:
        B, maxp, H, _, D = s.meta.shape
        at = (s.seq * maxp + s.pos // PAGE).long()
        first = torch.zeros(B * maxp, device=DEV)
        first.scatter_reduce_(0, at, (s.pos % PAGE == 0).float(), "amax")
        first = first.view(-1, 1, 1) > 0                                   # pages that begin here
        old = s.meta.float().view(B * maxp, H, 2, D)
        lo = torch.where(first, math.inf, old[:, :, 0])
        hi = torch.where(first, -math.inf, old[:, :, 1])
        rows = at.view(-1, 1, 1).expand(-1, H, D)
        lo.scatter_reduce_(0, rows, s.k_new.float(), "amin")
        hi.scatter_reduce_(0, rows, s.k_new.float(), "amax")
        s.meta.copy_(torch.stack([lo, hi], 2).view(B, maxp, H, 2, D))
    s.ctx_len.scatter_reduce_(0, s.seq.long(), s.pos + 1, "amax")


def _attn_plain(s):
    case = s.case
    B, H, D, Hq = case["batch"], case["kv"], case["dim"], case["heads"]
    G, nmax, window, sink = Hq // H, case["new_hi"], case["window"], case["sink"]
    i = torch.arange(nmax, device=DEV)
    row = (s.start[:-1, None] + i).clamp(max=s.rows - 1).long()                   # [B][nmax]
    q = s.q[row].float().view(B, nmax, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, nmax * G, D)
    bt = s.block_table.clamp(min=0).long()
    L = s.maxp * PAGE
    j = torch.arange(L, device=DEV)
    held = (j < s.ctx_len[:, None])[:, None, :, None]                             # [B][1][L][1]
    k = s.k[bt].transpose(1, 2).reshape(B, H, L, D).float()
    v = torch.where(held, s.v[bt].transpose(1, 2).reshape(B, H, L, D).float(), 0.0)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s.scale)                          # [B][H][nmax*G][L]
    p = (s.pos[s.start[:-1].long()][:, None] + i)[:, :, None]                     # [B][nmax][1]
    see = (j <= p) & (j < s.ctx_len[:, None, None])
    if window:
        see &= (j > p - window) | (j < sink)
    see = see[:, None, :, None, :].expand(B, 1, nmax, G, L).reshape(B, 1, nmax * G, L)
    x.masked_fill_(~see, -math.inf)
    top = x.amax(3, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(3, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).view(B, H, nmax, G).permute(0, 2, 1, 3).reshape(B, nmax, Hq)
    o = o.view(B, H, nmax, G, D).permute(0, 2, 1, 3, 4).reshape(B, nmax, Hq, D)
    t = torch.arange(s.rows, device=DEV)
    live = s.seq >= 0
    b = s.seq.clamp(min=0).long()
    at = torch.where(live, t - s.start[b], 0)
    s.out.copy_(torch.where(live[:, None, None], o[b, at], s.out.float()))
    s.lse.copy_(torch.where(live[:, None], lse[b, at], s.lse))


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# ---------------------------------------------------------------------------

def _seen(ctx, new, window, sink):
    """(query-key pairs, distinct keys) of one sequence."""
    pairs, lowest = 0, ctx
    for p in range(ctx, ctx + new):
        if window and p + 1 > window:
            lo = p + 1 - window
            pairs += window + min(sink, lo)
        else:
            pairs += p + 1
    low = max(0, ctx + 1 - window) if window else 0
    return pairs, ctx + new - low + min(sink, low)


def work(case):
    ctx, new = _lengths(case)
    B, total = case["batch"], sum(new)
    if case["op"] == "tables":
        after = sum(-(-n // PAGE) for n in new)
        return dict(bytes=4 * (6 * B + 3 * total + 2 * after), flops=0)
    H, D, Hq = case["kv"], case["dim"], case["heads"]
    if case["op"] == "append":
        pages = sum(-(-(c + n) // PAGE) - c // PAGE for c, n in zip(ctx, new))
        meta = pages * H * 2 * D * 2 if case["summaries"] else 0
        return dict(bytes=2 * total * H * D * 2 * 2 + meta + 12 * total, flops=0)
    pairs = keys = 0
    for c, n in zip(ctx, new):
        a, b = _seen(c, n, case["window"], case["sink"])
        pairs, keys = pairs + a, keys + b
    return dict(bytes=keys * H * D * 2 * 2 + total * Hq * (D * (6 if case["fp32"] else 4) + 4),
                flops=4 * D * Hq * pairs)


def exact(case, seed):
    if case["op"] == "tables":
        return None                                          # whole numbers throughout
    s = prepare(case, seed)
    ctx, new = _lengths(case)
    H, D, Hq = case["kv"], case["dim"], case["heads"]
    if case["op"] == "append":
        out = dict(k=s.k.double(), v=s.v.double(), meta=None, ctx_len=None)
        meta = None if s.meta is None else s.meta.double()
        at = 0
        for b, (c, n) in enumerate(zip(ctx, new)):
            bt = s.block_table[b, :-(-(c + n) // PAGE)].long()
            for name, fresh in (("k", s.k_new), ("v", s.v_new)):
                seq = out[name][bt].transpose(0, 1).reshape(H, -1, D)
                seq[:, c:c + n] = fresh[at:at + n].double().transpose(0, 1)
                out[name][bt] = seq.view(H, -1, PAGE, D).transpose(0, 1)
            if meta is not None:
                p0 = c // PAGE
                rows = out["k"][bt[p0:]].clone()
                last = c + n - PAGE * (len(bt) - 1)
                rows[-1, :, last:] = rows[-1, :, :1]
                meta[b, p0:len(bt)] = torch.stack([rows.amin(2), rows.amax(2)], 2)
            at += n
        out["meta"] = meta
        return out
    if 4 * D * Hq * sum(_seen(c, n, 0, 0)[0] for c, n in zip(ctx, new)) > 4e12:
        return None
    out, lse = s.out.double(), s.lse.double()
    G = Hq // H
    at = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        L = c + n
        bt = s.block_table[b, :-(-L // PAGE)].long()
        for h in range(H):
            K = s.k[bt, h].reshape(-1, D)[:L].double()
            V = s.v[bt, h].reshape(-1, D)[:L].double()
            for i0 in range(0, n, 1024):
                i1 = min(n, i0 + 1024)
                p = torch.arange(c + i0, c + i1, device=DEV)[:, None]
                j = torch.arange(L, device=DEV)[None, :]
                hide = j > p
                if case["window"]:
                    hide |= (j <= p - case["window"]) & (j >= case["sink"])
                for g in range(G):
                    x = s.q[at + i0:at + i1, h * G + g].double() @ K.T / math.sqrt(D)
                    x[hide] = -math.inf
                    z = torch.logsumexp(x, 1)
                    out[at + i0:at + i1, h * G + g] = torch.exp(x - z[:, None]) @ V
                    lse[at + i0:at + i1, h * G + g] = z
        at += n
    return dict(out=out, lse=lse)
