// Paging of chunks of new tokens: which pages and rows they get
// (se_chunk_plan), pages taken back (se_pages_release), and the append of the
// rows with their page summaries (se_kv_append_chunk).  Pages of 16 tokens
// with a token->page table follow the paged KV layout of "长程 agent 把显存撑爆以后",
// section "四、为什么进不了 vLLM 一类的引擎".
#include <math_constants.h>

#include <algorithm>

#include "append.cuh"
#include "common.cuh"
#include "internal.h"

namespace se {
namespace {

// Workspace: the status word, then at byte 256 the arrival counter of the
// kernel's blocks (zero between calls).
constexpr int kCounterWord = 64;

// Exclusive block-wide sums of two 64-bit values per thread (lengths come from
// the device and may be anything: 64 bits hold the sum of any 1024 of them).
// `tmp` holds 2 * 33 values.  All threads call it; *ta, *tb receive the totals.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long* tmp,
                                            long long* ta, long long* tb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    long long x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, x, o);
        const long long v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    if (lane == 31) {
        tmp[warp] = x;
        tmp[33 + warp] = y;
    }
    __syncthreads();
    if (warp == 0) {
        long long p = lane < nw ? tmp[lane] : 0, q = lane < nw ? tmp[33 + lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, p, o);
            const long long v = __shfl_up_sync(0xffffffffu, q, o);
            if (lane >= o) {
                p += u;
                q += v;
            }
        }
        if (lane < nw) {
            tmp[lane] = p;
            tmp[33 + lane] = q;
        }
    }
    __syncthreads();
    *ta = tmp[nw - 1];
    *tb = tmp[33 + nw - 1];
    a = x - a + (warp > 0 ? tmp[warp - 1] : 0);
    b = y - b + (warp > 0 ? tmp[33 + warp - 1] : 0);
    __syncthreads();
}

// True in every thread of the last block of the grid to get here; what the
// other blocks read before is then read, and their writes are visible.
__device__ __forceinline__ bool last_block(int* counter) {
    __shared__ int s_last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_last = atomicAdd(counter, 1) == static_cast<int>(gridDim.x) - 1;
    __syncthreads();
    __threadfence();
    return s_last != 0;
}

struct SeqPlan {
    int ctx, held, n;       // tokens and pages held, new tokens (rows in the packed arrays)
    int need;               // pages it takes when it is served (counted for those behind it)
    int flags;              // SE_DEV_* bits
    bool ok;                // lengths consistent
};

__device__ __forceinline__ SeqPlan seq_plan(const se_page_pool& p, const int32_t* new_len, int b) {
    SeqPlan s;
    s.ctx = p.ctx_len[b];
    s.held = p.n_pages[b];
    const int n = new_len[b];
    s.n = max(n, 0);
    s.flags = 0;
    s.need = 0;
    const long long cap = static_cast<long long>(p.max_pages_per_seq) * kPage;
    s.ok = n >= 0 && s.ctx >= 0 && s.ctx <= cap && s.held >= (s.ctx + kPage - 1) / kPage &&
           s.held <= p.max_pages_per_seq;
    if (!s.ok) {
        s.flags = SE_DEV_BAD_LENGTH;
    } else if (static_cast<long long>(s.ctx) + s.n > cap) {
        s.ok = false;
        s.flags = SE_DEV_CAPACITY;
    } else {
        const int pages = static_cast<int>((static_cast<long long>(s.ctx) + s.n + kPage - 1) / kPage);
        s.need = max(0, pages - s.held);
    }
    return s;
}

// One launch for the whole plan.  Every block scans all sequences (a few
// words each, from L2) and writes its own range of the packed rows: a row's
// page comes straight from the free stack or from the part of the block table that
// was there before, so no block waits for another.  What the scan read
// (n_pages, n_free) is updated by the last block to finish, which scans again.
// Latency bound: the bytes (12 per row, 4 per new page, 12 per sequence) take
// less time than the launch up to some hundred thousand rows.
__global__ void __launch_bounds__(1024)
    chunk_plan_kernel(se_page_pool pool, const int32_t* new_len, int batch, se_chunk ck,
                      int rows_per_block, int* ws) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) int smem[];
    const int nt = blockDim.x;
    int* s_start = smem;            // [nt + 1] first row of each sequence of the pass
    int* s_ctx = s_start + nt + 1;
    int* s_held = s_ctx + nt;
    int* s_top = s_held + nt;       // stack index of the sequence's first new page; -1: not served
    __shared__ long long tmp[66];
    int* status = ws;
    const long long max_rows = ck.max_tokens;
    const int r0 = min(blockIdx.x * rows_per_block, ck.max_tokens);
    const int r1 = min(r0 + rows_per_block, ck.max_tokens);
    int n_free = *pool.n_free;
    int bad_flags = 0;
    if (n_free < 0 || n_free > pool.num_pages) {
        bad_flags |= SE_DEV_BAD_LENGTH;
        n_free = n_free < 0 ? 0 : pool.num_pages;
    }
    // in one pass (batch <= nt): what this thread's sequence holds afterwards (-1: as
    // before), and the pages taken by all
    int holds = -1;
    __shared__ int s_taken;
    if (threadIdx.x == 0) s_taken = 0;
    long long row_base = 0, need_base = 0;
    for (int b0 = 0; b0 < batch; b0 += nt) {
        const int b = b0 + threadIdx.x;
        SeqPlan s = {};
        if (b < batch) s = seq_plan(pool, new_len, b);
        long long row = s.n, need = s.need, rows = 0, needs = 0;
        block_scan2(row, need, tmp, &rows, &needs);
        row += row_base;
        // a sequence whose rows pass max_tokens takes no page, and those behind
        // it neither (their rows pass it too); their needs stay out of the count,
        // which only they would have read
        bool ok = s.ok;
        if (ok && row + s.n > max_rows) {
            ok = false;
            s.flags |= SE_DEV_CAPACITY;
        }
        need += need_base;
        if (ok && s.need > 0 && need + s.need > n_free) {
            ok = false;
            s.flags |= SE_DEV_CAPACITY;
        }
        // pages go out in sequence order, so the last served sequence's end is the sum
        if (batch <= nt && ok && s.need > 0) {
            holds = s.held + s.need;
            atomicMax(&s_taken, static_cast<int>(need + s.need));
        }
        s_start[threadIdx.x] = static_cast<int>(min(row, max_rows));
        s_ctx[threadIdx.x] = s.ctx;
        s_held[threadIdx.x] = s.held;
        s_top[threadIdx.x] = ok ? static_cast<int>(max(0ll, n_free - 1 - need)) : -1;
        const int c_end = static_cast<int>(min(row_base + rows, max_rows));
        if (threadIdx.x == 0) s_start[nt] = c_end;
        if (blockIdx.x == 0 && b < batch) {
            if (b == 0) ck.start[0] = 0;
            ck.start[b + 1] = static_cast<int>(min(row + s.n, max_rows));
            bad_flags |= s.flags;
        }
        __syncthreads();
        const int lo = max(r0, static_cast<int>(min(row_base, max_rows)));
        const int hi = min(r1, c_end);
        // four rows a thread at once: their searches and loads overlap
        for (int t0 = lo + threadIdx.x; t0 < hi; t0 += 4 * nt) {
            int at[4], pos[4], phys[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) at[k] = 0;
            // the last sequence of the pass that starts at or before row t
            for (int step = nt >> 1; step > 0; step >>= 1)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (s_start[at[k] + step] <= t0 + k * nt) at[k] += step;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = t0 + k * nt, i = at[k];
                pos[k] = phys[k] = -1;
                if (t < hi && s_top[i] >= 0) {
                    pos[k] = s_ctx[i] + (t - s_start[i]);
                    const int fresh = pos[k] / kPage - s_held[i];
                    phys[k] = fresh < 0 ? pool.block_table[(int64_t)(b0 + i) * pool.max_pages_per_seq +
                                                           pos[k] / kPage]
                                        : pool.free_pages[s_top[i] - fresh];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = t0 + k * nt, i = at[k];
                if (t >= hi) break;
                if (pos[k] >= 0) {
                    if (phys[k] < 0 || phys[k] >= pool.num_pages) {
                        bad_flags |= SE_DEV_BAD_INDEX;
                        phys[k] = -1;
                    }
                    const int pg = pos[k] / kPage;
                    if (pg >= s_held[i] && pos[k] % kPage == 0)
                        pool.block_table[(int64_t)(b0 + i) * pool.max_pages_per_seq + pg] = phys[k];
                }
                ck.seq[t] = b0 + i;
                ck.pos[t] = pos[k];
                ck.slot[t] = phys[k] >= 0 ? phys[k] * kPage + pos[k] % kPage : -1;
            }
        }
        row_base += rows;
        need_base += needs;
        __syncthreads();
    }
    const int live = static_cast<int>(min(row_base, max_rows));
    if (blockIdx.x == 0 && batch == 0 && threadIdx.x == 0) ck.start[0] = 0;
    for (int t = max(r0, live) + threadIdx.x; t < r1; t += nt) {
        ck.seq[t] = -1;
        ck.pos[t] = -1;
        ck.slot[t] = -1;
    }
    if (bad_flags) flag(status, bad_flags);
    if (gridDim.x > 1 && !last_block(ws + kCounterWord)) return;
    if (batch <= nt) {
        // every block knows what each sequence takes
        if (holds >= 0) pool.n_pages[threadIdx.x] = holds;
        if (threadIdx.x == 0) {
            *pool.n_free = n_free - s_taken;
            ws[kCounterWord] = 0;
        }
        return;
    }
    __syncthreads();                             // (one block: its reads of n_pages are done)
    // the same scan again, now storing what each served sequence holds
    long long taken = 0;
    row_base = need_base = 0;
    for (int b0 = 0; b0 < batch; b0 += nt) {
        const int b = b0 + threadIdx.x;
        SeqPlan s = {};
        if (b < batch) s = seq_plan(pool, new_len, b);
        long long row = s.n, need = s.need, rows = 0, needs = 0;
        block_scan2(row, need, tmp, &rows, &needs);
        const bool ok = s.ok && row_base + row + s.n <= max_rows && s.need > 0 &&
                        need_base + need + s.need <= n_free;
        if (ok) pool.n_pages[b] = s.held + s.need;
        long long got = ok ? s.need : 0, none = 0, gots = 0, nones = 0;
        block_scan2(got, none, tmp, &gots, &nones);
        taken += gots;
        row_base += rows;
        need_base += needs;
    }
    if (threadIdx.x == 0) {
        *pool.n_free = n_free - static_cast<int>(taken);
        ws[kCounterWord] = 0;
    }
}

// Pages of the flagged sequences back onto the stack: i-th released page (in
// sequence order) to the i-th place below the new top.  Every block scans all
// sequences and copies its share of the pages; the last block to finish
// clears the lengths and moves the top.
__global__ void __launch_bounds__(1024)
    pages_release_kernel(se_page_pool pool, const int32_t* done, int batch, int* ws) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) int smem[];
    const int nt = blockDim.x;
    long long* s_first = reinterpret_cast<long long*>(smem);    // [nt + 1]
    __shared__ long long tmp[66];
    int* status = ws;
    int bad_flags = 0;
    int n_free = *pool.n_free;
    if (n_free < 0 || n_free > pool.num_pages) {
        bad_flags |= SE_DEV_BAD_LENGTH;
        n_free = n_free < 0 ? 0 : pool.num_pages;
    }
    auto held_of = [&](int b) -> long long {
        if (b >= batch || done[b] == 0) return 0;
        const int n = pool.n_pages[b];
        if (n < 0 || n > pool.max_pages_per_seq) {
            bad_flags |= SE_DEV_BAD_LENGTH;
            return n < 0 ? 0 : pool.max_pages_per_seq;
        }
        return n;
    };
    long long total = 0, mine = 0;             // mine: in one pass, pages before this sequence's
    for (int b0 = 0; b0 < batch; b0 += nt) {
        long long none = 0, sum = 0, nones = 0;
        mine = held_of(b0 + threadIdx.x);
        block_scan2(mine, none, tmp, &sum, &nones);
        total += sum;
    }
    const bool fits = n_free + total <= pool.num_pages;
    if (!fits) bad_flags |= SE_DEV_CAPACITY;
    long long base = 0;
    for (int b0 = 0; fits && b0 < batch; b0 += nt) {
        long long first = mine, none = 0, sum = total, nones = 0;
        if (batch > nt) {
            first = held_of(b0 + threadIdx.x);
            block_scan2(first, none, tmp, &sum, &nones);
        }
        s_first[threadIdx.x] = first;
        if (threadIdx.x == 0) s_first[nt] = sum;
        __syncthreads();
        for (long long i = (long long)blockIdx.x * nt + threadIdx.x; i < sum;
             i += (long long)gridDim.x * nt) {
            int k = 0;
            for (int step = nt >> 1; step > 0; step >>= 1)
                if (s_first[k + step] <= i) k += step;
            const int pg = static_cast<int>(i - s_first[k]);
            pool.free_pages[n_free + total - 1 - (base + i)] =
                pool.block_table[(int64_t)(b0 + k) * pool.max_pages_per_seq + pg];
        }
        base += sum;
        __syncthreads();
    }
    if (bad_flags) flag(status, bad_flags);
    if (gridDim.x > 1 && !last_block(ws + kCounterWord)) return;
    __syncthreads();                             // (one block: its reads of n_pages are done)
    if (fits) {
        for (int b = threadIdx.x; b < batch; b += nt) {
            if (done[b] == 0) continue;
            pool.n_pages[b] = 0;
            pool.ctx_len[b] = 0;
        }
        if (threadIdx.x == 0) *pool.n_free = n_free + static_cast<int>(total);
    }
    if (threadIdx.x == 0) ws[kCounterWord] = 0;
}

// Row t of a chunk: slot is -1 where it has none, where it is dropped (`bad`: the slot
// is outside the pages, or seq or pos outside the block table) and past the arrays.
struct ChunkRow {
    int slot, pos, seq;
    bool bad;
};
__device__ __forceinline__ ChunkRow chunk_row(const se_paged_kv& kv, const se_chunk& ck, int batch,
                                              int t) {
    ChunkRow r = {-1, -1, -1, false};
    if (t < 0 || t >= ck.max_tokens) return r;
    r.slot = ck.slot[t];
    r.pos = ck.pos[t];
    r.seq = ck.seq[t];
    r.bad = r.slot != -1 &&
            (r.slot < 0 || r.slot / kPage >= kv.num_pages || r.seq < 0 || r.seq >= batch ||
             r.pos < 0 || r.pos / kPage >= kv.max_pages_per_seq ||
             r.pos % kPage != r.slot % kPage);
    if (r.bad) {
        r.slot = -1;
        if (r.seq == -1) r.seq = -2;                // names none, but is no row past the last sequence
    }
    return r;
}

// Lengths: each sequence's last row with a slot sets ctx_len, and no other row writes it.
// Lane l holds row t of 32; lanes 1..16 hold the rows this warp answers for.  The row after
// such a row tells, unless that one has no slot (a page that was not found, a dropped
// row): then the warp looks on, past rows without a slot that are the same sequence's or
// name none that exists, 32 at a time, to the next row that decides.
__device__ __forceinline__ void commit_lengths(const se_paged_kv& kv, const se_chunk& ck, int batch,
                                               int t, int lane, const ChunkRow& row) {
    const bool mine = row.slot >= 0 && lane >= 1 && lane <= kPage;
    const int nslot = __shfl_down_sync(0xffffffffu, row.slot, 1);
    const int nseq = __shfl_down_sync(0xffffffffu, row.seq, 1);
    auto passes = [&](int s, int b) { return s == b || s < -1 || s >= batch; };
    const bool hole = mine && nslot < 0 && passes(nseq, row.seq);
    if (mine && !hole && (nslot < 0 || nseq != row.seq)) kv.ctx_len[row.seq] = row.pos + 1;
    for (uint32_t m = __ballot_sync(0xffffffffu, hole); m != 0; m &= m - 1) {
        const int f = __ffs(m) - 1;
        const int b = __shfl_sync(0xffffffffu, row.seq, f);
        const int len = __shfl_sync(0xffffffffu, row.pos, f) + 1;
        uint32_t more, end;                         // rows that go on, rows that are another's or none's
        for (int r = __shfl_sync(0xffffffffu, t, f) + 1;; r += 32) {
            const ChunkRow x = chunk_row(kv, ck, batch, r + lane);
            more = __ballot_sync(0xffffffffu, x.slot >= 0 && x.seq == b);
            end = __ballot_sync(0xffffffffu,
                                x.slot >= 0 ? x.seq != b : !passes(x.seq, b));
            if ((more | end) != 0) break;           // (rows past max_tokens end it)
        }
        if (lane == 0 && __ffs(more | end) == __ffs(end)) kv.ctx_len[b] = len;
    }
}

// Append of packed rows.  Block i looks at rows [16i, 16i + 16); the rows of one sequence that
// lie in one page are a piece (at most 16 rows apart, whatever rows between them have no
// slot), the work of one warp for one KV head, which owns that page's summary: no
// atomics and a fixed result.  Each warp finds the pieces that begin in the block
// from the slots of 32 rows around it (ballots).  A row is D/8 16-byte vectors, so
// RP rows move side by side; all loads of a piece are in flight before the
// first store.  HBM bound for long chunks (each byte read once and written once),
// latency bound for a few rows.
template <int D>
__global__ void __launch_bounds__(128)
    kv_append_chunk_kernel(se_paged_kv kv, const uint4* k_new, const uint4* v_new,
                           int64_t row_stride, se_chunk ck, int batch, int* status) {
    constexpr int SEGS = D / 8, RP = 32 / SEGS, IT = kPage / RP;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int H = kv.num_kv_heads;
    // lane l looks at row 16i - 1 + l
    const int t = static_cast<int>(blockIdx.x) * kPage - 1 + lane;
    const ChunkRow row = chunk_row(kv, ck, batch, t);
    if (row.bad && lane >= 1 && lane <= kPage && warp == 0) flag(status, SE_DEV_BAD_INDEX);
    const int slot = row.slot, pos = row.pos, seq = row.seq;
    const bool valid = slot >= 0;
    const int pslot = __shfl_up_sync(0xffffffffu, slot, 1);
    const int pseq = __shfl_up_sync(0xffffffffu, seq, 1);
    const int ppos = __shfl_up_sync(0xffffffffu, pos, 1);
    const bool begins = valid && lane >= 1 && lane <= kPage &&
                        !(pslot >= 0 && pseq == seq && ppos + 1 == pos && pslot + 1 == slot &&
                          pos % kPage != 0);
    // rows of a piece: slot and position go with the row
    auto same_piece = [&](int d, int slot_d, int pos_d, int seq_d, int slot0, int pos0, int seq0) {
        return slot_d >= 0 && seq_d == seq0 && slot_d - slot0 == d && pos_d - pos0 == d &&
               pos_d / kPage == pos0 / kPage;
    };
    uint32_t lead_m = __ballot_sync(0xffffffffu, begins);
    // behind rows without a slot a page may have begun before them: up to 15 rows back
    const bool unsure = begins && pslot < 0 && t > 0 && pos % kPage != 0 &&
                        (pseq == seq || pseq < 0 || pseq >= batch);
    uint32_t look = __ballot_sync(0xffffffffu, unsure);
    if (look != 0) {
        const ChunkRow far = chunk_row(kv, ck, batch, t - 32);
        for (; look != 0; look &= look - 1) {
            const int f = __ffs(look) - 1;
            const int slot0 = __shfl_sync(0xffffffffu, slot, f);
            const int pos0 = __shfl_sync(0xffffffffu, pos, f);
            const int seq0 = __shfl_sync(0xffffffffu, seq, f);
            if (__any_sync(0xffffffffu,
                           (lane < f && same_piece(lane - f, slot, pos, seq, slot0, pos0, seq0)) ||
                               same_piece(lane - 32 - f, far.slot, far.pos, far.seq, slot0, pos0,
                                          seq0)))
                lead_m &= ~(1u << f);
        }
    }
    if (warp == 0 && blockIdx.y == 0) commit_lengths(kv, ck, batch, t, lane, row);
    const int seg = lane % SEGS, rp = lane / SEGS;
    uint4* K = static_cast<uint4*>(kv.k);
    uint4* V = static_cast<uint4*>(kv.v);
    uint4* M = static_cast<uint4*>(kv.meta);
    const int units = __popc(lead_m) * H;
    const int nw = (blockDim.x >> 5) * gridDim.y;
    for (int u = warp + (blockDim.x >> 5) * blockIdx.y; u < units; u += nw) {
        const int h = u % H;
        uint32_t rest = lead_m;
        for (int i = u / H; i > 0; --i) rest &= rest - 1;
        const int f = __ffs(rest) - 1;                              // lane of the piece's first row
        const int slot0 = __shfl_sync(0xffffffffu, slot, f);
        const int pos0 = __shfl_sync(0xffffffffu, pos, f);
        const int seq0 = __shfl_sync(0xffffffffu, seq, f);
        // bit r: row r behind the first is of the piece
        const uint32_t rows =
            __ballot_sync(0xffffffffu, same_piece(lane - f, slot, pos, seq, slot0, pos0, seq0)) >> f;
        const int64_t src = (int64_t)(static_cast<int>(blockIdx.x) * kPage - 1 + f) * row_stride +
                            h * SEGS + seg;
        uint4 k[IT], v[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = i * RP + rp;
            if ((rows >> r) & 1) {
                k[i] = k_new[src + r * row_stride];
                v[i] = v_new[src + r * row_stride];
            }
        }
        const int64_t m0 =
            ((((int64_t)seq0 * kv.max_pages_per_seq + pos0 / kPage) * H + h) * 2) * SEGS + seg;
        const bool fold = pos0 % kPage != 0;
        uint4 old_mn = make_uint4(0, 0, 0, 0), old_mx = old_mn;
        if (M != nullptr && fold && rp == 0) {
            old_mn = M[m0];
            old_mx = M[m0 + SEGS];
        }
        const int64_t dst =
            (((int64_t)(slot0 / kPage) * H + h) * kPage + slot0 % kPage) * SEGS + seg;
        Bf8 mn, mx;
#pragma unroll
        for (int e = 0; e < 8; ++e)              // none yet: min and max pass a NaN over
            mn.x[e] = mx.x[e] = CUDART_NAN_F;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = i * RP + rp;
            if ((rows >> r) & 1) {
                K[dst + r * SEGS] = k[i];
                V[dst + r * SEGS] = v[i];
                const Bf8 x = unpack8(k[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    mn.x[e] = fminf(mn.x[e], x.x[e]);
                    mx.x[e] = fmaxf(mx.x[e], x.x[e]);
                }
            }
        }
        if (M == nullptr) continue;
#pragma unroll
        for (int o = SEGS; o < 32; o <<= 1)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                mn.x[e] = fminf(mn.x[e], __shfl_xor_sync(0xffffffffu, mn.x[e], o));
                mx.x[e] = fmaxf(mx.x[e], __shfl_xor_sync(0xffffffffu, mx.x[e], o));
            }
        if (rp == 0) {
            if (fold) {
                const Bf8 a = unpack8(old_mn), c = unpack8(old_mx);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    mn.x[e] = fminf(a.x[e], mn.x[e]);
                    mx.x[e] = fmaxf(c.x[e], mx.x[e]);
                }
            }
            M[m0] = pack8(mn);
            M[m0 + SEGS] = pack8(mx);
        }
    }
}

}  // namespace

// A thread per sequence, up to 1024 of them in one pass.
static int scan_threads(int batch) { return batch > 512 ? 1024 : batch > 256 ? 512 : 256; }

size_t page_pool_ws_bytes() { return 512; }

cudaError_t launch_chunk_plan(const se_page_pool& pool, const int32_t* new_len, int batch,
                              const se_chunk& ck, int* ws, cudaStream_t s) {
    const int nt = scan_threads(batch);
    const int grid = max(1, min(num_sms(), (ck.max_tokens + 2 * nt - 1) / (2 * nt)));
    const int per = (ck.max_tokens + grid - 1) / grid;
    return launch_pdl(chunk_plan_kernel, dim3(grid), dim3(nt), (4 * nt + 1) * sizeof(int), s, pool,
                      new_len, batch, ck, per, ws);
}

cudaError_t launch_pages_release(const se_page_pool& pool, const int32_t* done, int batch, int* ws,
                                 cudaStream_t s) {
    const int nt = scan_threads(batch);
    // a block for every 4096 table entries that could be released
    const int64_t most = std::min<int64_t>((int64_t)batch * pool.max_pages_per_seq, pool.num_pages);
    const int grid =
        static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(num_sms(), most / 4096)));
    return launch_pdl(pages_release_kernel, dim3(grid), dim3(nt), (nt + 1) * sizeof(long long), s,
                      pool, done, batch, ws);
}

cudaError_t launch_kv_append_chunk(const se_paged_kv& kv, const void* k_new, const void* v_new,
                                   int64_t row_stride, const se_chunk& ck, int batch, int* status,
                                   cudaStream_t s) {
    const int blocks = (ck.max_tokens + kPage - 1) / kPage;
    if (blocks == 0) return cudaSuccess;
    // few rows: more blocks share one group of 16, down to one piece a warp
    // (16 pieces x the heads, four warps a block)
    const int share = std::max(1, std::min(4 * num_sms() / blocks, 4 * kv.num_kv_heads));
    const dim3 grid(blocks, share);
    const uint4* k = static_cast<const uint4*>(k_new);
    const uint4* v = static_cast<const uint4*>(v_new);
    if (kv.head_dim == 128)
        return launch_pdl(kv_append_chunk_kernel<128>, grid, dim3(128), 0, s, kv, k, v,
                          row_stride / 8, ck, batch, status);
    return launch_pdl(kv_append_chunk_kernel<64>, grid, dim3(128), 0, s, kv, k, v, row_stride / 8,
                      ck, batch, status);
}

}  // namespace se
