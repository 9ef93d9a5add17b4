// Sequences that share pages: forks (se_pages_fork), lengths cut back with the pages that nobody
// holds any more going back on the stack (se_pages_truncate), and what each layer's cache takes
// over (se_pages_carry).  Pages of 16 tokens with a token->page table follow the paged KV
// layout of "长程 agent 把显存撑爆以后", section "四、为什么进不了 vLLM 一类的引擎".
//
// One rule keeps every append away from shared pages: a sequence's last, partly filled page is its
// own.  Full pages may be shared (page_refs counts the holders beside the first); a fork takes a
// page for the part that is not full, and so does a cut that ends inside a shared page.
#include <math_constants.h>

#include <algorithm>
#include <atomic>

#include "append.cuh"
#include "common.cuh"
#include "internal.h"
#include "page_tables.cuh"

namespace se {
namespace {

constexpr int kMaxBatch = 8192;              // sequences whose entries shared memory numbers
constexpr int kWhoWord = 128;                // a workspace word for each page from here on, zero
                                             // between calls (se_pages_truncate)

__device__ __forceinline__ int clamped_free(const se_page_pool& pool, int& flags) {
    const int n = *pool.n_free;
    if (n >= 0 && n <= pool.num_pages) return n;
    flags |= SE_DEV_BAD_LENGTH;
    return n < 0 ? 0 : pool.num_pages;
}
__device__ __forceinline__ bool in_pool(const se_page_pool& pool, int page) {
    return page >= 0 && page < pool.num_pages;
}
// Whether ctx tokens in `held` pages make sense.
__device__ __forceinline__ bool consistent(const se_page_pool& pool, int ctx, int held) {
    return ctx >= 0 && held >= 0 && held <= pool.max_pages_per_seq &&
           ctx <= (long long)pool.max_pages_per_seq * kPage && held >= (ctx + kPage - 1) / kPage;
}
// The sequence whose entries (numbered over all sequences, first[] its running sum) hold entry i.
__device__ __forceinline__ int owner_of(const int* first, int batch, int i) {
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// ---- fork ---------------------------------------------------------------------------------
struct Fork {
    int src, ctx, flags;
    bool want, page;             // to be forked; needs a page of its own
};
__device__ __forceinline__ Fork fork_of(const se_page_pool& p, const int32_t* src, int batch,
                                        int b) {
    Fork f = {src[b], 0, 0, false, false};
    if (f.src < 0) return f;
    if (f.src >= batch) {
        f.flags = SE_DEV_BAD_INDEX;
        return f;
    }
    const int its_own = src[f.src], mine = p.n_pages[b], theirs = p.n_pages[f.src];
    f.ctx = p.ctx_len[f.src];                                // (one latency for the four)
    if (its_own >= 0) {
        f.flags = SE_DEV_BAD_INDEX;
    } else if (mine != 0 || !consistent(p, f.ctx, theirs)) {
        f.flags = SE_DEV_BAD_LENGTH;
    } else if (f.ctx % kPage != 0 &&                         // (it asks for no page that it cannot use)
               !in_pool(p, p.block_table[(int64_t)f.src * p.max_pages_per_seq + f.ctx / kPage])) {
        f.flags = SE_DEV_BAD_INDEX;
    } else {
        f.want = true;
        f.page = f.ctx % kPage != 0;
    }
    return f;
}

// Every block scans all sequences (a thread a run of them) and writes its share of the
// table entries; the last block to finish, which has read what the others have, commits
// counts and lengths.  Latency bound: four samples of a 2K prompt about 4 us, 64 of a 32K one
// (131,008 table entries, each with an atomic count) 9.
__global__ void __launch_bounds__(1024, 1)
    pages_fork_kernel(se_page_pool pool, int32_t* refs, const int32_t* src, int batch,
                      se_page_carry carry, int* ws) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) int smem[];
    int* s_first = smem;                     // [batch] first of the sequence's entries
    int* s_fresh = smem + batch;             // [batch] its own page; -1: needs none; -2: not served
    __shared__ long long tmp[66];
    int flags = 0;
    const int n_free = clamped_free(pool, flags);
    // this thread's sequences [b0, b1)
    const int per = (batch + blockDim.x - 1) / blockDim.x;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, batch), b1 = min(b0 + per, batch);
    Fork mine = {-1, 0, 0, false, false};
    if (b0 < b1) mine = fork_of(pool, src, batch, b0);
    long long asked = 0, entries = 0, asks, all;
    for (int b = b0; b < b1; ++b) {
        const Fork f = b == b0 ? mine : fork_of(pool, src, batch, b);
        asked += f.page;
        entries += f.want ? f.ctx / kPage : 0;
    }
    block_scan2(asked, entries, tmp, &asks, &all);
    long long run = asked, at = entries;
    bool less = false;                       // one is not served: fewer entries before the next
    for (int b = b0; b < b1; ++b) {
        const Fork f = b == b0 ? mine : fork_of(pool, src, batch, b);
        flags |= f.flags;
        int fresh = f.want ? -1 : -2;
        if (f.page) {
            ++run;
            if (run > n_free) {
                flags |= SE_DEV_CAPACITY;
                fresh = -2;
            } else {
                fresh = pool.free_pages[n_free - run];
                if (!in_pool(pool, fresh)) {
                    flags |= SE_DEV_BAD_INDEX;
                    fresh = -2;
                }
            }
            less |= fresh == -2;
        }
        s_fresh[b] = fresh;
        s_first[b] = static_cast<int>(at);
        at += f.want ? f.ctx / kPage : 0;
    }
    if (__syncthreads_or(less)) {
        long long n = 0, none = 0, nones;
        for (int b = b0; b < b1; ++b) n += s_fresh[b] == -2 ? 0 : pool.ctx_len[src[b]] / kPage;
        block_scan2(n, none, tmp, &all, &nones);
        for (int b = b0; b < b1; ++b) {
            s_first[b] = static_cast<int>(n);
            n += s_fresh[b] == -2 ? 0 : pool.ctx_len[src[b]] / kPage;
        }
    }
    __syncthreads();
    // table entries (a block table of these calls has at most 2^30)
    const int total = static_cast<int>(all);
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (long long)gridDim.x * blockDim.x) {
        const int b = owner_of(s_first, batch, static_cast<int>(i));
        const int64_t p = i - s_first[b];
        const int page = pool.block_table[(int64_t)src[b] * pool.max_pages_per_seq + p];
        pool.block_table[(int64_t)b * pool.max_pages_per_seq + p] = page;
        if (in_pool(pool, page))
            atomicAdd(refs + page, 1);
        else
            flags |= SE_DEV_BAD_INDEX;
    }
    if (flags) flag(ws, flags);
    if (gridDim.x > 1 && !last_block(ws + kCounterWord)) return;
    __syncthreads();
    // (each thread its own sequences: sources are no forks, so nothing read here is written)
    for (int b = threadIdx.x; b < batch; b += blockDim.x) {
        const int fresh = s_fresh[b];
        int from_seq = -1, from_page = -1;
        if (fresh != -2) {
            from_seq = src[b];
            const int ctx = pool.ctx_len[from_seq];
            if (fresh >= 0) {
                const int64_t maxp = pool.max_pages_per_seq;
                from_page = pool.block_table[from_seq * maxp + ctx / kPage];
                pool.block_table[b * maxp + ctx / kPage] = fresh;
            }
            pool.ctx_len[b] = ctx;
            pool.n_pages[b] = (ctx + kPage - 1) / kPage;
        }
        carry.from_seq[b] = from_seq;
        carry.from_page[b] = from_page;
    }
    if (threadIdx.x == 0) {
        *pool.n_free = n_free - static_cast<int>(min(asks, (long long)n_free));
        ws[kCounterWord] = 0;
    }
}

// ---- truncation ---------------------------------------------------------------------------
struct Cut {
    int n, ctx, held, after;     // tokens and pages it is cut to
    int last, flags;             // the page that is then its last
    bool act, copy;              // cut at all; needs a page of its own for the last one's rows
};
__device__ __forceinline__ Cut cut_of(const se_page_pool& p, const int32_t* refs,
                                      const int32_t* keep, int b) {
    Cut c = {keep[b], p.ctx_len[b], p.n_pages[b], 0, -1, 0, false, false};
    if (c.n < 0) return c;
    if (!consistent(p, c.ctx, c.held)) {
        c.flags = SE_DEV_BAD_LENGTH;
        return c;
    }
    c.n = min(c.n, c.ctx);
    c.after = (c.n + kPage - 1) / kPage;
    if (c.n % kPage != 0) {
        c.last = p.block_table[(int64_t)b * p.max_pages_per_seq + c.after - 1];
        if (!in_pool(p, c.last)) {
            c.flags = SE_DEV_BAD_INDEX;
            return c;
        }
        c.copy = refs != nullptr && refs[c.last] > 0;
    }
    c.act = true;
    return c;
}

// One cluster of blocks, whose hardware barrier divides the phases; every block scans all
// sequences itself, then takes a contiguous part of the entries (a page that a sequence lets go,
// in the order of sequence and logical page).
//   count down  each entry takes one off its page's count and notes its sequence as the
//               page's last, if it is that
//   count       an entry is freed when its page's count fell below zero and it is the last:
//               which entry that is depends on no timing
//   push        freed entries to their place by a running sum, counts and notes back to zero
//   commit      tables, lengths, the stack's top
// Few entries (a decode step's: a page here and there) are the first block's alone; then the
// others leave after the scan.
// Latency bound: nothing let go 4 us, a decode step's pages 7 to 11, 64 samples of a 32K prompt
// (131,008 entries, all of shared pages) about 24: random counts from 16 SMs.  With cold
// caches: on one block 1694 us, on eight 82, on sixteen, with the entries that the next
// sequence follows uncounted, 36, each thread's entries fetched once 28.  A launch over all
// SMs would need a barrier across them for each phase.  1024 threads have 64 registers each: 28
// bytes are spilled.
constexpr int kEntries = 8;                  // of a thread at once, at most
constexpr int kAsks = -3;                    // asks for a page of its own

__global__ void __launch_bounds__(1024, 1)
    pages_truncate_kernel(se_page_pool pool, int32_t* refs, const int32_t* keep, int batch,
                          se_page_carry carry, int* ws) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) int smem[];
    int* s_first = smem;                     // [batch] first of the sequence's entries
    int* s_base = smem + batch;              // [batch] logical page of its first entry
    int* s_fresh = smem + 2 * batch;         // [batch] page for the last rows; -1: none; -2: not cut
    __shared__ long long tmp[66];
    __shared__ int s_count, s_scan[33];
    int* who = ws + kWhoWord;
    const int nt = blockDim.x;
    int rank = cluster_rank(), ranks = cluster_size(), flags = 0;
    const int n_free = clamped_free(pool, flags);
    // this thread's sequences [b0, b1)
    const int per = (batch + nt - 1) / nt;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, batch), b1 = min(b0 + per, batch);
    Cut mine = {-1, 0, 0, 0, -1, 0, false, false};           // (the first of them)
    long long asked = 0, entries = 0, asks, all;
    for (int b = b0; b < b1; ++b) {
        const Cut c = cut_of(pool, refs, keep, b);
        if (b == b0) mine = c;
        flags |= c.flags;
        s_fresh[b] = !c.act ? -2 : c.copy ? kAsks : -1;
        s_base[b] = c.after - c.copy;
        s_first[b] = c.act ? c.held - s_base[b] : 0;         // (their count, so far)
        asked += c.copy;
        entries += s_first[b];
    }
    block_scan2(asked, entries, tmp, &asks, &all);
    bool less = false;                       // one is not served: fewer entries before the next
    for (int b = b0; b < b1; ++b) {
        if (s_fresh[b] == kAsks) {
            ++asked;
            int fresh = -2;
            if (asked > n_free) {
                flags |= SE_DEV_CAPACITY;
            } else {
                fresh = pool.free_pages[n_free - asked];
                if (!in_pool(pool, fresh)) {
                    flags |= SE_DEV_BAD_INDEX;
                    fresh = -2;
                }
            }
            s_fresh[b] = fresh;
            less |= fresh == -2;
        }
        const int n = s_first[b];
        s_first[b] = static_cast<int>(entries);
        entries += n;
    }
    if (__syncthreads_or(less)) {
        auto lets = [&](int b) { return s_fresh[b] == -2 ? 0 : pool.n_pages[b] - s_base[b]; };
        long long n = 0, none = 0, nones;
        for (int b = b0; b < b1; ++b) n += lets(b);
        block_scan2(n, none, tmp, &all, &nones);
        for (int b = b0; b < b1; ++b) {
            s_first[b] = static_cast<int>(n);
            n += lets(b);
        }
    }
    const int taken = static_cast<int>(min(asks, (long long)n_free));
    const int total = static_cast<int>(all);
    if (ranks > 1)
        cluster_sync();                      // all have read what was there before the call
    else
        __syncthreads();
    const bool wide = ranks > 1 && total > nt * kEntries;
    if (!wide) {
        if (rank != 0) return;
        ranks = 1;
    }
    auto all_sync = [&]() {
        if (wide)
            cluster_sync();
        else
            __syncthreads();
    };
    // this block's entries [e0, e1), `each` of a thread side by side (few: one)
    const int e0 = static_cast<int>((long long)total * rank / ranks);
    const int e1 = static_cast<int>((long long)total * (rank + 1) / ranks);
    const int each = min(kEntries, max(1, (e1 - e0 + nt - 1) / nt)), step = nt * each;
    const bool once = e1 - e0 <= step;       // they stay in registers
    auto first_of = [&](int b) { return b < batch ? s_first[b] : total; };
    int page[kEntries], seq[kEntries];
    uint32_t open = 0;                       // bit r: entry r may be its page's last of this call
    uint32_t freed_bits = 0, last_bits = 0;  // of the first steps: found once
    bool have = false, shared = refs != nullptr, fits = true;
    int before = 0, all_freed = 0, place = 0, top = 0, count = 0;
    // probe: does any entry's page have other holders (as most have not: nothing to count)?
    enum { kProbe, kCountDown, kCount, kPush, kEnd };
    int phase = total == 0 ? kEnd : !shared ? kCount : once && !wide ? kProbe : kCountDown;
    while (phase != kEnd) {
        bool any = false;
        int k = 0;
        for (int base = e0; base < e1; base += step, ++k) {
            if (!have || !once) {
                have = true;
                open = 0;
                const int i0 = base + threadIdx.x * each;
                int b = owner_of(s_first, batch, min(i0, e1 - 1)), next[kEntries];
#pragma unroll
                for (int r = 0; r < kEntries; ++r) {
                    page[r] = next[r] = -1;
                    seq[r] = 0;
                    if (r < each && i0 + r < e1) {
                        while (b + 1 < batch && s_first[b + 1] <= i0 + r) ++b;
                        const int at = s_base[b] + (i0 + r - s_first[b]);
                        const int32_t* table =
                            pool.block_table + (int64_t)b * pool.max_pages_per_seq + at;
                        seq[r] = b;
                        page[r] = table[0];
                        // samples of one prompt lie side by side: where the next sequence lets
                        // go of the same page, this entry is not the last, and asks no counter
                        const int j = at - s_base[min(b + 1, batch - 1)];
                        const int n = b + 1 < batch ? first_of(b + 2) - s_first[b + 1] : 0;
                        if (shared && j >= 0 && j < n) next[r] = table[pool.max_pages_per_seq];
                    }
                }
#pragma unroll
                for (int r = 0; r < kEntries; ++r) {
                    if (r < each && i0 + r < e1 && !in_pool(pool, page[r])) {
                        flags |= SE_DEV_BAD_INDEX;
                        page[r] = -1;
                    }
                    if (page[r] != next[r]) open |= 1u << r;
                }
            }
            // bit r of m: entry r is freed; of last: it is its page's last of this call
            uint32_t m = 0, last = 0;
            if (phase == kPush && k < 32 / kEntries) {
                m = freed_bits >> (k * kEntries) & ((1u << kEntries) - 1);
                last = last_bits >> (k * kEntries) & ((1u << kEntries) - 1);
            } else if (phase >= kCount) {
#pragma unroll
                for (int r = 0; r < kEntries; ++r) {
                    if (page[r] < 0) continue;
                    if (!shared) {
                        m |= 1u << r;
                    } else if ((open >> r) & 1) {
                        const int n = __ldcg(refs + page[r]), of = __ldcg(who + page[r]);
                        if (of == seq[r] + 1) last |= 1u << r;
                        if (n < 0 && of == seq[r] + 1) m |= 1u << r;
                    }
                }
            }
            if (phase == kCount) {
                count += __popc(m);
                if (k < 32 / kEntries) {
                    freed_bits |= m << (k * kEntries);
                    last_bits |= last << (k * kEntries);
                }
                continue;
            }
            int tile = 0;
            if (phase == kPush && !(once && !wide))
                place = block_exclusive_scan(__popc(m), s_scan, &tile);
#pragma unroll
            for (int r = 0; r < kEntries; ++r) {
                const int p = page[r];
                if (p < 0) continue;
                if (phase == kProbe) {
                    any |= refs[p] > 0;
                } else if (phase == kCountDown) {
                    atomicSub(refs + p, 1);
                    if ((open >> r) & 1) atomicMax(who + p, seq[r] + 1);
                } else {
                    const bool f = (m >> r) & 1;
                    if (f && fits) pool.free_pages[top - place] = p;
                    place += f;
                    if (!shared) continue;
                    if (!fits) atomicAdd(refs + p, 1);
                    if (fits && f) refs[p] = 0;
                    if (!fits || ((last >> r) & 1)) who[p] = 0;
                }
            }
            top -= tile;
        }
        if (phase == kProbe) {
            shared = __syncthreads_or(any);
            phase = shared ? kCountDown : kCount;
        } else if (phase == kCountDown) {
            __threadfence();
            all_sync();
            phase = kCount;
        } else if (phase == kCount) {
            place = block_exclusive_scan(count, s_scan, &all_freed);
            if (wide) {
                if (threadIdx.x == 0) s_count = all_freed;
                cluster_sync();
                all_freed = 0;
                for (int r = 0; r < ranks; ++r) {
                    const int n = cluster_peek(&s_count, r);
                    before += r < rank ? n : 0;
                    all_freed += n;
                }
            }
            fits = (long long)n_free - taken + all_freed <= pool.num_pages;
            if (!fits) flags |= SE_DEV_CAPACITY;
            top = n_free - taken + all_freed - 1 - before;   // the stack's entries from here down
            phase = kPush;
        } else {
            if (wide || !once) all_sync();                   // the tables have been read
            phase = kEnd;
        }
    }
    if (flags) flag(ws, flags);
    if (rank != 0) return;
    for (int b = b0; b < b1; ++b) {
        const int fresh = fits ? s_fresh[b] : -2;
        int from_page = -1;
        if (fresh != -2) {
            const int ctx = b == b0 ? mine.ctx : pool.ctx_len[b];
            const int n = b == b0 ? mine.n : min(keep[b], ctx), after = (n + kPage - 1) / kPage;
            int32_t* last = pool.block_table + (int64_t)b * pool.max_pages_per_seq + after - 1;
            if (n % kPage != 0 && (n < ctx || fresh >= 0)) from_page = b == b0 ? mine.last : *last;
            if (fresh >= 0) *last = fresh;
            pool.ctx_len[b] = n;
            pool.n_pages[b] = after;
        }
        carry.from_seq[b] = -1;
        carry.from_page[b] = from_page;
    }
    if (fits && threadIdx.x == 0) *pool.n_free = n_free - taken + all_freed;
}

// ---- carry --------------------------------------------------------------------------------
// Block (x, b) copies its share of sequence b's summaries; block (0, b) also the rows of
// its last page, a warp for each KV head, whose summary it makes from them.  HBM bound when
// many summaries are copied (64 samples of a 32K prompt: 268 MB written in 43.9 us, 6.1 TB/s,
// their source read once into L2), else latency (2.6 to 4.3 us).  At 64 registers, twice the
// warps, 42 to 50 us.
template <int D>
__global__ void __launch_bounds__(128)
    pages_carry_kernel(se_paged_kv kv, se_page_carry carry, int batch, int* status) {
    constexpr int SEGS = D / 8, RP = 32 / SEGS, IT = kPage / RP, U = 8;
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.y, H = kv.num_kv_heads;
    const int from_seq = carry.from_seq[b], from_page = carry.from_page[b];
    if (from_seq < 0 && from_page < 0) return;
    const int n = kv.ctx_len[b], lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (n < 0 || n > (long long)kv.max_pages_per_seq * kPage) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag(status, SE_DEV_BAD_LENGTH);
        return;
    }
    uint4* M = static_cast<uint4*>(kv.meta);
    const int64_t page_vecs = (int64_t)H * 2 * SEGS, seq_vecs = kv.max_pages_per_seq * page_vecs;
    if (M != nullptr && from_seq >= 0 && from_seq != b) {
        if (from_seq >= batch) {
            if (blockIdx.x == 0 && threadIdx.x == 0) flag(status, SE_DEV_BAD_INDEX);
        } else {
            const uint4* src = M + from_seq * seq_vecs;
            uint4* dst = M + b * seq_vecs;
            const int64_t vecs = (n / kPage) * page_vecs, step = (int64_t)gridDim.x * blockDim.x;
            for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < vecs;
                 i += U * step) {
                uint4 x[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i + u * step < vecs) x[u] = src[i + u * step];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i + u * step < vecs) dst[i + u * step] = x[u];
            }
        }
    }
    const int rows = n % kPage;
    if (blockIdx.x != 0 || from_page < 0 || rows == 0) return;
    const int to = kv.block_table[(int64_t)b * kv.max_pages_per_seq + n / kPage];
    if (from_page >= kv.num_pages || to < 0 || to >= kv.num_pages) {
        if (threadIdx.x == 0) flag(status, SE_DEV_BAD_INDEX);
        return;
    }
    const bool move = from_page != to;
    uint4* K = static_cast<uint4*>(kv.k);
    uint4* V = static_cast<uint4*>(kv.v);
    const int seg = lane % SEGS, rp = lane / SEGS;
    for (int h = warp; h < H; h += blockDim.x >> 5) {
        const int64_t from = ((int64_t)from_page * H + h) * kPage * SEGS + seg;
        const int64_t at = ((int64_t)to * H + h) * kPage * SEGS + seg;
        uint4 k[IT], v[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = i * RP + rp;
            if (r < rows) {
                k[i] = K[from + r * SEGS];
                if (move) v[i] = V[from + r * SEGS];
            }
        }
        Bf8 mn, mx;
#pragma unroll
        for (int e = 0; e < 8; ++e)              // none yet: min and max pass a NaN over
            mn.x[e] = mx.x[e] = CUDART_NAN_F;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = i * RP + rp;
            if (r < rows) {
                if (move) {
                    K[at + r * SEGS] = k[i];
                    V[at + r * SEGS] = v[i];
                }
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
            const int64_t m0 = b * seq_vecs + (n / kPage) * page_vecs + (int64_t)h * 2 * SEGS + seg;
            M[m0] = pack8(mn);
            M[m0 + SEGS] = pack8(mx);
        }
    }
}

// Blocks of the truncation's cluster: 16 where the device has room for such a cluster, else the
// portable 8 (found once per device).
cudaError_t cluster_blocks(cudaLaunchConfig_t cfg, unsigned* blocks) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        e = cudaFuncSetAttribute(pages_truncate_kernel,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 16;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(1024);
        cfg.dynamicSmemBytes = 3 * kMaxBatch * sizeof(int);
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int fits = 0;
        if (cudaOccupancyMaxActiveClusters(&fits, pages_truncate_kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            fits = 0;
        }
        n = fits > 0 ? 16 : 8;
        if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    }
    *blocks = n;
    return cudaSuccess;
}

int table_threads(int batch) { return batch > 512 ? 1024 : batch > 256 ? 512 : 256; }

std::atomic<uint64_t> g_fork_smem, g_truncate_smem;

}  // namespace

int page_share_max_batch() { return kMaxBatch; }

size_t pages_truncate_ws_bytes(int num_pages) {
    return (kWhoWord * sizeof(int) + (size_t)num_pages * sizeof(int) + 255) & ~(size_t)255;
}

cudaError_t launch_pages_fork(const se_page_pool& pool, int32_t* refs, const int32_t* src, int batch,
                              const se_page_carry& carry, int* ws, cudaStream_t s) {
    const int nt = table_threads(batch);
    const cudaError_t e = allow_smem(pages_fork_kernel, 2 * kMaxBatch * sizeof(int), g_fork_smem);
    if (e != cudaSuccess) return e;
    // a block for every 1024 table entries that could be written
    const int grid = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(num_sms(), (int64_t)batch * pool.max_pages_per_seq / 1024)));
    return launch_pdl(pages_fork_kernel, dim3(grid), dim3(nt), 2 * batch * sizeof(int), s, pool,
                      refs, src, batch, carry, ws);
}

cudaError_t launch_pages_truncate(const se_page_pool& pool, int32_t* refs, const int32_t* keep,
                                  int batch, const se_page_carry& carry, int* ws, cudaStream_t s) {
    cudaError_t e = allow_smem(pages_truncate_kernel, 3 * kMaxBatch * sizeof(int), g_truncate_smem);
    if (e != cudaSuccess) return e;

    // a cluster when more pages could be let go than a block takes at once (shared pages
    // count each time), with the threads that hold them all: 1024 of them wait for empty SMs
    // (16 sequences of 1,848 pages at most that let go of a few, with their append: 18.5 us
    // with 256 threads, 20.8 with 1024; 133,000 at most, all let go: 90 us with 512, 80 with 1024)
    int64_t most = (int64_t)batch * pool.max_pages_per_seq;
    if (refs == nullptr) most = std::min<int64_t>(most, pool.num_pages);
    unsigned ranks = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(table_threads(batch));
    if (most > 4 * 1024) {
        while (cfg.blockDim.x < 1024 && most > 16 * kEntries * cfg.blockDim.x) cfg.blockDim.x *= 2;
        e = cluster_blocks(cfg, &ranks);
        if (e != cudaSuccess) return e;
    }
    return launch_cluster(pages_truncate_kernel, dim3(ranks), cfg.blockDim, 3 * batch * sizeof(int),
                          ranks, s, pool, refs, keep, batch, carry, ws);
}

cudaError_t launch_pages_carry(const se_paged_kv& kv, const se_page_carry& carry, int batch,
                               int* status, cudaStream_t s) {
    // a block moves 16 KB of summaries at once; as many a sequence as fill the GPU
    const int64_t vecs = (int64_t)kv.max_pages_per_seq * kv.num_kv_heads * kv.head_dim / 4;
    const int split = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>((vecs + 1023) / 1024, 16 * num_sms() / batch)));
    const dim3 grid(kv.meta != nullptr ? split : 1, batch);
    if (kv.head_dim == 128)
        return launch_pdl(pages_carry_kernel<128>, grid, dim3(128), 0, s, kv, carry, batch, status);
    return launch_pdl(pages_carry_kernel<64>, grid, dim3(128), 0, s, kv, carry, batch, status);
}

}  // namespace se
