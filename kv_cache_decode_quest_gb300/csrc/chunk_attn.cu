// Attention of a chunk of new tokens over a paged cache (se_chunk_attn), on the
// 5th-generation tensor cores.
//
// Rows (token, query head of the KV head's group) of one (sequence, KV head)
// share its keys.  A block is up to 256 such rows; it walks its keys in tiles of
// 128 (8 pages):  S = Q K^T,  P = exp2(S' - m),  l <- l + rowsum P,  O <- O + P V, with
// S' the logits times log2 e; where the reference m moves up to m', l and O are multiplied by
// exp2(m - m') first; at the end out = O / l and lse = ln 2 (m + log2 l).  Every running
// value is fp32; P is rounded to bf16 for the product with V (bf16 output: the result is
// rounded as coarsely anyway) or split into two bf16 terms (fp32 output: 16 mantissa bits).
// Relative L2 error of the output: 2.2 to 2.4e-3 for bf16, where rounding the output alone gives
// 1.7e-3 (two terms would bring it there for half as many MMAs again); for fp32 2e-6
// over 2K keys, 6e-5 over 32K in one accumulator, which the tensor cores round toward zero
// in every step of 16 keys.
//
// One resident CTA per SM takes an equal share of all key tiles of all blocks
// (a share may begin and end inside a block's keys), found from the lengths on the
// device, so there is no plan kernel and no host knowledge of lengths.  Warp roles:
//   producer  block-table look-ups, TMA copies of Q, and of K and V pages into a
//             ring of tiles (128-byte swizzle)
//   MMA       issues tcgen05.mma: S into tensor memory, P V with P read from tensor
//             memory (it replaces S in place)
//   softmax   two groups of four warps, one thread per row
// A block of more than 128 rows gives each softmax group its own 128 rows and both use
// each tile; a smaller one (short chunks, single tokens) gives them alternate
// tiles of the same rows, joined at the end through tensor memory.  While one group
// computes its exponentials, the tensor cores work for the other.  O stays in
// tensor memory and is rescaled only when a row's logits have outgrown the reference
// (the true maximum is not needed: any reference near it keeps P and l far from
// overflow, and the same one divides out).
// A block cut between CTAs is joined by the last of them to finish, in the
// order of its keys (the result does not depend on timing).
//
// Bound: 4 D flops per row and key on the tensor cores for chunks (32 MMAs of 64 clocks a
// tile for 256 rows: 2060 clocks), K and V from HBM for few rows.  Measured on a GB300
// (head_dim 128, 32 query heads, 4 KV heads, bf16; 20 calls after a rest / for two seconds on end,
// where the GPU is at its power limit): the last 2048 tokens of 32K in 650 / 696 us (1.65 /
// 1.54 PFLOP/s), a prompt of 8192 in 369 / 389 us (1.49 / 1.41 PFLOP/s); 16 sequences of 32K
// checking 8 tokens each in 169 us (6.4 TB/s).  A tile for 256 rows takes about 2950 clocks: without
// its softmax 2370, without the tensor cores 2500, its loads alone 2000.  What was
// measured (in bursts) and not kept: sixteen softmax warps, two threads a row (690 us against 665: issue
// slots, not latency, are short); an MMA warp for each group (789 us: the two fall into step
// instead of alternating); handing P over in halves (no difference); the running maximum in
// every tile (the row sum does: 2% on a mixed batch).
#include <algorithm>
#include <cstddef>

#include "cudaTypedefs.h"

#include "common.cuh"
#include "internal.h"

namespace se {
namespace {

constexpr int kBlockRows = 256;                    // rows of a block: two accumulators of 128
constexpr int kKeys = 128;                         // keys of a tile
constexpr int kTilePages = kKeys / kPage;
constexpr int kSoftWarps = 8;
constexpr int kThreads = (kSoftWarps + 4) * 32;    // + producer, MMA, two idle warps
// Registers a thread: the launch gives 384 threads 168 each; the four warps that
// do not compute rows hand theirs to the eight that do (88 * 128 + 208 * 256 =
// 168 * 384), which hold a row of 128 logits.
constexpr int kRegsFew = 88, kRegsMany = 208;
static_assert(kRegsFew * 128 + kRegsMany * 256 <= 168 * kThreads, "registers of the launch");
constexpr int kItems = 4;                          // work items in flight between the roles
constexpr int kMaxCtas = 256;
// Units of work, about 700 clocks each: a tile for two row groups is bound by the tensor
// cores and the softmax between them, one for a single group is shorter, and a block has a
// fixed part (Q, the pipeline's fill, the rows' output).
constexpr int kTileBoth = 4, kTileOne = 3, kBlockCost = 10;
constexpr int kJoinFlat = 8;                       // pieces joined in one go at most
// Units that a CTA should take: 8 suits a single query (11.9 us against 12.4 over 2K) and
// costs where there are several heads (24.0 against 22.9 over 16K); 24 costs both (13.9,
// 25.4).  U units go to ceil(U / kMinShare) CTAs at most, so a share is smaller where they do not
// divide: floor(U / n) for U >= kMinShare (n - 1) + 1, at the least (kMinShare + 1) / 2, with two
// CTAs.  That is more than a tile's units, which the joins rely on: every CTA between a cut
// block's first tile and its last holds one of them.
constexpr int kMinShare = 12;
static_assert((kMinShare + 1) / 2 >= kTileBoth, "a share holds a tile's first unit");
constexpr int kMaxBatch = 8192;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrowSum = 16384.f;                // a row sum of P above this moves the reference

// Workspace: status word, at byte 256 the arrival counters [kMaxCtas][2 levels][8 warps], then
// the partial results: two pieces per CTA (the one it takes over and the one it hands
// on), each [2 groups][128] (reference, sum) and [2][128][D] fp32.
constexpr size_t kCounterOff = 256;
constexpr size_t kPartOff = kCounterOff + kMaxCtas * 16 * sizeof(int);

template <int D>
struct Shape {
    static constexpr int kHalves = D / 64;                  // 64-column regions
    static constexpr int kRegion = 128 * 128;               // 128 rows of 128 bytes
    static constexpr int kTile = kHalves * kRegion;         // 128 rows of Q, K or V
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr size_t kCtrl = 3 * 1024;
    static constexpr size_t kSmem = (size_t)(2 + kStages) * kTile + kCtrl;
};

struct Item {
    int b, h;
    int tok0;          // packed row of the block's first token
    int rows;          // rows of the block (tokens * G)
    int pos0;          // position of the block's first token
    int len;           // tokens held
    int ts, tl;        // tile j is key tile j (j < ts), else j - ts + tl
    int j0, n;         // this piece: tiles [j0, j0 + n); n = 0: no more work
    int split;         // the block is cut: this piece is partial
    long long t0, t1;  // first units of the block's first and last tile
};

struct Params {
    se_paged_kv kv;
    se_chunk ck;
    int batch, G, lg, Hq;          // G = 1 << lg query heads per KV head
    int window, sink;
    float scale_log2;              // > 0
    uint32_t negate;               // instruction descriptor bit for a negative scale
    uint32_t wait_tries;           // a wait's failed tries before it gives up
    void* out;
    float* lse;
    uint8_t* ws;
};

struct Seq {
    int s0, n, p0, len;            // first packed row, new tokens, first position, tokens held
};

__device__ __forceinline__ Seq seq_info(const Params& p, int b, int& bad) {
    int s0 = p.ck.start[b], s1 = p.ck.start[b + 1];
    int len = p.kv.ctx_len[b];
    if (s0 < 0 || s0 > p.ck.max_tokens || s1 < s0 || s1 > p.ck.max_tokens) bad |= SE_DEV_BAD_LENGTH;
    s0 = min(max(s0, 0), p.ck.max_tokens);
    s1 = min(max(s1, 0), p.ck.max_tokens);
    const int cap = p.kv.max_pages_per_seq * kPage;
    if (len < 0 || len > cap) bad |= SE_DEV_BAD_LENGTH;
    Seq s;
    s.s0 = s0;
    s.n = max(0, s1 - s0);
    s.len = min(max(len, 0), cap);
    s.p0 = s.n > 0 ? p.ck.pos[s0] : 0;
    if (s.p0 < 0) {                 // no page was found for the chunk: its rows see nothing
        s.p0 = 0;
        s.len = 0;
    } else {
        s.p0 = min(s.p0, cap);
        if (s.n > 0 && s.p0 + s.n > s.len) bad |= SE_DEV_BAD_LENGTH;
    }
    return s;
}

// Blocks of sequence b are numbered from floor(start[b] * G / 256) + b on: each
// sequence has at most as many as the next one's first number leaves, and no
// scan over the sequences is needed.
__device__ __forceinline__ int first_block(int s0, int G, int b) { return s0 * G / kBlockRows + b; }

// Key tiles that block blk of a sequence looks at (at least one: a block that sees
// nothing has one tile, all of it masked).
struct Tiles {
    int rows, ts, tl, n;
};
__device__ __forceinline__ Tiles block_tiles(const Params& p, const Seq& s, int blk) {
    Tiles t = {0, 0, 0, 0};
    const int row0 = blk * kBlockRows;
    t.rows = min(kBlockRows, s.n * p.G - row0);
    if (blk < 0 || t.rows <= 0) return t;
    const int p_lo = s.p0 + (row0 >> p.lg);
    const int keys = min(p_lo + ((t.rows + p.G - 1) >> p.lg), s.len);    // keys below this are seen
    const int th = (keys + kKeys - 1) / kKeys;
    if (p.window > 0) {
        t.tl = min(max(0, p_lo - p.window + 1) / kKeys, th);
        t.ts = min(p.sink / kKeys + (p.sink % kKeys != 0), t.tl);
    }
    t.n = max(1, t.ts + th - t.tl);
    return t;
}

// Shares of U units over n CTAs: the first `extra` CTAs get one more than the others.
__device__ __forceinline__ unsigned long long udiv(unsigned long long a, unsigned long long b) {
    return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}
struct Shares {
    long long each, extra;
    __device__ __forceinline__ Shares(long long U, long long n)
        : each(static_cast<long long>(udiv(U, n))), extra(U - each * n) {}
    __device__ __forceinline__ Shares(long long each, long long extra, int)
        : each(each), extra(extra) {}
    __device__ __forceinline__ long long begin(int c) const {
        return each * c + min((long long)c, extra);
    }
    __device__ __forceinline__ int of(long long u) const {       // the CTA whose share holds unit u
        const long long big = extra * (each + 1);
        const long long c = u < big ? udiv(u, each + 1) : extra + udiv(u - big, each);
        return static_cast<int>(min(c, (long long)kMaxCtas - 1));   // (whatever `start` holds)
    }
};

__device__ __forceinline__ int tile_cost(int rows) { return rows > 128 ? kTileBoth : kTileOne; }
__device__ __forceinline__ int block_cost(const Tiles& t) {
    return t.n > 0 ? t.n * tile_cost(t.rows) + kBlockCost : 0;
}

__device__ __forceinline__ int tile_of(const Item& it, int j) {
    return j < it.ts ? j : j - it.ts + it.tl;
}

struct Ctrl {
    // barriers (initialised by a thread each: see barrier_count)
    uint64_t full[10], empty[10];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], o_done[2];
    uint64_t item_full[kItems], done;
    uint64_t p_full[2];                    // 4 warps each
    uint64_t ml_full, ml_empty;            // a shared block's two groups: all softmax warps
    uint64_t item_empty[kItems];           // all softmax warps and the MMA warp
    uint32_t tmem;
    int abort;
    uint32_t wait_tries;                   // Params::wait_tries, beside the flag it is looked at with
    int any_absent;                        // a block-table entry named no page
    long long share_each, share_extra;
    Item items[kItems];
    float2 ml[2][128];                     // of a block that both groups share
};

constexpr int kOnes = 10 + 10 + 2 + 2 + 2 + kItems + 1;
constexpr int kBarriers = kOnes + 2 + 2 + kItems;
__device__ __forceinline__ uint32_t barrier_count(int i) {
    return i < kOnes ? 1 : i < kOnes + 2 ? 4 : i < kOnes + 4 ? kSoftWarps : kSoftWarps + 1;
}

// Warp-uniform bounded wait.  Tries are counted rather than a clock read: that keeps the code
// of the many waits short, and a first pass through this kernel runs at the rate its
// code arrives.  A try that fails has been suspended by the hardware for a fixed time (3.75 us
// measured on a GB300), so the count is a time.  A suspension hint, or polling without one,
// made a chunk of 2048 at 32K 5% slower than this form.
constexpr int kTryNs = 3750;
constexpr int kWaitLimitDefaultNs = 1000 * 1000 * 1000;
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Ctrl* c, int* status) {
#pragma unroll 1
    for (uint32_t n = 0;; ++n) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (n >= c->wait_tries || __any_sync(0xffffffffu, *static_cast<volatile int*>(&c->abort)))
            break;
    }
    *static_cast<volatile int*>(&c->abort) = 1;
    flag(status, SE_DEV_TIMEOUT);
    return false;
}

// Two barriers at once.
__device__ __forceinline__ bool warp_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                           Ctrl* c, int* status) {
#pragma unroll 1
    for (uint32_t n = 0;; ++n) {
        const bool x = mbar_try_wait(a, pa), y = mbar_try_wait(b, pb);
        if (__all_sync(0xffffffffu, x && y)) return true;
        if (n >= c->wait_tries || __any_sync(0xffffffffu, *static_cast<volatile int*>(&c->abort)))
            break;
    }
    *static_cast<volatile int*>(&c->abort) = 1;
    flag(status, SE_DEV_TIMEOUT);
    return false;
}

// 4 x 4 transpose of 16-byte units over each group of four lanes: lane i ends with
// unit i of the rows that lanes 0..3 of the group held.
__device__ __forceinline__ void transpose4(uint4 (&x)[4], int lane) {
    auto swap = [&](uint4& a, uint4& b, int bit) {
        const bool up = lane & bit;
        const uint4 give = up ? a : b;
        uint4 got;
        got.x = __shfl_xor_sync(0xffffffffu, give.x, bit);
        got.y = __shfl_xor_sync(0xffffffffu, give.y, bit);
        got.z = __shfl_xor_sync(0xffffffffu, give.z, bit);
        got.w = __shfl_xor_sync(0xffffffffu, give.w, bit);
        if (up) a = got;
        else b = got;
    };
    swap(x[0], x[1], 1);
    swap(x[2], x[3], 1);
    swap(x[0], x[2], 2);
    swap(x[1], x[3], 2);
}

// Low n bits set (n clamped to [0, 32]).
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

template <int D, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const Params p) {
    using S = Shape<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* qs = smem;                                  // [2][kTile]
    uint8_t* ring = smem + 2 * S::kTile;                 // [kStages][kTile]
    Ctrl* c = reinterpret_cast<Ctrl*>(ring + S::kStages * S::kTile);
    static_assert(sizeof(Ctrl) <= S::kCtrl, "control block");
    static_assert((size_t)kMaxBatch * 20 + 1024 <= S::kSmem - S::kCtrl, "lengths fit beside");
    int* status = reinterpret_cast<int*>(p.ws);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = p.kv.num_kv_heads, G = p.G;

    static_assert(offsetof(Ctrl, tmem) == kBarriers * 8, "barriers first");
    if (threadIdx.x < kBarriers) {
        mbar_init(c->full + threadIdx.x, barrier_count(threadIdx.x));
        fence_barrier_init();
    }
    if (threadIdx.x == 0) {
        c->abort = 0;
        c->wait_tries = p.wait_tries;
        c->any_absent = 0;
    }
    if (warp == kSoftWarps + 1) tmem_alloc(&c->tmem, 512);
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share (the lengths are staged where Q and the ring will be) ----
    int* sums = reinterpret_cast<int*>(smem);
    Seq* seqs = reinterpret_cast<Seq*>(smem + 1024);
    int* firsts = reinterpret_cast<int*>(smem + 1024 + (size_t)kMaxBatch * sizeof(Seq));
    int max_blocks = 0;                              // blocks up to the last one with rows
    {
        int bad = 0;
        for (int b = threadIdx.x; b < p.batch; b += kThreads) {
            const Seq s = seq_info(p, b, bad);
            seqs[b] = s;
            firsts[b] = first_block(s.s0, G, b);
            if (s.n > 0) max_blocks = first_block(s.s0 + s.n, G, b) + 1;
        }
        if (bad && blockIdx.x == 0) flag(status, bad);
        max_blocks = __reduce_max_sync(0xffffffffu, max_blocks);
        if (lane == 0) sums[32 + warp] = max_blocks;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) max_blocks = max(max_blocks, sums[32 + w]);
    auto find_seq = [&](int x) {                     // last sequence whose first number is <= x
        int lo = 0, hi = p.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (firsts[mid] <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    // exclusive prefix of `v` over the threads; total in *sum (one barrier: the warps'
    // sums alternate between two buffers)
    int flip = 0;
    auto scan = [&](int v, long long* sum) -> long long {
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        int* part = sums + flip * 16;
        flip ^= 1;
        if (lane == 31) part[warp] = x;
        __syncthreads();
        long long before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const int y = part[w];
            before += w < warp ? y : 0;
            all += y;
        }
        *sum = all;
        return before + x - v;
    };
    // units in the order (block, head, tile); the fixed cost comes before a block's first
    // tile, and a tile belongs to the share that holds its first unit
    long long total = 0, mine = 0;
    int nt = 0, my_b = 0;
    const int passes = (max_blocks + kThreads - 1) / kThreads;
    for (int i = 0; i < passes; ++i) {
        const int x = i * kThreads + threadIdx.x;
        my_b = find_seq(x);
        nt = x < max_blocks ? block_cost(block_tiles(p, seqs[my_b], x - firsts[my_b])) : 0;
        long long sum;
        mine = scan(nt, &sum);
        total += sum;
    }
    // (every share has units for a tile: a block's pieces are those of consecutive CTAs)
    const long long U = total * H;
    const long long NC = min((long long)gridDim.x, (U + kMinShare - 1) / kMinShare);
    const Shares shares(U, max(1ll, NC));
    const bool idle = blockIdx.x >= NC;
    const long long u0 = idle ? 0 : shares.begin(blockIdx.x);
    const long long u1 = idle ? 0 : shares.begin(blockIdx.x + 1);
    long long* s_start = reinterpret_cast<long long*>(smem + 256);   // sequence, block, prefix
    if (u0 < u1) {
        long long base = 0;
        for (int i = 0; i < passes; ++i) {
            const int x = i * kThreads + threadIdx.x;
            long long sum;
            if (passes > 1) {
                my_b = find_seq(x);
                nt = x < max_blocks ? block_cost(block_tiles(p, seqs[my_b], x - firsts[my_b])) : 0;
                mine = scan(nt, &sum);
            } else {
                sum = total;
            }
            if ((base + mine) * H <= u0 && u0 < (base + mine + nt) * H) {
                s_start[0] = my_b;
                s_start[1] = x - firsts[my_b];
                s_start[2] = base + mine;
            }
            base += sum;
            if (base * H > u0) break;                // uniform
        }
    }
    if (threadIdx.x == 0) {
        c->share_each = shares.each;
        c->share_extra = shares.extra;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int b = 0, blk = 0;
    long long pre = 0;
    Seq win = {0, 0, 0, 0};                          // lane i: sequence b_win + i
    int b_win = 0;
    if (warp == kSoftWarps && u0 < u1) {
        b = static_cast<int>(s_start[0]);
        blk = static_cast<int>(s_start[1]);
        pre = s_start[2];
        b_win = b;
        if (b + lane < p.batch) win = seqs[b + lane];
    }
    const uint32_t tmem = c->tmem;

    if (warp >= kSoftWarps) {
        regs_fewer<kRegsFew>();
        if (warp == kSoftWarps) {
            // ------------------------------ producer ------------------------------
            fence_proxy_async_smem();                    // the staged lengths are read: TMA may write
            if (lane == 0) {
                prefetch_tmap(&tq);
                prefetch_tmap(&tk);
                prefetch_tmap(&tv);
            }
            uint32_t seq = 0;                            // ring positions used
            int items = 0, loads_q = 0;
            long long u = u0;
            int h = 0;
            bool first = true, go = true;
            while (go) {
                // the next block with tiles
                Seq s = {0, 0, 0, 0};
                Tiles t = {0, 0, 0, 0};
                if (u < u1) {
                    while (true) {
                        if (b >= b_win + 32) {
                            b_win = b;
                            int bad = 0;
                            if (b + lane < p.batch) win = seq_info(p, b + lane, bad);
                        }
                        const int src = b - b_win;
                        s.s0 = __shfl_sync(0xffffffffu, win.s0, src);
                        s.n = __shfl_sync(0xffffffffu, win.n, src);
                        s.p0 = __shfl_sync(0xffffffffu, win.p0, src);
                        s.len = __shfl_sync(0xffffffffu, win.len, src);
                        t = block_tiles(p, s, blk);
                        if (t.n > 0 || b + 1 >= p.batch) break;
                        ++b;
                        blk = 0;
                    }
                }
                const int cost = block_cost(t);
                Item it = {};
                it.b = b;
                it.n = 0;
                long long next = u1;
                if (u < u1 && t.n > 0) {             // (n is 0 if the share ends before a tile)
                    if (first) {
                        h = static_cast<int>(udiv(u - pre * H, cost));
                        first = false;
                    }
                    const long long us = pre * H + (long long)h * cost;      // the item's first unit
                    const long long t0 = us + kBlockCost;                    // its first tile's
                    next = min(u1, us + cost);
                    it.h = h;
                    it.tok0 = s.s0 + blk * (kBlockRows >> p.lg);
                    it.rows = t.rows;
                    it.pos0 = s.p0 + blk * (kBlockRows >> p.lg);
                    it.len = s.len;
                    it.ts = t.ts;
                    it.tl = t.tl;
                    const int per = tile_cost(t.rows);
                    it.j0 = static_cast<int>(udiv(max(0ll, u - t0) + per - 1, per));
                    it.n = static_cast<int>(udiv(max(0ll, next - t0) + per - 1, per)) - it.j0;
                    it.split = it.n < t.n;
                    it.t0 = t0;
                    it.t1 = us + cost - per;             // the last tile's first unit
                }
                // on to the next item: heads within the block, then the next block
                auto advance = [&]() {
                    u = next;
                    if (++h == H) {
                        h = 0;
                        pre += cost;
                        ++blk;
                    }
                };
                if (it.n == 0 && next < u1) {        // the share begins in the block's last tile
                    advance();
                    continue;
                }
                // lanes 0..15 issue a tile's boxes: page lane & 7, columns 64 * (lane >> 3)
                const int32_t* bt = p.kv.block_table + (int64_t)it.b * p.kv.max_pages_per_seq;
                const int absent_row = p.kv.num_pages * H * kPage;     // past the map: reads zero
                auto fetch = [&](int j) -> int {         // -1: a page past the end, or past the piece
                    const int pg = tile_of(it, it.j0 + j) * kTilePages + (lane & 7);
                    return (j < it.n && pg * kPage < it.len) ? bt[pg] : -1;
                };
                auto row_of = [&](int j, int phys) -> int {
                    const int pg = tile_of(it, it.j0 + j) * kTilePages + (lane & 7);
                    if (pg * kPage >= it.len) return absent_row;
                    if (phys < 0 || phys >= p.kv.num_pages) {
                        *static_cast<volatile int*>(&c->any_absent) = 1;
                        __threadfence_block();
                        flag(status, SE_DEV_BAD_INDEX);
                        return absent_row;
                    }
                    return (phys * H + it.h) * kPage;
                };
                // K's 64-column halves are regions of 128 rows (the tensor cores want all keys
                // at one stride); V's are kept page by page, so one box brings a page
                auto load = [&](bool keys, int row) -> bool {
                    const int st = seq % S::kStages;
                    if (!warp_wait(&c->empty[st], ((seq / S::kStages) & 1) ^ 1, c, status))
                        return false;
                    if (lane == 0) mbar_arrive_expect_tx(&c->full[st], S::kTile);
                    __syncwarp();
                    uint8_t* to = ring + st * S::kTile;
                    if (keys && lane < 8 * S::kHalves)
                        tma_load_2d(to + (lane >> 3) * S::kRegion + (lane & 7) * 2048, &tk,
                                    &c->full[st], (lane >> 3) * 64, row);
                    if (!keys && lane < 8)
                        tma_load_3d(to + lane * (2048 * S::kHalves), &tv, &c->full[st], 0, row, 0);
                    ++seq;
                    return true;
                };
                int nxt1 = fetch(0), nxt2 = fetch(1);
                const int slot = items % kItems;
                if (!warp_wait(&c->item_empty[slot], ((items / kItems) & 1) ^ 1, c, status)) break;
                if (lane == 0) {
                    c->items[slot] = it;
                    mbar_arrive(&c->item_full[slot]);
                }
                ++items;
                if (it.n == 0) break;
                int row_k = row_of(0, nxt1), row_v;
                go = load(true, row_k);
                if (go) {
                    go = warp_wait(&c->q_empty, (loads_q & 1) ^ 1, c, status);
                    if (go && lane == 0) {
                        const int tiles = it.rows > 128 ? 2 : 1;
                        mbar_arrive_expect_tx(&c->q_full, tiles * S::kTile);
                        for (int w = 0; w < tiles; ++w)
                            for (int hf = 0; hf < S::kHalves; ++hf)
                                tma_load_3d(qs + w * S::kTile + hf * S::kRegion, &tq, &c->q_full,
                                            hf * 64, it.h * G, it.tok0 + w * (128 >> p.lg));
                    }
                    __syncwarp();
                    if (go) ++loads_q;
                }
                for (int j = 0; go && j < it.n; ++j) {   // K of tile j + 1, then V of tile j
                    row_v = row_k;
                    nxt1 = nxt2;
                    nxt2 = fetch(j + 2);
                    if (j + 1 < it.n) {
                        row_k = row_of(j + 1, nxt1);
                        go = load(true, row_k);
                    }
                    if (go) go = load(false, row_v);
                }
                advance();
            }
            if (lane == 0) {
                // every copy has landed before the block exits
                volatile int never = 0;
                const uint32_t from = seq > (uint32_t)S::kStages ? seq - S::kStages : 0;
                for (uint32_t i = from; i < seq; ++i)
                    mbar_wait(&c->full[i % S::kStages], (i / S::kStages) & 1, &never);
                if (loads_q > 0) mbar_wait(&c->q_full, (loads_q - 1) & 1, &never);
            }
            __syncwarp();
        } else if (warp == kSoftWarps + 1) {
            // ------------------------------ MMA issuer ------------------------------
            // The whole warp runs this with the same values; an elected lane issues.
            // Descriptor words: the high one is the operand's layout, the low one
            // its address / 16 (and V's column stride), to which offsets are added.
            const uint64_t qd = umma_desc_sw128(smem_u32(qs)), kd = umma_desc_sw128(smem_u32(ring));
            const uint64_t vd = umma_desc_mn_sw128(smem_u32(ring), 2048);
            const uint32_t q_lo = static_cast<uint32_t>(qd), q_hi = static_cast<uint32_t>(qd >> 32);
            const uint32_t k_lo = static_cast<uint32_t>(kd), k_hi = static_cast<uint32_t>(kd >> 32);
            const uint32_t v_lo = static_cast<uint32_t>(vd), v_hi = static_cast<uint32_t>(vd >> 32);
            const uint32_t idesc_s = umma_idesc_bf16_f32(128, kKeys) | p.negate;
            const uint32_t idesc_o = umma_idesc_bf16_f32(128, D) | kUmmaBMnMajor;
            const uint32_t bar_empty = smem_u32(&c->empty[0]);
            const uint32_t bar_s = smem_u32(&c->s_full[0]), bar_o = smem_u32(&c->o_done[0]);
            const uint32_t bar_q = smem_u32(&c->q_empty);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            uint32_t st = 0, ph = 0;                     // ring stage and its phase
            uint32_t np0 = 0, np1 = 0;                   // phases of P of each group
            auto wait_stage = [&]() { return warp_wait(&c->full[st], ph, c, status); };
            auto next_stage = [&]() {
                if (++st == S::kStages) {
                    st = 0;
                    ph ^= 1;
                }
            };
            // S_w = Q_qt K^T; `beside` runs before the last four instructions, while those ahead of
            // them are being carried out
            auto scores = [&](uint32_t w, uint32_t qt, uint32_t stage, auto beside) {
                const uint32_t ka = k_lo + stage * (S::kTile / 16), qa = q_lo + qt * (S::kTile / 16);
#pragma unroll
                for (int x = 0; x < S::kHalves; ++x) {
                    if (x + 1 == S::kHalves) beside();
                    umma_bf16_warp4(tm + w * 128, qa + x * (S::kRegion / 16), q_hi,
                                    ka + x * (S::kRegion / 16), k_hi, idesc_s, x > 0);
                }
                umma_commit_warp(bar_s + w * 8);
            };
            constexpr int kPageV = 2048 * S::kHalves;    // bytes of a page of V: 16 keys, one K step
            // O_w (+)= P_w V; `there`: P is known to be there
            auto product = [&](uint32_t w, uint32_t stage, uint32_t acc, uint32_t phase,
                               bool there) -> bool {
                if (!there && !warp_wait(&c->p_full[w], phase, c, status)) return false;
                tc_fence_after();
                const uint32_t va = v_lo + stage * (S::kTile / 16);
#pragma unroll
                for (int part = 0; part < (F32 ? 2 : 1); ++part)
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        umma_bf16_ts_warp4<kPageV / 16>(tm + 256 + w * D,
                                                        tm + w * 128 + part * 64 + half * 32,
                                                        va + half * (4 * kPageV / 16), v_hi, idesc_o,
                                                        half + part > 0 ? 1u : acc);
                return true;
            };
            auto test = [&](uint64_t* bar, uint32_t phase) {
                return __all_sync(0xffffffffu, mbar_test_wait(bar, phase)) != 0;
            };
            for (int items = 0;; ++items) {
                const int slot = items % kItems;
                if (!warp_wait(&c->item_full[slot], (items / kItems) & 1, c, status)) break;
                const Item* ip = &c->items[slot];
                const int n = __shfl_sync(0xffffffffu, ip->n, 0);
                const bool both = __shfl_sync(0xffffffffu, ip->rows, 0) > 128;   // own rows each
                const int len = ip->len, ts = ip->ts, tl = ip->tl, j0 = ip->j0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&c->item_empty[slot]);
                if (n == 0) break;
                // rows of the last page past the held tokens may be anything, and 0 * NaN is
                // not 0: V's are cleared before the product.  They are in the piece's tile
                // `tail_j`, if any (the tiles of a block are in key order).
                const int tail_k0 = len / kKeys * kKeys;
                const int tail_t = tail_k0 / kKeys;
                const int tail_at = tail_t < ts ? tail_t : tail_t - tl + ts;
                const int tail_j =
                    len % kPage == 0 || (tail_t >= ts && tail_t < tl) ? -1 : tail_at - j0;
                auto clear_tail = [&](uint32_t stage) {
                    const int row = len % kPage;         // of the last page: 16 rows per half
                    uint8_t* v = ring + stage * S::kTile + (len - tail_k0) / kPage * kPageV;
                    for (int i = lane; i < (kPage - row) * 8 * S::kHalves; i += 32) {
                        const int x = row + i / (8 * S::kHalves), o = i % (8 * S::kHalves);
                        *reinterpret_cast<uint4*>(v + (o >> 3) * 2048 + x * 128 + (o & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                };
                // Ring order: K0, then for each tile j: K_{j + 1}, V_j.
                // This warp's own instructions decide how well the tensor cores are fed: a wait
                // that finds its barrier complete takes 100 to 160 clocks beside busy warps, and the
                // queue holds some 250 clocks of work.  So barriers that are needed after a
                // batch of instructions are tested before its end.
                if (!warp_wait2(&c->q_full, items & 1, &c->full[st], ph, c, status)) break;
                tc_fence_after();
                auto nothing = [] {};
                bool go = true;
                if (both) {
                    scores(0, 0, st, nothing);
                    scores(1, 1, st, nothing);
                    umma_commit_warp(bar_empty + st * 8);
                    if (n == 1) umma_commit_warp(bar_q);
                    next_stage();
                    bool kv = false, p0 = false, p1 = false;      // known to be there
#pragma unroll 1
                    for (int j = 0; j < n; ++j) {
                        const bool more = j + 1 < n;
                        const uint32_t ks = st, kph = ph;
                        if (more) next_stage();
                        const uint32_t vs = st, vph = ph;
                        next_stage();
                        if (!kv) go = warp_wait2(&c->full[ks], kph, &c->full[vs], vph, c, status);
                        if (!go) break;
                        if (j == tail_j) clear_tail(vs);
                        go = product(0, vs, j > 0, np0, p0);
                        if (!go) break;
                        np0 ^= 1;
                        if (more)
                            scores(0, 0, ks, [&] { p1 = test(&c->p_full[1], np1); });
                        else
                            umma_commit_warp(bar_o);
                        go = product(1, vs, j > 0, np1, more && p1);
                        if (!go) break;
                        np1 ^= 1;
                        umma_commit_warp(bar_empty + vs * 8);
                        if (more) {
                            // K_{j + 2} and V_{j + 1} follow in the ring
                            const uint32_t ka = st, kap = ph;
                            const bool far = j + 2 < n;
                            const uint32_t va = !far ? ka : ka + 1 == S::kStages ? 0 : ka + 1;
                            const uint32_t vap = va < ka ? kap ^ 1 : kap;
                            scores(1, 1, ks, [&] {
                                kv = test(&c->full[ka], kap) && test(&c->full[va], vap);
                                p0 = test(&c->p_full[0], np0);
                            });
                            umma_commit_warp(bar_empty + ks * 8);
                            if (!far) umma_commit_warp(bar_q);
                        } else {
                            umma_commit_warp(bar_o + 8);
                        }
                    }
                } else {
                    // tile j is group j & 1's; the scores run two tiles ahead
                    scores(0, 0, st, nothing);
                    umma_commit_warp(bar_empty + st * 8);
                    next_stage();
                    if (n > 1) {
                        if (!wait_stage()) break;
                        tc_fence_after();
                        scores(1, 0, st, nothing);
                        umma_commit_warp(bar_empty + st * 8);
                        next_stage();
                    }
                    if (n <= 2) umma_commit_warp(bar_q);
#pragma unroll 1
                    for (int j = 0; j < n; ++j) {
                        const uint32_t w = j & 1, vs = st;
                        go = wait_stage();
                        if (!go) break;
                        next_stage();
                        if (j == tail_j) clear_tail(vs);
                        go = product(w, vs, j > 1, w ? np1 : np0, false);
                        if (!go) break;
                        if (w) np1 ^= 1;
                        else np0 ^= 1;
                        umma_commit_warp(bar_empty + vs * 8);
                        if (j + 2 < n) {
                            go = wait_stage();
                            if (!go) break;
                            tc_fence_after();
                            scores(w, 0, st, nothing);
                            umma_commit_warp(bar_empty + st * 8);
                            next_stage();
                            if (j + 3 == n) umma_commit_warp(bar_q);
                        } else {
                            umma_commit_warp(bar_o + w * 8);
                        }
                    }
                }
                if (!go) break;
            }
            __syncwarp();
            umma_commit_warp(smem_u32(&c->done));        // every MMA of this CTA has finished
            volatile int never = 0;
            mbar_wait(&c->done, 0, &never);
            __syncwarp();
        }
    } else {
        // ------------------------------ softmax ------------------------------
        regs_more<kRegsMany>();
        const int w = warp >> 2, q4 = warp & 3;      // group, lane quadrant of tensor memory
        const int r = q4 * 32 + lane;                // row of the accumulator
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        const uint32_t t_s = lane_base + w * 128;
        const int lg = p.lg;
        const float sl2 = p.scale_log2;
        uint32_t ns = 0;                             // S tiles seen by this group
        uint32_t no = 0;                             // items with a product of this group's
        uint32_t n_ml = 0;
        for (int items = 0;; ++items) {
            const int slot = items % kItems;
            if (!warp_wait(&c->item_full[slot], (items / kItems) & 1, c, status)) break;
            const Item it = c->items[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->item_empty[slot]);
            if (it.n == 0) break;
            const bool both = it.rows > 128;
            const int wrow0 = both ? w * 128 : 0;    // the accumulator's first row in the block
            const int row = wrow0 + r;
            const bool warp_live = wrow0 + q4 * 32 < it.rows;
            // padding rows repeat the last row
            const int pos = it.pos0 + (min(row, it.rows - 1) >> lg);
            const int pos_lo = __shfl_sync(0xffffffffu, pos, 0);
            const int pos_hi = __shfl_sync(0xffffffffu, pos, 31);
            const int last = min(pos, it.len - 1);   // last key seen
            const int last_lo = min(pos_lo, it.len - 1);
            float m = -INFINITY, l = 0.f;            // reference (log2 units) and sum
            const int mine_n = both ? it.n : (it.n - w + 1) / 2;
            bool ok = true;
            for (int i = 0; i < mine_n; ++i) {
                ok = warp_wait(&c->s_full[w], ns & 1, c, status);
                if (!ok) break;
                ++ns;
                tc_fence_after();
                if (warp_live) {
                    const int j = both ? i : 2 * i + w;
                    const int k0 = tile_of(it, it.j0 + j) * kKeys;
                    float v[kKeys];
                    tmem_ld128(t_s, v);
                    const bool absent =
                        __any_sync(0xffffffffu, *static_cast<volatile int*>(&c->any_absent) != 0);
                    const bool whole = k0 + kKeys - 1 <= last_lo && !absent &&
                                       (p.window == 0 || k0 > pos_hi - p.window ||
                                        k0 + kKeys <= p.sink);
                    if (!whole) {
                        uint32_t pages = 0xffu;      // pages of the tile that are there
                        if (absent) {
                            bool there = false;
                            const int pg = k0 / kPage + (lane & 7);
                            if (pg * kPage < it.len) {
                                const int phys =
                                    p.kv.block_table[(int64_t)it.b * p.kv.max_pages_per_seq + pg];
                                there = phys >= 0 && phys < p.kv.num_pages;
                            }
                            pages = __ballot_sync(0xffffffffu, there) & 0xffu;
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int at = k0 + 32 * x;
                            uint32_t see = low_bits(last - at + 1);
                            if (p.window > 0)
                                see &= ~low_bits(pos - p.window + 1 - at) | low_bits(p.sink - at);
                            see &= ((pages >> (2 * x)) & 1 ? 0xffffu : 0u) |
                                   ((pages >> (2 * x + 1)) & 1 ? 0xffff0000u : 0u);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                v[32 * x + e] = (see >> e) & 1 ? v[32 * x + e] : -INFINITY;
                        }
                    }
                    // P is computed with the reference as it was, and its row sum, which is
                    // needed anyway, shows whether that still serves: no logit is more than
                    // log2(kGrowSum) above it if the sum is at most kGrowSum, and nothing comes
                    // near overflow.  So no maximum is taken but for rows that have outgrown their
                    // reference or have none yet; those are done again.  P goes to tensor
                    // memory, which nobody reads before it is handed over.
                    const uint64_t scale2 = f32x2(sl2, sl2);
                    uint64_t sum[2] = {0, 0};
                    float neg = m == -INFINITY ? 0.f : -m;
                    // keys per store of P: the fewer stores, the less the exponentials ahead of
                    // them drain (the two terms of fp32 output want the registers)
                    constexpr int kRun = F32 ? 32 : 64;
                    auto run_of = [&](int x) {
                        const uint64_t neg2 = f32x2(neg, neg);
                        uint32_t hi[kRun / 2], lo[kRun / 2];
#pragma unroll
                        for (int e = 0; e < kRun; e += 2) {
                            float a, d;
                            const uint64_t s2 = f32x2(v[kRun * x + e], v[kRun * x + e + 1]);
                            f32x2_split(fma_f32x2(s2, scale2, neg2), a, d);
                            a = ex2_approx(a);
                            d = ex2_approx(d);
                            sum[(e >> 1) & 1] = add_f32x2(sum[(e >> 1) & 1], f32x2(a, d));
                            hi[e / 2] = pack_bf16(a, d);
                            if (F32)
                                lo[e / 2] = pack_bf16(a - bf_lo(hi[e / 2]), d - bf_hi(hi[e / 2]));
                        }
                        if constexpr (F32) {
                            tmem_st16(t_s + 16 * x, hi);
                            tmem_st16(t_s + 64 + 16 * x, lo);
                        } else {
                            tmem_st32(t_s + 32 * x, hi);
                        }
                    };
                    bool settled = false;
                    float total;
#pragma unroll 1
                    while (true) {                   // (one copy of the code: it is long)
                        if (settled || i > 0) {
#pragma unroll
                            for (int x = 0; x < kKeys / kRun; ++x) run_of(x);
                            float s0, s1;
                            f32x2_split(add_f32x2(sum[0], sum[1]), s0, s1);
                            total = s0 + s1;
                        }
                        if (settled) break;
                        settled = true;
                        const bool grow = i == 0 || m == -INFINITY || !(total <= kGrowSum);
                        if (!__any_sync(0xffffffffu, grow)) break;
                        float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                        for (int e = 4; e + 8 <= kKeys; e += 8)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                mx[x] = fmaxf(fmaxf(mx[x], v[e + x]), v[e + 4 + x]);
#pragma unroll
                        for (int x = 0; x < 4; ++x) mx[x] = fmaxf(mx[x], v[kKeys - 4 + x]);
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
                        const float to = grow ? fmaxf(top, m) : m;
                        if (i > 0) {
                            // (the previous product was issued before these scores, so it is
                            // complete)
                            const float alpha = to == m ? 1.f : ex2_approx(m - to);
#pragma unroll 1
                            for (int x = 0; x < D; x += 16) {
                                uint32_t o[16];
                                tmem_ld16(lane_base + 256 + w * D + x, o);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st16(lane_base + 256 + w * D + x, o);
                            }
                            l *= alpha;
                        }
                        m = to;
                        neg = m == -INFINITY ? 0.f : -m;
                        sum[0] = sum[1] = 0;
                        tmem_st_wait();
                    }
                    l += total;
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c->p_full[w]);
            }
            if (!ok) break;
            // ---- the item's rows ----
            // columns of this group's share: all D of its rows, or half of D of the rows
            // that both groups share
            const int cols = both ? D : D / 2, col0 = both ? 0 : w * (D / 2);
            const int n1 = both ? 0 : it.n / 2;      // tiles of group 1 (shared rows)
            float w0 = 1.f, w1 = 0.f;                // weights of the two accumulators
            // (each group has at least one tile, but group 1 of one shared tile)
            if (mine_n > 0 && !warp_wait(&c->o_done[w], no++ & 1, c, status)) break;
            if (!both) {
                c->ml[w][r] = make_float2(m, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c->ml_full);
                if (!warp_wait(&c->ml_full, n_ml & 1, c, status)) break;
                const float2 a = c->ml[0][r], d = n1 > 0 ? c->ml[1][r] : make_float2(-INFINITY, 0.f);
                m = fmaxf(a.x, d.x);
                w0 = m == -INFINITY ? 1.f : ex2_approx(a.x - m);
                w1 = m == -INFINITY ? 0.f : ex2_approx(d.x - m);
                l = a.y * w0 + d.y * w1;
            }
            tc_fence_after();
            const bool live = row < it.rows;
            const float inv = l > 0.f ? 1.f / l : 0.f;
            // (token, head) row of `out` that row `x` of the block is
            auto out_row = [&](int x) {
                return (int64_t)(it.tok0 + (x >> lg)) * p.Hq + it.h * G + (x & (G - 1));
            };
            // 32 columns of the warp's 32 rows to `out`: four lanes write 64 bytes
            // of one row together (a lane by itself would touch one line per 16 bytes)
            auto store32 = [&](const float (&o)[32], float k, int x) {
                constexpr int kParts = F32 ? 2 : 1;
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    uint4 u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float* f = o + (F32 ? 16 * part + 4 * e : 8 * e);
                        if (F32)
                            u[e] = make_uint4(__float_as_uint(f[0] * k), __float_as_uint(f[1] * k),
                                              __float_as_uint(f[2] * k), __float_as_uint(f[3] * k));
                        else
                            u[e] = make_uint4(
                                pack_bf16(f[0] * k, f[1] * k), pack_bf16(f[2] * k, f[3] * k),
                                pack_bf16(f[4] * k, f[5] * k), pack_bf16(f[6] * k, f[7] * k));
                    }
                    transpose4(u, lane);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int x_row = wrow0 + q4 * 32 + (lane & ~3) + e;
                        const int64_t at = out_row(x_row) * D + x + (F32 ? 16 * part : 0);
                        uint8_t* to = static_cast<uint8_t*>(p.out) + at * (F32 ? 4 : 2);
                        if (x_row < it.rows) reinterpret_cast<uint4*>(to)[lane & 3] = u[e];
                    }
                }
            };
            // partial results of a cut block: [piece][group] (reference, sum) of 128 rows and
            // 16-byte column units of 128 rows each
            const size_t part_rows = (size_t)2 * 128;
            uint8_t* parts = p.ws + kPartOff;
            const size_t slot_bytes = part_rows * (8 + 4 * D);
            int c0 = 0, pieces = 1;                  // CTAs [c0, c0 + pieces) share the block
            if (it.split) {
                const Shares sh(c->share_each, c->share_extra, 0);
                c0 = sh.of(it.t0);
                pieces = sh.of(it.t1) - c0 + 1;
            }
            const int piece = 2 * blockIdx.x + (static_cast<int>(blockIdx.x) == c0 ? 1 : 0);
            auto part_ml = [&](int s) {
                return reinterpret_cast<float2*>(parts + s * slot_bytes) + w * 128;
            };
            auto part_o = [&](int s) {
                return reinterpret_cast<float4*>(parts + s * slot_bytes + part_rows * 8) +
                       (size_t)w * 32 * D + r;
            };
            if (warp_live) {
                if (it.split) {
                    part_ml(piece)[r] = make_float2(m, l);
                } else if (p.lse && live && (both || w == 0)) {
                    p.lse[out_row(row)] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
                }
#pragma unroll 1
                for (int x0 = 0; x0 < cols; x0 += 32) {
                    const int x = col0 + x0;
                    float o[32];
                    tmem_ld32(lane_base + 256 + (both ? w * D : 0) + x, o);
                    if (!both && n1 > 0) {
                        float o1[32];
                        tmem_ld32(lane_base + 256 + D + x, o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = o[e] * w0 + o1[e] * w1;
                    }
                    if (it.split) {
                        float4* dst = part_o(piece) + x0 / 4 * 128;
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                dst[e * 128] =
                                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                        __syncwarp();
                    } else {
                        store32(o, inv, x);
                    }
                }
            }
            tc_fence_before();
            if (!both) {
                // neither group's next product may start before both have read
                __syncwarp();
                if (lane == 0) mbar_arrive(&c->ml_empty);
                if (!warp_wait(&c->ml_empty, n_ml & 1, c, status)) break;
                ++n_ml;
            }
            if (!it.split || !warp_live) continue;
            // ---- the pieces of a cut block are joined by the last to finish: the warps of a
            // quadrant of a group, one in each CTA, by themselves.  Reading one piece after
            // another is bound by one SM's share of L2 (about 64 bytes a clock), so
            // many pieces are first joined in groups, by different SMs: about 2 sqrt(n) pieces
            // one after another instead of n.  Groups and order are fixed. ----
            const int mine = static_cast<int>(blockIdx.x) - c0;          // this CTA's piece
            int per = pieces;                                           // pieces in a group
            if (pieces > kJoinFlat)
                per = static_cast<int>(ceilf(sqrtf(static_cast<float>(pieces))));
            int first = mine / per * per;                               // the group's first piece
            int count = min(per, pieces - first), step = 1;
            bool final = per == pieces;
            while (true) {
                int is_last = 1;
                __syncwarp();
                if (lane == 0 && count > 1) {
                    int* counter = reinterpret_cast<int*>(p.ws + kCounterOff) +
                                   16 * (c0 + first) + (final ? 8 : 0) + warp;
                    // releases this warp's rows (ordered before it by the warp barrier) and
                    // acquires those of the warps that arrived earlier
                    int before;
                    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                                 : "=r"(before)
                                 : "l"(counter)
                                 : "memory");
                    is_last = before == count - 1;
                    if (is_last) *counter = 0;
                }
                if (!__shfl_sync(0xffffffffu, is_last, 0)) break;
                __syncwarp();
                auto slot_of = [&](int i) {
                    const int s = first + i * step;
                    return 2 * (c0 + s) + (s == 0 ? 1 : 0);
                };
                if (count > 1) {
                    // one pass over the pieces with a running reference: their loads overlap
                    float mm, ll;
#pragma unroll 1
                    for (int x0 = 0; x0 < cols; x0 += 32) {
                        float o[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.f;
                        mm = -INFINITY;
                        ll = 0.f;
#pragma unroll 2
                        for (int i = 0; i < count; ++i) {
                            const int sl = slot_of(i);
                            const float2 x = __ldcg(&part_ml(sl)[r]);
                            float4 y[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                y[e] = live ? __ldcg(part_o(sl) + (x0 / 4 + e) * 128)
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
                            const float up = fmaxf(mm, x.x), ref = up == -INFINITY ? 0.f : up;
                            const float was = ex2_approx(mm - ref), k = ex2_approx(x.x - ref);
                            mm = up;
                            ll = ll * was + x.y * k;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                o[4 * e] = o[4 * e] * was + y[e].x * k;
                                o[4 * e + 1] = o[4 * e + 1] * was + y[e].y * k;
                                o[4 * e + 2] = o[4 * e + 2] * was + y[e].z * k;
                                o[4 * e + 3] = o[4 * e + 3] * was + y[e].w * k;
                            }
                        }
                        __syncwarp();
                        if (final) {
                            store32(o, ll > 0.f ? 1.f / ll : 0.f, col0 + x0);
                        } else if (live) {           // in the place of the group's first piece
                            float4* dst = part_o(slot_of(0)) + x0 / 4 * 128;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                dst[e * 128] =
                                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                    }
                    if (!final)
                        part_ml(slot_of(0))[r] = make_float2(mm, ll);
                    else if (p.lse && live && (both || w == 0))
                        p.lse[out_row(row)] = ll > 0.f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
                }
                if (final) break;
                final = true;
                first = 0;
                step = per;
                count = (pieces + per - 1) / per;
            }
        }
    }
    // every role is done (copies landed, MMAs completed, tensor memory read)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftWarps + 1) tmem_dealloc(tmem, 512);
}

template <int D, bool F32>
cudaError_t run(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                const Params& p, int grid, cudaStream_t s) {
    auto kern = chunk_attn_kernel<D, F32>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, Shape<D>::kSmem, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(kThreads), Shape<D>::kSmem, s, tq, tk, tv, p);
}

}  // namespace

int chunk_attn_max_batch() { return kMaxBatch; }

size_t chunk_attn_ws_bytes(int, int, int, int, int D) {
    return kPartOff + (size_t)kMaxCtas * 2 * 256 * (8 + 4 * (size_t)D);
}

cudaError_t launch_chunk_attn(const se_paged_kv& kv, const se_chunk& ck, int batch,
                              const ChunkAttnArgs& a, void* ws, cudaEvent_t ev_begin,
                              cudaEvent_t ev_end, cudaStream_t s) {
    const int D = kv.head_dim, H = kv.num_kv_heads;
    Params p;
    p.kv = kv;
    p.ck = ck;
    p.batch = batch;
    p.G = a.Hq / H;
    for (p.lg = 0; 1 << p.lg < p.G;) ++p.lg;
    p.Hq = a.Hq;
    p.window = a.window;
    p.sink = a.sink;
    // a negative scale negates the products; a zero one becomes so small that
    // every logit is zero to fp32 (masked ones stay -inf)
    p.scale_log2 = std::max(std::abs(a.scale) * kLog2e, 1e-37f);
    p.negate = a.scale < 0.f ? kUmmaNegateA : 0u;
    p.wait_tries =
        static_cast<uint32_t>((a.wait_limit_ns > 0 ? a.wait_limit_ns : kWaitLimitDefaultNs) / kTryNs);
    p.out = a.out;
    p.lse = a.lse;
    p.ws = static_cast<uint8_t*>(ws);
    CUtensorMap tq, tk, tv;
    if (!encode_rows_map(&tk, kv.k, (int64_t)kv.num_pages * H * kPage, D) ||
        !encode_pages_map(&tv, kv.v, (int64_t)kv.num_pages * H * kPage, D) ||
        !encode_heads_map(&tq, a.q, ck.max_tokens, a.Hq, a.q_stride, p.G, D))
        return cudaErrorInvalidValue;
    const int grid = std::min(num_sms(), kMaxCtas);
    // inside a stream capture the timing events become event-record nodes
    auto record = [&](cudaEvent_t ev) {
        cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
        cudaError_t e2 = cudaStreamIsCapturing(s, &cs);
        if (e2 != cudaSuccess) return e2;
        return cs == cudaStreamCaptureStatusActive
                   ? cudaEventRecordWithFlags(ev, s, cudaEventRecordExternal)
                   : cudaEventRecord(ev, s);
    };
    cudaError_t e;
    if (ev_begin && (e = record(ev_begin)) != cudaSuccess) return e;
    const bool f32 = a.out_dtype == 1;
    if (D == 128)
        e = f32 ? run<128, true>(tq, tk, tv, p, grid, s) : run<128, false>(tq, tk, tv, p, grid, s);
    else
        e = f32 ? run<64, true>(tq, tk, tv, p, grid, s) : run<64, false>(tq, tk, tv, p, grid, s);
    if (e != cudaSuccess) return e;
    if (ev_end && (e = record(ev_end)) != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace se
