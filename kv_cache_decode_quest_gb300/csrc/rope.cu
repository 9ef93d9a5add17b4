// Norms of queries and keys per head with the rotation to the token's position
// (se_qk_rope), and the same ahead of the append of a chunk (se_rope_append_chunk): what a
// layer does to its packed q | k | v rows before the attention over the paged cache (pages and
// a table from tokens to pages: "长程 agent 把显存撑爆以后", section "四、为什么进不了 vLLM 一类的引擎").
//
// A head's row is x' = R(pos) diag(w) x / sqrt(mean x^2 + eps), R a rotation of pairs of
// channels by pos * f_i.  The angle is kept in turns as a 64-bit fraction: pos * turns[i]
// mod 2^64 is exact in integers at any position (two 32-bit multiplies), where pos * f_i in
// fp32 would be off by 2^-24 of the angle itself, 0.06 rad at position 10^6.  Its upper 32
// bits are half a turn's signed fraction for sincospif.  Norm, weights and rotation are fp32
// (packed two by two), rounded once, to bf16.
//
// Layout: a lane owns 8 whole pairs of a head, two 16-byte vectors: with halves, vector j
// and vector j + rot_dim / 16; with pairs, vectors 2j and 2j + 1.  Either way its angles
// are 8j .. 8j + 7, no value crosses lanes in the rotation, and a head takes D / 16 lanes:
// a warp has 512 / D heads side by side.  Channels past rot_dim lie in lanes of their own,
// which leave the rotation out.
#include <algorithm>

#include "chunk_rows.cuh"
#include "common.cuh"
#include "internal.h"

namespace se {
namespace {

// The lane's place in a head of D channels: its two vectors, and whether it rotates.
template <int D, bool PAIRS>
struct HeadLane {
    int j, a, b;
    bool turns;
    __device__ HeadLane(int lane, int rot) {
        j = lane % (D / 16);
        const int r = rot / 16;                          // lanes that rotate
        turns = j < r;
        a = PAIRS ? 2 * j : turns ? j : 2 * j;
        b = PAIRS || !turns ? a + 1 : j + r;
    }
};

// Eight pairs (x, y) of two vectors, two by two in packed fp32: of halves, channel i of one
// and of the other; of pairs, channels 2i and 2i + 1 of the two as one run.
template <bool PAIRS>
__device__ __forceinline__ void to_pairs(uint4 u, uint4 v, uint64_t* x, uint64_t* y) {
    const uint32_t p[4] = {u.x, u.y, u.z, u.w}, q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (PAIRS) {
            const uint32_t a = i < 2 ? p[(2 * i) & 3] : q[(2 * i) & 3];
            const uint32_t b = i < 2 ? p[(2 * i + 1) & 3] : q[(2 * i + 1) & 3];
            x[i] = f32x2(bf_lo(a), bf_lo(b));
            y[i] = f32x2(bf_hi(a), bf_hi(b));
        } else {
            x[i] = f32x2(bf_lo(p[i]), bf_hi(p[i]));
            y[i] = f32x2(bf_lo(q[i]), bf_hi(q[i]));
        }
    }
}
// The i-th two pairs back, rounded to bf16.
template <bool PAIRS>
__device__ __forceinline__ void from_pairs(int i, uint64_t x, uint64_t y, uint32_t* p,
                                           uint32_t* q) {
    float a, b, c, d;
    f32x2_split(x, a, b);
    f32x2_split(y, c, d);
    if (PAIRS) {
        (i < 2 ? p : q)[(2 * i) & 3] = pack_bf16(a, c);
        (i < 2 ? p : q)[(2 * i + 1) & 3] = pack_bf16(b, d);
    } else {
        p[i] = pack_bf16(a, b);
        q[i] = pack_bf16(c, d);
    }
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Cosine and sine of one pair's angle at position pos, times the amplitude.
__device__ __forceinline__ void turn_of(unsigned long long turns, float amplitude, int pos,
                                        float& c, float& s) {
    const unsigned long long t = static_cast<uint32_t>(pos) * turns;
    const float half_turns = static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f;
    sincospif(half_turns, &s, &c);
    c *= amplitude;
    s *= amplitude;
}

// The norm's weights of this lane's pairs.
struct Weight {
    uint64_t x[4], y[4];
};
template <int D, bool PAIRS>
__device__ __forceinline__ Weight load_weight(const void* w, const HeadLane<D, PAIRS>& l) {
    Weight r = {};
    if (w != nullptr) {
        const uint4* v = static_cast<const uint4*>(w);
        to_pairs<PAIRS>(v[l.a], v[l.b], r.x, r.y);
    }
    return r;
}

// A row's rotation of this lane's pairs: cosines, sines, and the sines negated.
struct Turn {
    uint64_t c[4], s[4], n[4];
    __device__ __forceinline__ void set(const float* cos, const float* sin) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = f32x2(cos[2 * i], cos[2 * i + 1]);
            s[i] = f32x2(sin[2 * i], sin[2 * i + 1]);
            n[i] = f32x2(-sin[2 * i], -sin[2 * i + 1]);
        }
    }
};

// One head's two vectors of this lane: normed over the head's D / 16 lanes, weighted,
// rotated, rounded.  ALL: every channel is rotated; else only the lanes of which `turns` holds
// rotate (a cosine of 1 and a sine of 0 would make NaN of a value beside an infinity).  The
// choice costs two selects a value: 16,384 rows of 16 heads of 64 channels take 14.3 us with it,
// 13.8 where all rotate and it is left out; the append of 8 x 8192 rows 214 and 210 us.
template <int D, bool PAIRS, bool ALL>
__device__ __forceinline__ void norm_turn(uint4& u, uint4& v, bool norm, const Weight& w, float eps,
                                          bool turns, const Turn& t) {
    uint64_t x[4], y[4], both = 0;
    to_pairs<PAIRS>(u, v, x, y);
    if (norm) {
        uint64_t sum = mul_f32x2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) sum = fma_f32x2(x[i], x[i], sum);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = fma_f32x2(y[i], y[i], sum);
        float lo, hi;
        f32x2_split(sum, lo, hi);
        float ss = lo + hi;
#pragma unroll
        for (int o = 1; o < D / 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(fmaf(ss, 1.0f / D, eps));
        both = f32x2(inv, inv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = mul_f32x2(x[i], w.x[i]);
            y[i] = mul_f32x2(y[i], w.y[i]);
        }
    }
    uint32_t p[4], q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t a = x[i], b = y[i];
        if (ALL || turns) {
            a = fma_f32x2(x[i], t.c[i], mul_f32x2(y[i], t.n[i]));
            b = fma_f32x2(y[i], t.c[i], mul_f32x2(x[i], t.s[i]));
        }
        if (norm) {
            a = mul_f32x2(a, both);
            b = mul_f32x2(b, both);
        }
        from_pairs<PAIRS>(i, a, b, p, q);
    }
    u = make_uint4(p[0], p[1], p[2], p[3]);
    v = make_uint4(q[0], q[1], q[2], q[3]);
}

struct HeadRows {
    const uint4* in;
    uint4* out;
    int64_t in_stride, out_stride;      // 16-byte vectors between tokens
    int heads;
};

// ---- rows of heads --------------------------------------------------------------------------
// A warp takes a row, or one of `parts` parts of its passes (512 / D heads each, queries
// first, then keys) when there are few rows.  Its lanes make the row's angles together (two
// each at most) and hand them round.
// A row is two latencies (its position with the first pass, then the stores), so what counts
// is how many warps wait at once: 64 registers, one pass at a time, 32 warps an SM (up to 32
// bytes are spilled).  16,384 rows of 16 heads of 64 channels, pairs: 13.4 us where 32 rotate,
// 5.0 TB/s of rows read and written (74% of the copy rate), issue slots half busy; with norms
// 14.3, halves 14.6; where all rotate 13.9 and 14.4.  What was 12.9 then took 18.0 us with four
// passes a warp in flight and 100 registers, 18.7 to 20.6 through a ring in shared memory, 16.5
// with a table of angles for 16 rows a block.  64 rows of 36 heads of 128 (a decode step): 1.9 us.
// AHEAD: the next pass is loaded before this one is worked on, at 72 registers and 24 to 64 bytes
// spilled (16,384 rows of 36 heads of 128 channels, nine passes: 49.6 to 50.6 us, 89% of the copy
// rate, against 52.7 us; rows of two passes 13.7 us against 12.9).
template <int D, bool PAIRS, bool ALL, bool AHEAD>
__global__ void __launch_bounds__(128, AHEAD ? 7 : 8)
    qk_rope_kernel(se_rope rope, const int32_t* pos, int rows, int parts, HeadRows q, HeadRows k) {
    constexpr int HP = 512 / D, A = D / 64;                  // heads a pass, angles a lane
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, mine = lane / (D / 16);
    const int nq = (q.heads + HP - 1) / HP, n = nq + (k.heads + HP - 1) / HP;
    int row = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), p0 = 0, p1 = n;
    if (parts > 1) {
        const int part = row % parts;
        row /= parts;
        p0 = n * part / parts;
        p1 = n * (part + 1) / parts;
    }
    if (row >= rows) return;
    const HeadLane<D, PAIRS> l(lane, rope.rot_dim);
    uint4 u = make_uint4(0, 0, 0, 0), v = u;
    auto load = [&](int p) {
        const HeadRows& h = p < nq ? q : k;
        const int head = (p < nq ? p : p - nq) * HP + mine;
        if (p < p1 && head < h.heads) {
            const uint4* in = h.in + (int64_t)row * h.in_stride + head * (D / 8);
            u = in[l.a];
            v = in[l.b];
        }
    };
    load(p0);
    const int at = pos[row];
    unsigned long long step[A];
#pragma unroll
    for (int i = 0; i < A; ++i)
        step[i] = A * lane + i < rope.rot_dim / 2 ? rope.turns[A * lane + i] : 0;
    if (at < 0) return;
    Turn t;
    {
        float ca[A], sa[A], c[8], s[8];
#pragma unroll
        for (int i = 0; i < A; ++i) turn_of(step[i], rope.amplitude, at, ca[i], sa[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = __shfl_sync(0xffffffffu, ca[i % A], (8 * l.j + i) / A);
            s[i] = __shfl_sync(0xffffffffu, sa[i % A], (8 * l.j + i) / A);
        }
        t.set(c, s);
    }
    auto turn = [&](const HeadRows& h, const void* weight, int begin, int end, int skip) {
        if (begin >= end) return;
        const Weight wt = load_weight<D, PAIRS>(weight, l);
        for (int p = begin; p < end; ++p) {
            auto pass = [&](uint4& a, uint4& b) {
                norm_turn<D, PAIRS, ALL>(a, b, weight != nullptr, wt, rope.eps, l.turns, t);
                const int head = (p - skip) * HP + mine;
                if (head < h.heads) {
                    uint4* out = h.out + (int64_t)row * h.out_stride + head * (D / 8);
                    out[l.a] = a;
                    out[l.b] = b;
                }
            };
            if (AHEAD) {
                uint4 a = u, b = v;
                load(p + 1);
                pass(a, b);
            } else {
                pass(u, v);
                load(p + 1);
            }
        }
    };
    turn(q, rope.q_weight, p0, min(p1, nq), 0);
    turn(k, rope.k_weight, max(p0, nq), p1, nq);
}

// ---- append ---------------------------------------------------------------------------------
constexpr int kRows = kPage;             // rows of a block
constexpr int kPasses = 4;               // passes (512 / D heads) of a unit of work
constexpr int kStages = 2;               // units in flight
constexpr int kAppendBlocks = 4;         // blocks an SM
constexpr int kTable = 2 * kRows - 1;    // rows of the table: a piece may reach past the block's

// The cosines and sines of the block's rows, in shared memory.  A lane finds its eight of
// either as four 16-byte words, the lanes' words side by side (no bank conflicts).
template <int D, bool PAIRS>
struct Turns {
    static constexpr int kLanes = D / 16;
    float* table;                        // [rows][4][D / 16][4]
    // This thread's angles: the same four of every row that it makes.
    unsigned long long step[4];
    __device__ __forceinline__ void load(const se_rope& rope) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = threadIdx.x % 16 + 16 * k;
            step[k] = i < rope.rot_dim / 2 ? rope.turns[i] : 0;
        }
    }
    // The rows of `mask` behind `first` that have a place (the others' entries mean nothing).
    __device__ __forceinline__ void make(const se_rope& rope, const int32_t* pos, int first,
                                         int rows, uint32_t mask) {
        for (int r = threadIdx.x / 16; r < kTable; r += blockDim.x / 16) {
            if (!((mask >> r) & 1)) continue;
            const int at = first + r < rows ? pos[first + r] : -1;
            if (at < 0) continue;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                const int i = threadIdx.x % 16 + 16 * k;
                float c, s;
                turn_of(step[k], rope.amplitude, at, c, s);
                float* t = table + r * D + ((i >> 2 & 1) * kLanes + (i >> 3)) * 4 + (i & 3);
                if (i < rope.rot_dim / 2) {
                    t[0] = c;
                    t[2 * kLanes * 4] = s;
                }
            }
        }
    }
    // This lane's of row r (nothing for a lane whose channels are not rotated).
    __device__ __forceinline__ void get(const HeadLane<D, PAIRS>& l, int r, Turn& turn) const {
        float c[8], s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = s[i] = 0.f;
        if (l.turns) {
            const float4* t = reinterpret_cast<const float4*>(table + r * D) + l.j;
            const float4 a = t[0], b = t[kLanes], d = t[2 * kLanes], e = t[3 * kLanes];
            c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
            c[4] = b.x; c[5] = b.y; c[6] = b.z; c[7] = b.w;
            s[0] = d.x; s[1] = d.y; s[2] = d.z; s[3] = d.w;
            s[4] = e.x; s[5] = e.y; s[6] = e.z; s[7] = e.w;
        }
        turn.set(c, s);
    }
};

// A warp's ring of kStages units of work, each of kPasses passes of two 16-byte vectors a
// lane: copied in by cp.async while the unit before is worked on.  A lane reads what it
// copied itself: no barriers.
constexpr int kRingWords = kStages * kPasses * 64;   // of a warp, 16 bytes each
struct Ring {
    uint4* mine;                         // this lane's first slot
    int in = 0, out = 0;                 // units copied and taken
    __device__ __forceinline__ uint4* slot(int unit, int pass) const {
        return mine + ((unit % kStages) * kPasses + pass) * 64;
    }
};

// The passes of the block's rows whose order is free, as a list: n a row, first its
// queries', then its values'.
struct PassList {
    HeadRows q;
    const uint4* v;
    int64_t v_stride;
    int nq, n, kv_heads;
    uint32_t inverse;                    // ceil(2^32 / n), 0 for n = 1
    __device__ __forceinline__ int row_of(int i) const {
        return inverse ? __umulhi(i, inverse) : i;
    }
};

// Two channels' smaller (larger) values at once; a NaN gives way to the other value.
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                     *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                     *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void fold(uint4& mn, uint4& mx, uint4 lo, uint4 hi) {
    mn = make_uint4(min2(mn.x, lo.x), min2(mn.y, lo.y), min2(mn.z, lo.z), min2(mn.w, lo.w));
    mx = make_uint4(max2(mx.x, hi.x), max2(mx.y, hi.y), max2(mx.z, hi.z), max2(mx.w, hi.w));
}
__device__ __forceinline__ uint4 shfl_xor4(uint4 x, int o) {
    return make_uint4(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o),
                      __shfl_xor_sync(0xffffffffu, x.z, o), __shfl_xor_sync(0xffffffffu, x.w, o));
}

// The cache row of head h of a token's slot.
__device__ __forceinline__ int64_t place_of(int slot, int heads, int h) {
    return ((int64_t)(slot / kPage) * heads + h) * kPage + slot % kPage;
}

// Append of packed rows with the rotation in front.  Pieces as in the plain append: the
// keys of one sequence's rows in one page, for the KV heads that a warp has side by side
// (fewer heads: rows beside them), are a warp's job; it rotates them, writes them and folds
// them, as rounded, into the page's summary, which it owns.  Rows follow one another in a
// lane, so the fold needs no exchange.  The queries and the values of the block's rows,
// whose order is free, are dealt out so that all warps have about as much to do.
// HBM bound for long chunks: eight prompts of 8192 rows (32 / 4 heads of 128) take 210 us, 6.4
// TB/s (94% of the copy rate), issue slots half busy.  What it took: copies a unit ahead (235
// us without), heads side by side instead of a head's rows (223), a short loop instead of four
// passes unrolled (232).  Latency bound below: 64 single tokens 5.1 us; 256 sequences with up
// to 65 rows 21.6 us (a third of the copy rate: 12 warps an SM, each a chain of some 17 passes).
template <int D, bool PAIRS, bool ALL>
__global__ void __launch_bounds__(128, kAppendBlocks)
    rope_append_chunk_kernel(se_paged_kv kv, se_rope rope, PassList list, const uint4* k_new,
                             int64_t k_stride, se_chunk ck, int batch, int side_shift,
                             int* status) {
    constexpr int SEGS = D / 8, HP = 512 / D;
    __shared__ __align__(16) float s_turns[kTable * D];
    __shared__ uint4 s_ring[4 * kRingWords];
    __shared__ uint32_t s_rows[4];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = lane / (D / 16);
    const int H = kv.num_kv_heads;
    const int first = static_cast<int>(blockIdx.x) * kRows;
    const HeadLane<D, PAIRS> l(lane, rope.rot_dim);
    Ring ring = {s_ring + warp * kRingWords + lane};
    Turns<D, PAIRS> turns;
    turns.table = s_turns;
    turns.load(rope);
    const int w = warp + (blockDim.x >> 5) * blockIdx.y, nw = (blockDim.x >> 5) * gridDim.y;
    const Pieces pieces = find_pieces(kv, ck, batch, static_cast<int>(blockIdx.x), lane);
    if (pieces.row.bad && lane >= 1 && lane <= kPage && warp == 0 && blockIdx.y == 0)
        flag(status, SE_DEV_BAD_INDEX);
    // keys: `side` heads side by side, HP / side rows beside them; job j is of piece j / groups
    const int side = 1 << side_shift, beside = HP >> side_shift;
    const int groups = (H + side - 1) >> side_shift;
    const int sub_head = mine & (side - 1), sub_row = mine >> side_shift;
    const int jobs = __popc(pieces.lead) * groups;
    // the list's passes: a warp has that much less of them as its jobs take
    const int passes = min(kRows, ck.max_tokens - first) * list.n;
    const int back = nw - 1 - w;                             // its first job
    int p0 = passes * w / nw, p1 = passes * (w + 1) / nw;
    if (nw <= 4 && jobs <= 64) {
        int cost = 0, all = 0;                               // lane i: of warp i's jobs
        for (int i = 0, job = 0; job < jobs; ++i) {
            const Piece pc = piece_at(pieces, i, lane);
            const int span = (32 - __clz(pc.rows) + beside - 1) / beside;
            for (int g = 0; g < groups; ++g, ++job) {
                if (job % nw == nw - 1 - lane) cost += span;
                all += span;
            }
        }
        int share = lane < nw ? max(0, (passes + all + nw - 1) / nw - cost) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, share, o);
            if (lane >= o) share += x;
        }
        const int total = max(1, __shfl_sync(0xffffffffu, share, 31));
        const int upto = __shfl_sync(0xffffffffu, share, w);
        const int before = __shfl_sync(0xffffffffu, share, max(w - 1, 0));
        p0 = passes * (w > 0 ? before : 0) / total;
        p1 = passes * upto / total;
    }
    const int units = (p1 - p0 + kPasses - 1) / kPasses;
    int copy_job = back, copy_sub = 0;
    auto piece_of = [&](int job) { return piece_at(pieces, job / groups, lane); };
    auto subs_of = [&](const Piece& pc) {                    // units of a job
        return (32 - __clz(pc.rows) + kPasses * beside - 1) / (kPasses * beside);
    };
    auto copy_next = [&]() {
        if (ring.in < units) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int p = p0 + ring.in * kPasses + i;
                if (p >= p1) break;
                const int r = list.row_of(p), at = p - r * list.n;
                const bool values = at >= list.nq;
                const int head = (values ? at - list.nq : at) * HP + mine;
                if (head < (values ? list.kv_heads : list.q.heads)) {
                    const uint4* in = values ? list.v + (first + r) * list.v_stride
                                             : list.q.in + (first + r) * list.q.in_stride;
                    in += head * SEGS;
                    cp_async16(ring.slot(ring.in, i), in + l.a, 16);
                    cp_async16(ring.slot(ring.in, i) + 32, in + l.b, 16);
                }
            }
        } else if (copy_job < jobs) {
            const Piece pc = piece_of(copy_job);
            const int head = (copy_job % groups) * side + sub_head;
            const uint4* in = k_new + (int64_t)(first + pc.f - 1) * k_stride + head * SEGS;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int r = (copy_sub * kPasses + i) * beside + sub_row;
                if (r < kPage && ((pc.rows >> r) & 1) && head < H) {
                    cp_async16(ring.slot(ring.in, i), in + r * k_stride + l.a, 16);
                    cp_async16(ring.slot(ring.in, i) + 32, in + r * k_stride + l.b, 16);
                }
            }
            if (++copy_sub == subs_of(pc)) {
                copy_sub = 0;
                copy_job += nw;
            }
        }
        ++ring.in;
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) copy_next();
    if (warp == 0 && blockIdx.y == 0)
        commit_lengths(kv, ck, batch, pieces.t, lane, pieces.row);
    // the rows whose angles the block's warps need (bits 16 and up: a piece may reach past
    // the block's rows)
    uint32_t need = 0;
    if (p0 < p1) need = (2u << list.row_of(p1 - 1)) - (1u << list.row_of(p0));
    for (int job = back; job < jobs; job += nw) {
        const Piece pc = piece_of(job);
        need |= pc.rows << (pc.f - 1);
    }
    if (lane == 0) s_rows[warp] = need;
    __syncthreads();
    turns.make(rope, ck.pos, first, ck.max_tokens, s_rows[0] | s_rows[1] | s_rows[2] | s_rows[3]);
    __syncthreads();
    uint4* K = static_cast<uint4*>(kv.k);
    uint4* V = static_cast<uint4*>(kv.v);
    uint4* M = static_cast<uint4*>(kv.meta);
    Turn t;
    if (units > 0) {
        const Weight wq = load_weight<D, PAIRS>(rope.q_weight, l);
        int row = -1, pos = -1, slot = -1;
        while (ring.out < units) {
            cp_async_wait<kStages - 1>();
#pragma unroll 1
            for (int i = 0; i < kPasses; ++i) {
                const int p = p0 + ring.out * kPasses + i;
                if (p >= p1) break;                          // (these are the same for the whole warp)
                const int r = list.row_of(p), at = p - r * list.n;
                if (r != row) {
                    row = r;
                    pos = __shfl_sync(0xffffffffu, pieces.row.pos, r + 1);
                    slot = __shfl_sync(0xffffffffu, pieces.row.slot, r + 1);
                    if (pos >= 0 && at < list.nq) turns.get(l, r, t);
                }
                uint4 u = ring.slot(ring.out, i)[0], v = ring.slot(ring.out, i)[32];
                if (at < list.nq) {
                    if (pos < 0) continue;
                    norm_turn<D, PAIRS, ALL>(u, v, rope.q_weight != nullptr, wq, rope.eps, l.turns, t);
                    const int head = at * HP + mine;
                    if (head < list.q.heads) {
                        uint4* out = list.q.out + (first + r) * list.q.out_stride + head * SEGS;
                        out[l.a] = u;
                        out[l.b] = v;
                    }
                } else {
                    const int head = (at - list.nq) * HP + mine;
                    if (slot >= 0 && head < H) {
                        uint4* out = V + place_of(slot, H, head) * SEGS;
                        out[l.a] = u;
                        out[l.b] = v;
                    }
                }
            }
            ++ring.out;
            copy_next();
        }
    }
    if (back >= jobs) return;
    const Weight wk = load_weight<D, PAIRS>(rope.k_weight, l);
    for (int job = back; job < jobs; job += nw) {
        const Piece pc = piece_of(job);
        const int head = (job % groups) * side + sub_head, r0 = pc.f - 1;
        const bool mine_too = head < H;
        uint4* out = K + place_of(pc.slot0, H, head) * SEGS;
        const int64_t page = (int64_t)pc.seq0 * kv.max_pages_per_seq + pc.pos0 / kPage;
        uint4* meta = M + (page * H + head) * 2 * SEGS;
        constexpr uint32_t kNone = 0x7fff7fffu;              // NaNs: the other value is taken
        uint4 mn[2], mx[2];
        mn[0] = mn[1] = mx[0] = mx[1] = make_uint4(kNone, kNone, kNone, kNone);
        const int subs = subs_of(pc), rows = 32 - __clz(pc.rows);
        for (int sub = 0; sub < subs; ++sub) {
            cp_async_wait<kStages - 1>();
#pragma unroll 1
            for (int i = 0; i < kPasses; ++i) {
                const int r = (sub * kPasses + i) * beside + sub_row;
                if ((sub * kPasses + i) * beside >= rows) break;   // the same for the whole warp
                const bool there = r < kPage && ((pc.rows >> r) & 1) && mine_too;
                uint4 a = ring.slot(ring.out, i)[0], b = ring.slot(ring.out, i)[32];
                turns.get(l, min(r0 + r, kTable - 1), t);
                norm_turn<D, PAIRS, ALL>(a, b, rope.k_weight != nullptr, wk, rope.eps, l.turns, t);
                if (there) {
                    out[r * SEGS + l.a] = a;
                    out[r * SEGS + l.b] = b;
                    fold(mn[0], mx[0], a, a);
                    fold(mn[1], mx[1], b, b);
                }
            }
            ++ring.out;
            copy_next();
        }
        if (M == nullptr) continue;
        uint4 old[4];
        const bool more = pc.pos0 % kPage != 0;              // the page has a summary already
        if (more && sub_row == 0 && mine_too) {
            old[0] = meta[l.a];
            old[1] = meta[l.b];
            old[2] = meta[SEGS + l.a];
            old[3] = meta[SEGS + l.b];
        }
        for (int o = side * (D / 16); o < 32; o <<= 1)
#pragma unroll
            for (int g = 0; g < 2; ++g)
                fold(mn[g], mx[g], shfl_xor4(mn[g], o), shfl_xor4(mx[g], o));
        if (sub_row == 0 && mine_too) {
            if (more) {
                fold(mn[0], mx[0], old[0], old[2]);
                fold(mn[1], mx[1], old[1], old[3]);
            }
            meta[l.a] = mn[0];
            meta[l.b] = mn[1];
            meta[SEGS + l.a] = mx[0];
            meta[SEGS + l.b] = mx[1];
        }
    }
}

HeadRows head_rows(const HeadArgs& a) {
    return HeadRows{static_cast<const uint4*>(a.in), static_cast<uint4*>(a.out), a.in_stride / 8,
                    a.out_stride / 8, a.heads};
}

template <int D, bool PAIRS>
cudaError_t rows_of(const se_rope& rope, const int32_t* pos, int rows, const HeadArgs& q,
                    const HeadArgs& k, cudaStream_t s) {
    constexpr int HP = 512 / D;
    const int passes = (q.heads + HP - 1) / HP + (k.heads + HP - 1) / HP;
    if (rows == 0 || passes == 0) return cudaSuccess;
    // few rows: their passes are spread over warps until the GPU has four a scheduler
    const int parts = std::max(1, std::min(passes, 16 * num_sms() / rows));
    const dim3 grid((rows * parts + 3) / 4);     // (parts is 1 for more than 16 num_sms() rows)
    auto run = [&](auto kernel) {
        return launch_pdl(kernel, grid, dim3(128), 0, s, rope, pos, rows, parts, head_rows(q),
                          head_rows(k));
    };
    if (rope.rot_dim == D)
        return passes > 2 * parts ? run(qk_rope_kernel<D, PAIRS, true, true>)
                                  : run(qk_rope_kernel<D, PAIRS, true, false>);
    return passes > 2 * parts ? run(qk_rope_kernel<D, PAIRS, false, true>)
                              : run(qk_rope_kernel<D, PAIRS, false, false>);
}

template <int D, bool PAIRS>
cudaError_t append_of(const se_paged_kv& kv, const se_rope& rope, const HeadArgs& q,
                      const void* k_new, const void* v_new, int64_t row_stride, const se_chunk& ck,
                      int batch, int* status, cudaStream_t s) {
    constexpr int HP = 512 / D;
    const int groups = (ck.max_tokens + kRows - 1) / kRows, H = kv.num_kv_heads;
    if (groups == 0) return cudaSuccess;
    PassList list = {head_rows(q), static_cast<const uint4*>(v_new), row_stride / 8,
                     (q.heads + HP - 1) / HP, 0, H, 0};
    list.n = list.nq + (H + HP - 1) / HP;
    if (list.n > 1) list.inverse = static_cast<uint32_t>(((1ull << 32) + list.n - 1) / list.n);
    const uint4* k = static_cast<const uint4*>(k_new);
    // few rows: several blocks share 16 of them, one wave of blocks at most, down to one pass a
    // warp (ragged chunks of 2,400 rows: 7.6 us; two waves 9.7)
    const int share = std::max(1, std::min(kAppendBlocks * num_sms() / groups,
                                           (kRows * (list.n + H) + 3) / 4));
    // KV heads side by side in a job of keys: many rows: as many as there are (a row's
    // rotation serves them together); few rows: one, so that a piece is several short jobs
    // (the ragged chunks 8.4 us against 13.2, the 65,536 rows 213 us against 211)
    int side_shift = 0;
    while (share == 1 && (2 << side_shift) <= std::min(H, HP)) ++side_shift;
    auto run = [&](auto kernel) {
        return launch_pdl(kernel, dim3(groups, share), dim3(128), 0, s, kv, rope, list, k,
                          row_stride / 8, ck, batch, side_shift, status);
    };
    return rope.rot_dim == D ? run(rope_append_chunk_kernel<D, PAIRS, true>)
                             : run(rope_append_chunk_kernel<D, PAIRS, false>);
}

}  // namespace

cudaError_t launch_qk_rope(const se_rope& rope, const int32_t* pos, int rows, int head_dim,
                           const HeadArgs& q, const HeadArgs& k, cudaStream_t s) {
    const bool pairs = rope.layout == SE_ROPE_PAIRS;
    if (head_dim == 128)
        return pairs ? rows_of<128, true>(rope, pos, rows, q, k, s)
                     : rows_of<128, false>(rope, pos, rows, q, k, s);
    return pairs ? rows_of<64, true>(rope, pos, rows, q, k, s)
                 : rows_of<64, false>(rope, pos, rows, q, k, s);
}

cudaError_t launch_rope_append_chunk(const se_paged_kv& kv, const se_rope& rope, const HeadArgs& q,
                                     const void* k_new, const void* v_new, int64_t row_stride,
                                     const se_chunk& ck, int batch, int* status, cudaStream_t s) {
    const bool pairs = rope.layout == SE_ROPE_PAIRS;
    auto run = [&](auto append) {
        return append(kv, rope, q, k_new, v_new, row_stride, ck, batch, status, s);
    };
    if (kv.head_dim == 128) return pairs ? run(append_of<128, true>) : run(append_of<128, false>);
    return pairs ? run(append_of<64, true>) : run(append_of<64, false>);
}

}  // namespace se
