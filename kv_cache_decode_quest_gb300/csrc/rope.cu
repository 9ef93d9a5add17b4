// Norms of queries and keys per head with the rotation to the token's position (se_qk_rope), and the
// same ahead of the append of a chunk (se_rope_append_chunk): what a layer does to its packed q | k | v
// rows before the attention over the paged cache ("长程 agent 把显存撑爆以后", section
// "四、为什么进不了 vLLM 一类的引擎": pages and a table from tokens to pages).
//
// A head's row is x' = R(pos) diag(w) x / sqrt(mean x^2 + eps), R a rotation of pairs of channels by pos * f_i.
// The angle is kept in turns as a 64-bit fraction: pos * turns[i] mod 2^64 is exact in integers at
// any position (two 32-bit multiplies), where pos * f_i in fp32 would be off by 2^-24 of the angle
// itself, 0.06 rad at position 10^6.  Its upper 32 bits are half a turn's signed fraction for sincospif.
//
// Layout: a lane owns 8 whole pairs of a head, two 16-byte vectors: with halves, vector j and vector j
// + rot_dim / 16; with pairs, vectors 2j and 2j + 1.  Either way its angles are 8j .. 8j + 7, no value
// crosses lanes in the rotation, and a head takes D / 16 lanes: a warp has 512 / D heads side by
// side.  Channels past rot_dim lie in lanes of their own (cosine 1, sine 0).
#include <algorithm>

#include "append.cuh"
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

// Eight pairs (x, y) of two vectors, two by two in packed fp32: of halves, channel i of one and of the
// other; of pairs, channels 2i and 2i + 1 of the two as one run.
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
__device__ __forceinline__ void from_pairs(int i, uint64_t x, uint64_t y, uint32_t* p, uint32_t* q) {
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
__device__ __forceinline__ void turn_of(unsigned long long turns, float amplitude, int pos, float& c,
                                        float& s) {
    const unsigned long long t = static_cast<uint32_t>(pos) * turns;
    const float half_turns = static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f;
    sincospif(half_turns, &s, &c);
    c *= amplitude;
    s *= amplitude;
}

// The norm's weights of this lane's two vectors, as stored.
struct Weight {
    uint4 a, b;
};
template <int D, bool PAIRS>
__device__ __forceinline__ Weight load_weight(const void* w, const HeadLane<D, PAIRS>& l) {
    Weight r = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (w != nullptr) {
        r.a = static_cast<const uint4*>(w)[l.a];
        r.b = static_cast<const uint4*>(w)[l.b];
    }
    return r;
}

// A row's rotation of this lane's pairs: cosines and sines.
struct Turn {
    float c[8], s[8];
};
// Two pairs of it with the norm's weights in it: out = inv (x xx + y xy, y yy + x yx).
struct Turn2 {
    uint64_t xx, xy, yy, yx;
};
__device__ __forceinline__ Turn2 weighed(const Turn& t, int i, bool norm, const uint64_t* wx,
                                         const uint64_t* wy) {
    Turn2 r;
    r.xx = r.yy = f32x2(t.c[2 * i], t.c[2 * i + 1]);
    r.xy = f32x2(-t.s[2 * i], -t.s[2 * i + 1]);
    r.yx = f32x2(t.s[2 * i], t.s[2 * i + 1]);
    if (norm) {
        r.xx = mul_f32x2(r.xx, wx[i]);
        r.xy = mul_f32x2(r.xy, wy[i]);
        r.yy = mul_f32x2(r.yy, wy[i]);
        r.yx = mul_f32x2(r.yx, wx[i]);
    }
    return r;
}

// One head's two vectors of this lane: normed over the head's D / 16 lanes, weighted, rotated, rounded.
// turn(i) gives the i-th two pairs' Turn2.
template <int D, bool PAIRS, typename F>
__device__ __forceinline__ void norm_turn(uint4& u, uint4& v, bool norm, float eps, F turn) {
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
    }
    uint32_t p[4], q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Turn2 t = turn(i);
        uint64_t a = fma_f32x2(x[i], t.xx, mul_f32x2(y[i], t.xy));
        uint64_t b = fma_f32x2(y[i], t.yy, mul_f32x2(x[i], t.yx));
        if (norm) {
            a = mul_f32x2(a, both);
            b = mul_f32x2(b, both);
        }
        from_pairs<PAIRS>(i, a, b, p, q);
    }
    u = make_uint4(p[0], p[1], p[2], p[3]);
    v = make_uint4(q[0], q[1], q[2], q[3]);
}

#ifndef RMIN
#define RMIN 8
#endif
#ifndef AMIN
#define AMIN 4
#endif
#ifndef RPASS
#define RPASS 1
#endif
struct HeadRows {
    const uint4* in;
    uint4* out;
    int64_t in_stride, out_stride;      // 16-byte vectors between tokens
    int heads;
};

constexpr int kRows = kPage;             // rows of a block
constexpr int kPasses = 4;               // passes of a unit of work
#ifndef STAGES
#define STAGES 2
#endif
constexpr int kStages = STAGES;
constexpr int kTable = 2 * kRows - 1;    // rows of the table: a piece may reach 15 rows past the block's

// The cosines and sines of the block's rows: a table in shared memory, or (few rows, many blocks that
// share them: TABLE false) made by each lane for itself as it needs them.  In the table a lane finds its
// eight of either as four 16-byte words, the lanes' words side by side (no bank conflicts).
template <int D, bool PAIRS, bool TABLE>
struct Turns {
    static constexpr int kLanes = D / 16;
    float* table;                        // [rows][4][D / 16][4]
    // Rows [0, n) behind `first`; pos says which have a place.  Every thread calls it.
    __device__ __forceinline__ void make(const se_rope& rope, const int32_t* pos, int first, int rows,
                                         int n) {
        if (!TABLE) return;
        const int half = rope.rot_dim / 2;
        for (int r = threadIdx.x / 16; r < n; r += blockDim.x / 16) {
            const int at = first + r < rows ? pos[first + r] : -1;
            for (int i = threadIdx.x % 16; i < half; i += 16) {
                float c = 1.f, s = 0.f;
                if (at >= 0) turn_of(rope.turns[i], rope.amplitude, at, c, s);
                float* t = table + r * D + ((i >> 2 & 1) * kLanes + (i >> 3)) * 4 + (i & 3);
                t[0] = c;
                t[2 * kLanes * 4] = s;
            }
        }
        __syncthreads();
    }
    // This lane's eight of row r (position at).
    __device__ __forceinline__ void get(const se_rope& rope, const HeadLane<D, PAIRS>& l, int r, int at,
                                        float* c, float* s) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = 1.f;
            s[i] = 0.f;
        }
        if (!l.turns) return;
        if (TABLE) {
            const float4* t = reinterpret_cast<const float4*>(table + r * D) + l.j;
            const float4 a = t[0], b = t[kLanes], d = t[2 * kLanes], e = t[3 * kLanes];
            c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
            c[4] = b.x; c[5] = b.y; c[6] = b.z; c[7] = b.w;
            s[0] = d.x; s[1] = d.y; s[2] = d.z; s[3] = d.w;
            s[4] = e.x; s[5] = e.y; s[6] = e.z; s[7] = e.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn_of(rope.turns[8 * l.j + i], rope.amplitude, at, c[i], s[i]);
        }
    }
};

// The heads of the block's rows, 512 / D side by side a pass, as a list of n passes a row.
struct PassList {
    HeadRows q;
    int n;
    uint32_t inverse;                    // ceil(2^32 / n), 0 for n = 1
    __device__ __forceinline__ int row_of(int i) const { return inverse ? __umulhi(i, inverse) : i; }
};
// A warp's ring of kStages units of work, each of kPasses passes of two 16-byte vectors a lane: copied in by
// cp.async while the unit before is worked on.  A lane reads what it copied itself: no barriers.
struct Ring {
    uint4* mine;                         // this lane's first slot
    __device__ __forceinline__ uint4* slot(int unit, int pass) const {
        return mine + ((unit % kStages) * kPasses + pass) * 64;
    }
};
constexpr int kRingWords = kStages * kPasses * 64;   // of a warp, 16 bytes each

// Copies the vectors of passes [p, p1) (kPasses at most) of the list as unit k.
template <int D, bool PAIRS>
__device__ __forceinline__ void copy_passes(const Ring& ring, int k, const PassList& list, int first,
                                            int p, int p1, const HeadLane<D, PAIRS>& l, int mine) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        if (p + i >= p1) break;
        const int r = list.row_of(p + i), head = (p + i - r * list.n) * (512 / D) + mine;
        if (head < list.q.heads) {
            const uint4* in = list.q.in + (first + r) * list.q.in_stride + head * (D / 8);
            cp_async16(ring.slot(k, i), in + l.a, 16);
            cp_async16(ring.slot(k, i) + 32, in + l.b, 16);
        }
    }
}
// The row that a warp is at, and its rotation: it serves the row's heads one after another.
struct RowTurn {
    int row = -1, pos = -1;
    Turn2 t[4];
};
// Turns passes [p, p1) (kPasses at most), which are unit k of the ring.
template <int D, bool PAIRS, bool TABLE>
__device__ __forceinline__ void turn_passes(const Ring& ring, int k, const PassList& list,
                                            const int32_t* pos, int first, int p, int p1,
                                            const HeadLane<D, PAIRS>& l, int mine, const se_rope& rope,
                                            const Turns<D, PAIRS, TABLE>& turns, RowTurn& now) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        if (p + i >= p1) break;                              // (these are the same for the whole warp)
        const int r = list.row_of(p + i), head = (p + i - r * list.n) * (512 / D) + mine;
        if (r != now.row) {
            now.row = r;
            now.pos = pos[first + r];
            if (now.pos >= 0) {
                Turn t;
                turns.get(rope, l, r, now.pos, t.c, t.s);
                const Weight w = load_weight<D, PAIRS>(rope.q_weight, l);
                uint64_t wx[4], wy[4];
                to_pairs<PAIRS>(w.a, w.b, wx, wy);
#pragma unroll
                for (int j = 0; j < 4; ++j) now.t[j] = weighed(t, j, rope.q_weight != nullptr, wx, wy);
            }
        }
        if (now.pos < 0) continue;
        uint4 u = ring.slot(k, i)[0], v = ring.slot(k, i)[32];
        norm_turn<D, PAIRS>(u, v, rope.q_weight != nullptr, rope.eps, [&](int j) { return now.t[j]; });
        if (head < list.q.heads) {
            uint4* out = list.q.out + (first + r) * list.q.out_stride + head * (D / 8);
            out[l.a] = u;
            out[l.b] = v;
        }
    }
}

// Rows of heads: a warp takes a row, or one of `parts` parts of its passes (512 / D heads each, queries
// first, then keys) when there are few rows.  Its lanes make the row's angles together (two each at most)
// and hand them round.  Few registers, so that many warps hide the two latencies (the position with the
// first passes, then the stores) that a row is.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(128, RMIN)
    qk_rope_kernel(se_rope rope, const int32_t* pos, int rows, int parts, HeadRows q, HeadRows k) {
    constexpr int HP = 512 / D, A = D / 64, U = RPASS;       // heads a pass, angles a lane, passes at once
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, mine = lane / (D / 16);
    const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int row = static_cast<int>(w / parts), part = static_cast<int>(w - (int64_t)row * parts);
    if (row >= rows) return;
    const HeadLane<D, PAIRS> l(lane, rope.rot_dim);
    const int nq = (q.heads + HP - 1) / HP, n = nq + (k.heads + HP - 1) / HP;
    const int p0 = n * part / parts, p1 = n * (part + 1) / parts;
    uint4 u[U], v[U];
    auto load = [&](int p) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const bool keys = p + i >= nq;
            const HeadRows& h = keys ? k : q;
            const int head = (p + i - (keys ? nq : 0)) * HP + mine;
            if (p + i < p1 && head < h.heads) {
                const uint4* in = h.in + row * h.in_stride + head * (D / 8);
                u[i] = in[l.a];
                v[i] = in[l.b];
            }
        }
    };
#pragma unroll
    for (int i = 0; i < U; ++i) u[i] = v[i] = make_uint4(0, 0, 0, 0);
    load(p0);
    const int at = pos[row];
    unsigned long long step[A];
#pragma unroll
    for (int i = 0; i < A; ++i)
        step[i] = A * lane + i < rope.rot_dim / 2 ? rope.turns[A * lane + i] : 0;
    if (at < 0) return;
    float ca[A], sa[A];
    Turn t;
#pragma unroll
    for (int i = 0; i < A; ++i) turn_of(step[i], rope.amplitude, at, ca[i], sa[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = __shfl_sync(0xffffffffu, ca[i % A], (8 * l.j + i) / A);
        const float y = __shfl_sync(0xffffffffu, sa[i % A], (8 * l.j + i) / A);
        t.c[i] = l.turns ? x : 1.f;
        t.s[i] = l.turns ? y : 0.f;
    }
    for (int p = p0; p < p1; p += U) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (p + i >= p1) break;                          // (the same for the whole warp)
            const bool keys = p + i >= nq;
            const void* weight = keys ? rope.k_weight : rope.q_weight;
            const Weight w = load_weight<D, PAIRS>(weight, l);
            norm_turn<D, PAIRS>(u[i], v[i], weight != nullptr, rope.eps, [&](int j) {
                uint64_t wx[4], wy[4];
                to_pairs<PAIRS>(w.a, w.b, wx, wy);           // (only the j-th are made)
                return weighed(t, j, weight != nullptr, wx, wy);
            });
            const HeadRows& h = keys ? k : q;
            const int head = (p + i - (keys ? nq : 0)) * HP + mine;
            if (head < h.heads) {
                uint4* out = h.out + row * h.out_stride + head * (D / 8);
                out[l.a] = u[i];
                out[l.b] = v[i];
            }
        }
        load(p + U);
    }
}

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

// Append of packed rows with the rotation in front.  Pieces as in the plain append: the keys of one sequence's
// rows in one page are the work of a warp for one KV head (512 / D rows side by side), which rotates
// them, writes them and folds them, as rounded, into the page's summary, which it owns.  The values of a
// piece are a unit of their own (32 registers of data either way); then every warp has its part of the
// rows' queries.
template <int D, bool PAIRS, bool TABLE>
__global__ void __launch_bounds__(128, AMIN)
    rope_append_chunk_kernel(se_paged_kv kv, se_rope rope, PassList list, const uint4* k_new,
                             const uint4* v_new, int64_t row_stride, se_chunk ck, int batch,
                             int* status) {
    constexpr int SEGS = D / 8, RP = 512 / D, IT = kPage / RP;
    static_assert(IT <= kPasses, "a piece is one unit");
    __shared__ __align__(16) float s_turns[TABLE ? kTable * D : 4];
    __shared__ uint4 s_ring[4 * kRingWords];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = lane / (D / 16);
    const int H = kv.num_kv_heads;
    const int first = static_cast<int>(blockIdx.x) * kRows;
    const HeadLane<D, PAIRS> l(lane, rope.rot_dim);
    const Ring ring = {s_ring + warp * kRingWords + lane};
    // a warp's units: its run of the queries' passes, then every nw-th of the pieces' keys and values
    const int w = warp + (blockDim.x >> 5) * blockIdx.y, nw = (blockDim.x >> 5) * gridDim.y;
    const int passes = min(kRows, ck.max_tokens - first) * list.n;
    const int p0 = passes * w / nw, p1 = passes * (w + 1) / nw, n_q = (p1 - p0 + kPasses - 1) / kPasses;
    auto copy_q = [&](int k) { copy_passes<D, PAIRS>(ring, k, list, first, p0 + k * kPasses, p1, l, mine); };
#pragma unroll
    for (int k = 0; k < kStages; ++k) {                      // (what needs no piece is on its way first)
        if (k < n_q) copy_q(k);
        if (k < n_q) cp_async_commit();
    }
    const Pieces pieces = find_pieces(kv, ck, batch, static_cast<int>(blockIdx.x), lane);
    if (pieces.row.bad && lane >= 1 && lane <= kPage && warp == 0 && blockIdx.y == 0)
        flag(status, SE_DEV_BAD_INDEX);
    if (warp == 0 && blockIdx.y == 0)
        commit_lengths(kv, ck, batch, pieces.t, lane, pieces.row);
    const int n_kv = __popc(pieces.lead) * H, back = nw - 1 - w;
    const int units = n_q + (2 * n_kv > back ? (2 * n_kv - back + nw - 1) / nw : 0);
    auto piece = [&](int k, bool& values, int& h) {
        const int u = back + (k - n_q) * nw;                 // keys of all pieces and heads, then values
        values = u >= n_kv;
        h = (values ? u - n_kv : u) % H;
        return piece_at(pieces, (values ? u - n_kv : u) / H, lane);
    };
    auto copy = [&](int k) {
        if (k < n_q) {
            copy_q(k);
        } else if (k < units) {
            bool values;
            int h;
            const Piece pc = piece(k, values, h);
            const uint4* in = (values ? v_new : k_new) + (int64_t)(first + pc.f - 1) * row_stride + h * SEGS;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = i * RP + mine;
                if ((pc.rows >> r) & 1) {
                    cp_async16(ring.slot(k, i), in + r * row_stride + l.a, 16);
                    cp_async16(ring.slot(k, i) + 32, in + r * row_stride + l.b, 16);
                }
            }
        }
        cp_async_commit();
    };
    for (int k = min(n_q, kStages); k < kStages; ++k) copy(k);
    Turns<D, PAIRS, TABLE> turns = {s_turns};
    if (TABLE) {
        // the block's 16 rows, and up to 15 behind them that its last piece reaches
        int reach = kRows;
        if (pieces.lead) {
            const Piece pc = piece_at(pieces, __popc(pieces.lead) - 1, lane);
            reach = max(reach, pc.f - 1 + 32 - __clz(pc.rows));
        }
        turns.make(rope, ck.pos, first, ck.max_tokens, min(reach, kTable));
    }
    uint4* K = static_cast<uint4*>(kv.k);
    uint4* V = static_cast<uint4*>(kv.v);
    uint4* M = static_cast<uint4*>(kv.meta);
    const Weight wk = load_weight<D, PAIRS>(rope.k_weight, l);
    {
        RowTurn now;
        for (int k = 0; k < n_q; ++k) {
            cp_async_wait<kStages - 1>();
            turn_passes<D, PAIRS, TABLE>(ring, k, list, ck.pos, first, p0 + k * kPasses, p1, l, mine, rope,
                                         turns, now);
            copy(k + kStages);
        }
    }
    for (int k = n_q; k < units; ++k) {
        bool values;
        int h;
        const Piece pc = piece(k, values, h);
        const int r0 = pc.f - 1, rows = 32 - __clz(pc.rows);  // the piece's first row in the block, its reach
        const int64_t dst =
            (((int64_t)(pc.slot0 / kPage) * H + h) * kPage + pc.slot0 % kPage) * SEGS;
        const int64_t m0 =
            ((((int64_t)pc.seq0 * kv.max_pages_per_seq + pc.pos0 / kPage) * H + h) * 2) * SEGS;
        constexpr uint32_t kNone = 0x7fff7fffu;              // NaNs: the other value is taken
        uint4 mn[2], mx[2], old[4];
        mn[0] = mn[1] = mx[0] = mx[1] = make_uint4(kNone, kNone, kNone, kNone);
        const bool more = pc.pos0 % kPage != 0;              // the page has a summary already
        if (!values && M != nullptr && more && mine == 0) {
            old[0] = M[m0 + l.a];
            old[1] = M[m0 + l.b];
            old[2] = M[m0 + SEGS + l.a];
            old[3] = M[m0 + SEGS + l.b];
        }
        cp_async_wait<kStages - 1>();
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = i * RP + mine;
            if (i * RP >= rows) break;                       // the same for the whole warp
            uint4 a = ring.slot(k, i)[0], b = ring.slot(k, i)[32];
            const bool there = (pc.rows >> r) & 1;
            if (!values) {
                Turn t;
                turns.get(rope, l, min(r0 + r, kTable - 1), pc.pos0 + r, t.c, t.s);
                norm_turn<D, PAIRS>(a, b, rope.k_weight != nullptr, rope.eps, [&](int j) {
                    uint64_t wx[4], wy[4];
                    to_pairs<PAIRS>(wk.a, wk.b, wx, wy);     // (only the j-th are made)
                    return weighed(t, j, rope.k_weight != nullptr, wx, wy);
                });
                if (there) {
                    fold(mn[0], mx[0], a, a);
                    fold(mn[1], mx[1], b, b);
                }
            }
            if (there) {
                uint4* out = (values ? V : K) + dst + r * SEGS;
                out[l.a] = a;
                out[l.b] = b;
            }
        }
        copy(k + kStages);
        if (values || M == nullptr) continue;
#pragma unroll
        for (int o = D / 16; o < 32; o <<= 1)
#pragma unroll
            for (int g = 0; g < 2; ++g)
                fold(mn[g], mx[g], shfl_xor4(mn[g], o), shfl_xor4(mx[g], o));
        if (mine == 0) {
            if (more) {
                fold(mn[0], mx[0], old[0], old[2]);
                fold(mn[1], mx[1], old[1], old[3]);
            }
            M[m0 + l.a] = mn[0];
            M[m0 + l.b] = mn[1];
            M[m0 + SEGS + l.a] = mx[0];
            M[m0 + SEGS + l.b] = mx[1];
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
    const int64_t warps = (int64_t)rows * parts;
    return launch_pdl(qk_rope_kernel<D, PAIRS>, dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0,
                      s, rope, pos, rows, parts, head_rows(q), head_rows(k));
}

template <int D, bool PAIRS>
cudaError_t append_of(const se_paged_kv& kv, const se_rope& rope, const HeadArgs& q, const void* k_new,
                      const void* v_new, int64_t row_stride, const se_chunk& ck, int batch, int* status,
                      cudaStream_t s) {
    const int groups = (ck.max_tokens + kRows - 1) / kRows;
    if (groups == 0) return cudaSuccess;
    constexpr int HP = 512 / D;
    PassList list = {head_rows(q), (q.heads + HP - 1) / HP, 0};
    if (list.n > 1) list.inverse = static_cast<uint32_t>(((1ull << 32) + list.n - 1) / list.n);
    const uint4* k = static_cast<const uint4*>(k_new);
    const uint4* v = static_cast<const uint4*>(v_new);
    // few rows: several blocks share 16 of them, down to one unit (a piece's keys of a head, a pass) a warp
    if (groups < num_sms()) {
        const int most = kRows * (2 * kv.num_kv_heads + list.n);
        const int share = std::max(1, std::min(8 * num_sms() / groups, (most + 3) / 4));
        return launch_pdl(rope_append_chunk_kernel<D, PAIRS, false>, dim3(groups, share), dim3(128), 0, s,
                          kv, rope, list, k, v, row_stride / 8, ck, batch, status);
    }
    return launch_pdl(rope_append_chunk_kernel<D, PAIRS, true>, dim3(groups), dim3(128), 0, s, kv, rope,
                      list, k, v, row_stride / 8, ck, batch, status);
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
    if (kv.head_dim == 128)
        return pairs ? append_of<128, true>(kv, rope, q, k_new, v_new, row_stride, ck, batch, status, s)
                     : append_of<128, false>(kv, rope, q, k_new, v_new, row_stride, ck, batch, status, s);
    return pairs ? append_of<64, true>(kv, rope, q, k_new, v_new, row_stride, ck, batch, status, s)
                 : append_of<64, false>(kv, rope, q, k_new, v_new, row_stride, ck, batch, status, s);
}

}  // namespace se
