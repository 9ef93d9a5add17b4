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

// Pairs (x, y) of two vectors: of halves, channel i of one and of the other; of pairs, channels
// 2i and 2i + 1 of the two as one run.
template <bool PAIRS>
__device__ __forceinline__ void to_pairs(uint4 u, uint4 v, float* x, float* y) {
    const Bf8 p = unpack8(u), q = unpack8(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = !PAIRS ? p.x[i] : i < 4 ? p.x[(2 * i) & 7] : q.x[(2 * i) & 7];
        y[i] = !PAIRS ? q.x[i] : i < 4 ? p.x[(2 * i + 1) & 7] : q.x[(2 * i + 1) & 7];
    }
}
template <bool PAIRS>
__device__ __forceinline__ void from_pairs(const float* x, const float* y, uint4& u, uint4& v) {
    Bf8 p, q;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p.x[i] = !PAIRS ? x[i] : i & 1 ? y[i >> 1] : x[i >> 1];
        q.x[i] = !PAIRS ? y[i] : i & 1 ? y[4 + (i >> 1)] : x[4 + (i >> 1)];
    }
    u = pack8(p);
    v = pack8(q);
}

// Cosine and sine of one pair's angle at position pos, times the amplitude.
__device__ __forceinline__ void turn_of(const se_rope& rope, int i, int pos, float& c, float& s) {
    const unsigned long long t = static_cast<unsigned long long>(static_cast<uint32_t>(pos)) *
                                 static_cast<unsigned long long>(rope.turns[i]);
    const float half_turns = static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f;
    sincospif(half_turns, &s, &c);
    c *= rope.amplitude;
    s *= rope.amplitude;
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

// One head's two vectors of this lane: normed over the head's D / 16 lanes, weighted, rotated, rounded.
template <int D, bool PAIRS>
__device__ __forceinline__ void norm_turn(uint4& u, uint4& v, bool norm, const Weight& w, float eps,
                                          const float* c, const float* s) {
    float x[8], y[8];
    to_pairs<PAIRS>(u, v, x, y);
    if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
        for (int o = 1; o < D / 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(fmaf(ss, 1.0f / D, eps));
        float wx[8], wy[8];
        to_pairs<PAIRS>(w.a, w.b, wx, wy);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = x[i] * inv * wx[i];
            y[i] = y[i] * inv * wy[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = x[i], b = y[i];
        x[i] = fmaf(a, c[i], -b * s[i]);
        y[i] = fmaf(b, c[i], a * s[i]);
    }
    from_pairs<PAIRS>(x, y, u, v);
}

struct HeadRows {
    const uint4* in;
    uint4* out;
    int64_t in_stride, out_stride;      // 16-byte vectors between tokens
    int heads;
};

constexpr int kPasses = 4;               // passes of heads whose loads are in flight together

// The vectors of kPasses passes (512 / D heads each, side by side) of one row: passes [0, nq) are
// queries, those behind them keys; places past the heads, or past pass p1, get zeros.
template <int D, bool PAIRS>
__device__ __forceinline__ void load_passes(const HeadRows& q, const HeadRows& k, int64_t row, int p,
                                            int p1, int nq, const HeadLane<D, PAIRS>& l, int mine,
                                            uint4* u, uint4* v) {
    constexpr int HP = 512 / D, SEGS = D / 8;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const bool keys = p + i >= nq;
        const HeadRows& r = keys ? k : q;
        const int h = (p + i - (keys ? nq : 0)) * HP + mine;
        u[i] = v[i] = make_uint4(0, 0, 0, 0);
        if (p + i < p1 && h < r.heads) {
            const uint4* in = r.in + row * r.in_stride + h * SEGS;
            u[i] = in[l.a];
            v[i] = in[l.b];
        }
    }
}
template <int D, bool PAIRS>
__device__ __forceinline__ void turn_passes(const HeadRows& q, const HeadRows& k, int64_t row, int p,
                                            int p1, int nq, const HeadLane<D, PAIRS>& l, int mine,
                                            uint4* u, uint4* v, const se_rope& rope,
                                            const Weight& wq, const Weight& wk, const float* c,
                                            const float* s) {
    constexpr int HP = 512 / D, SEGS = D / 8;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        if (p + i >= p1) break;                          // the same for the whole warp
        const bool keys = p + i >= nq;
        const HeadRows& r = keys ? k : q;
        const int h = (p + i - (keys ? nq : 0)) * HP + mine;
        norm_turn<D, PAIRS>(u[i], v[i], (keys ? rope.k_weight : rope.q_weight) != nullptr,
                            keys ? wk : wq, rope.eps, c, s);
        if (h < r.heads) {
            uint4* out = r.out + row * r.out_stride + h * SEGS;
            out[l.a] = u[i];
            out[l.b] = v[i];
        }
    }
}

// A warp takes a row, or one of `parts` parts of its heads when there are few rows.  Its lanes make the
// row's angles together (two each at most) and hand them round.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(128)
    qk_rope_kernel(se_rope rope, const int32_t* pos, int rows, int parts, HeadRows q, HeadRows k) {
    pdl_wait();
    pdl_trigger();
    constexpr int HP = 512 / D, A = D / 64;              // angles a lane
    const int lane = threadIdx.x & 31, mine = lane / (D / 16);
    const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int row = static_cast<int>(w / parts), part = static_cast<int>(w % parts);
    if (row >= rows) return;
    const HeadLane<D, PAIRS> l(lane, rope.rot_dim);
    const int nq = (q.heads + HP - 1) / HP, n = nq + (k.heads + HP - 1) / HP;
    const int p0 = static_cast<int>((int64_t)n * part / parts);
    const int p1 = static_cast<int>((int64_t)n * (part + 1) / parts);
    uint4 u[kPasses], v[kPasses];
    load_passes<D, PAIRS>(q, k, row, p0, p1, nq, l, mine, u, v);
    const Weight wq = load_weight<D, PAIRS>(rope.q_weight, l), wk = load_weight<D, PAIRS>(rope.k_weight, l);
    const int at = pos[row];
    if (at < 0) return;
    float ca[A], sa[A], c[8], s[8];
#pragma unroll
    for (int i = 0; i < A; ++i) {
        ca[i] = 1.f;
        sa[i] = 0.f;
        if (A * lane + i < rope.rot_dim / 2) turn_of(rope, A * lane + i, at, ca[i], sa[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = __shfl_sync(0xffffffffu, ca[i % A], (8 * l.j + i) / A);
        const float y = __shfl_sync(0xffffffffu, sa[i % A], (8 * l.j + i) / A);
        c[i] = l.turns ? x : 1.f;
        s[i] = l.turns ? y : 0.f;
    }
    turn_passes<D, PAIRS>(q, k, row, p0, p1, nq, l, mine, u, v, rope, wq, wk, c, s);
    for (int p = p0 + kPasses; p < p1; p += kPasses) {
        load_passes<D, PAIRS>(q, k, row, p, p1, nq, l, mine, u, v);
        turn_passes<D, PAIRS>(q, k, row, p, p1, nq, l, mine, u, v, rope, wq, wk, c, s);
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
// piece, and a row's queries (or a part of them), are units of their own: a unit then holds 32 registers of
// data, and warps find work of about one size.  The cosines of the block's rows are made once, in shared memory.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(128)
    rope_append_chunk_kernel(se_paged_kv kv, se_rope rope, HeadRows q, const uint4* k_new,
                             const uint4* v_new, int64_t row_stride, se_chunk ck, int batch, int parts,
                             int* status) {
    constexpr int SEGS = D / 8, RP = 512 / D, IT = kPage / RP, HALF = D / 2, TABLE = 2 * kPage - 1;
    __shared__ __align__(16) float s_cos[TABLE][HALF], s_sin[TABLE][HALF];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int H = kv.num_kv_heads;
    const int first = static_cast<int>(blockIdx.x) * kPage;
    const Pieces pieces = find_pieces(kv, ck, batch, static_cast<int>(blockIdx.x), lane);
    if (pieces.row.bad && lane >= 1 && lane <= kPage && warp == 0 && blockIdx.y == 0)
        flag(status, SE_DEV_BAD_INDEX);
    if (warp == 0 && blockIdx.y == 0)
        commit_lengths(kv, ck, batch, pieces.t, lane, pieces.row);
    // the block's 16 rows, and up to 15 behind them that a piece of theirs reaches
    int reach = kPage;
    if (pieces.lead) {
        const Piece pc = piece_at(pieces, __popc(pieces.lead) - 1, lane);
        reach = max(reach, pc.f - 1 + 32 - __clz(pc.rows));
    }
    const int half = rope.rot_dim / 2;
    for (int i = threadIdx.x; i < reach * half; i += blockDim.x) {
        const int r = i / half, a = i - r * half, at = first + r < ck.max_tokens ? ck.pos[first + r] : -1;
        float c = 1.f, s = 0.f;
        if (at >= 0) turn_of(rope, a, at, c, s);
        s_cos[r][a] = c;
        s_sin[r][a] = s;
    }
    __syncthreads();
    const HeadLane<D, PAIRS> l(lane, rope.rot_dim);
    const int mine = lane / (D / 16);
    float c[8], s[8];
    auto load_turns = [&](int r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = l.turns ? s_cos[r][8 * l.j + i] : 1.f;
            s[i] = l.turns ? s_sin[r][8 * l.j + i] : 0.f;
        }
    };
    uint4* K = static_cast<uint4*>(kv.k);
    uint4* V = static_cast<uint4*>(kv.v);
    uint4* M = static_cast<uint4*>(kv.meta);
    const int n_kv = __popc(pieces.lead) * H, n_q = q.heads > 0 ? kPage * parts : 0;
    const int nw = (blockDim.x >> 5) * gridDim.y;
    for (int u = warp + (blockDim.x >> 5) * blockIdx.y; u < 2 * n_kv + n_q; u += nw) {
        if (u >= 2 * n_kv) {
            const int r = (u - 2 * n_kv) / parts, part = (u - 2 * n_kv) % parts, t = first + r;
            if (t >= ck.max_tokens || ck.pos[t] < 0) continue;
            const int n = (q.heads + RP - 1) / RP;
            const int p0 = n * part / parts, p1 = n * (part + 1) / parts;
            const Weight w = load_weight<D, PAIRS>(rope.q_weight, l);
            load_turns(r);
            for (int p = p0; p < p1; p += kPasses) {
                uint4 x[kPasses], y[kPasses];
                load_passes<D, PAIRS>(q, q, t, p, p1, n, l, mine, x, y);
                turn_passes<D, PAIRS>(q, q, t, p, p1, n, l, mine, x, y, rope, w, w, c, s);
            }
            continue;
        }
        const bool values = u >= n_kv;
        const int h = (values ? u - n_kv : u) % H;
        const Piece pc = piece_at(pieces, (values ? u - n_kv : u) / H, lane);
        const int r0 = pc.f - 1;                             // the piece's first row in the block
        const int64_t src = (int64_t)(first + r0) * row_stride + h * SEGS;
        const int64_t dst =
            (((int64_t)(pc.slot0 / kPage) * H + h) * kPage + pc.slot0 % kPage) * SEGS;
        uint4 a[IT], b[IT];
        const uint4* in = values ? v_new : k_new;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = i * RP + mine;
            a[i] = b[i] = make_uint4(0, 0, 0, 0);
            if ((pc.rows >> r) & 1) {
                a[i] = in[src + r * row_stride + l.a];
                b[i] = in[src + r * row_stride + l.b];
            }
        }
        if (values) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = i * RP + mine;
                if ((pc.rows >> r) & 1) {
                    V[dst + r * SEGS + l.a] = a[i];
                    V[dst + r * SEGS + l.b] = b[i];
                }
            }
            continue;
        }
        const int64_t m0 =
            ((((int64_t)pc.seq0 * kv.max_pages_per_seq + pc.pos0 / kPage) * H + h) * 2) * SEGS;
        const Weight w = load_weight<D, PAIRS>(rope.k_weight, l);
        constexpr uint32_t kNone = 0x7fff7fffu;              // NaNs: the other value is taken
        uint4 mn[2], mx[2];
        mn[0] = mn[1] = mx[0] = mx[1] = make_uint4(kNone, kNone, kNone, kNone);
        if (M != nullptr && pc.pos0 % kPage != 0 && mine == 0) {
            mn[0] = M[m0 + l.a];
            mn[1] = M[m0 + l.b];
            mx[0] = M[m0 + SEGS + l.a];
            mx[1] = M[m0 + SEGS + l.b];
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = i * RP + mine;
            if (i * RP >= 32 - __clz(pc.rows)) break;        // the same for the whole warp
            load_turns(min(r0 + r, TABLE - 1));
            norm_turn<D, PAIRS>(a[i], b[i], rope.k_weight != nullptr, w, rope.eps, c, s);
            if ((pc.rows >> r) & 1) {
                K[dst + r * SEGS + l.a] = a[i];
                K[dst + r * SEGS + l.b] = b[i];
                fold(mn[0], mx[0], a[i], a[i]);
                fold(mn[1], mx[1], b[i], b[i]);
            }
        }
        if (M == nullptr) continue;
#pragma unroll
        for (int o = D / 16; o < 32; o <<= 1)
#pragma unroll
            for (int g = 0; g < 2; ++g)
                fold(mn[g], mx[g], shfl_xor4(mn[g], o), shfl_xor4(mx[g], o));
        if (mine == 0) {
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

}  // namespace

template <int D, bool PAIRS>
static cudaError_t launch_rows(const se_rope& rope, const int32_t* pos, int rows, const HeadArgs& q,
                               const HeadArgs& k, cudaStream_t s) {
    constexpr int HP = 512 / D;
    const int passes = (q.heads + HP - 1) / HP + (k.heads + HP - 1) / HP;
    if (rows == 0 || passes == 0) return cudaSuccess;
    // few rows: their heads are spread over warps until the GPU has four a scheduler
    const int parts = std::max(1, std::min(passes, 16 * num_sms() / rows));
    const int64_t warps = (int64_t)rows * parts;
    return launch_pdl(qk_rope_kernel<D, PAIRS>, dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0,
                      s, rope, pos, rows, parts, head_rows(q), head_rows(k));
}

cudaError_t launch_qk_rope(const se_rope& rope, const int32_t* pos, int rows, int head_dim,
                           const HeadArgs& q, const HeadArgs& k, cudaStream_t s) {
    const bool pairs = rope.layout == SE_ROPE_PAIRS;
    if (head_dim == 128)
        return pairs ? launch_rows<128, true>(rope, pos, rows, q, k, s)
                     : launch_rows<128, false>(rope, pos, rows, q, k, s);
    return pairs ? launch_rows<64, true>(rope, pos, rows, q, k, s)
                 : launch_rows<64, false>(rope, pos, rows, q, k, s);
}

template <int D, bool PAIRS>
static cudaError_t launch_append(const se_paged_kv& kv, const se_rope& rope, const HeadArgs& q,
                                 const void* k_new, const void* v_new, int64_t row_stride,
                                 const se_chunk& ck, int batch, int* status, cudaStream_t s) {
    const int blocks = (ck.max_tokens + kPage - 1) / kPage;
    if (blocks == 0) return cudaSuccess;
    // few rows: more blocks share one group of 16, down to one unit a warp
    constexpr int HP = 512 / D;
    const int passes = std::max(1, (q.heads + HP - 1) / HP);
    const int parts = std::max(1, std::min(passes, num_sms() / blocks));
    const int most = kPage * (2 * kv.num_kv_heads + (q.heads > 0 ? parts : 0));
    const int share = std::max(1, std::min(4 * num_sms() / blocks, (most + 3) / 4));
    return launch_pdl(rope_append_chunk_kernel<D, PAIRS>, dim3(blocks, share), dim3(128), 0, s, kv, rope,
                      head_rows(q), static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new),
                      row_stride / 8, ck, batch, parts, status);
}

cudaError_t launch_rope_append_chunk(const se_paged_kv& kv, const se_rope& rope, const HeadArgs& q,
                                     const void* k_new, const void* v_new, int64_t row_stride,
                                     const se_chunk& ck, int batch, int* status, cudaStream_t s) {
    const bool pairs = rope.layout == SE_ROPE_PAIRS;
    if (kv.head_dim == 128)
        return pairs ? launch_append<128, true>(kv, rope, q, k_new, v_new, row_stride, ck, batch, status, s)
                     : launch_append<128, false>(kv, rope, q, k_new, v_new, row_stride, ck, batch, status,
                                                 s);
    return pairs ? launch_append<64, true>(kv, rope, q, k_new, v_new, row_stride, ck, batch, status, s)
                 : launch_append<64, false>(kv, rope, q, k_new, v_new, row_stride, ck, batch, status, s);
}

}  // namespace se
