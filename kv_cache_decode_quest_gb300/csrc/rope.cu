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
#include <math_constants.h>

#include <algorithm>

#include "append.cuh"
#include "chunk_rows.cuh"
#include "common.cuh"
#include "internal.h"

namespace se {
namespace {

// The lane's place in a head of D channels: its two vectors, and whether it rotates.
template <int D>
struct HeadLane {
    int j, a, b;
    bool turns;
    __device__ HeadLane(int lane, int rot, int layout) {
        constexpr int L = D / 16;
        j = lane % L;
        const int r = rot / 16;                          // lanes that rotate
        turns = j < r;
        if (layout == SE_ROPE_PAIRS) {
            a = 2 * j;
            b = 2 * j + 1;
        } else {
            a = turns ? j : 2 * r + 2 * (j - r);
            b = turns ? j + r : a + 1;
        }
    }
};

// Pairs (x, y) of two vectors: of halves, channel i of one and of the other; of pairs, channels
// 2i and 2i + 1 of the two as one run.
__device__ __forceinline__ void to_pairs(uint4 u, uint4 v, bool pairs, float* x, float* y) {
    const Bf8 p = unpack8(u), q = unpack8(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float lo = i < 4 ? p.x[(2 * i) & 7] : q.x[(2 * i) & 7];
        const float hi = i < 4 ? p.x[(2 * i + 1) & 7] : q.x[(2 * i + 1) & 7];
        x[i] = pairs ? lo : p.x[i];
        y[i] = pairs ? hi : q.x[i];
    }
}
__device__ __forceinline__ void from_pairs(const float* x, const float* y, bool pairs, uint4& u,
                                           uint4& v) {
    Bf8 p, q;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p.x[i] = pairs ? (i & 1 ? y[i >> 1] : x[i >> 1]) : x[i];
        q.x[i] = pairs ? (i & 1 ? y[4 + (i >> 1)] : x[4 + (i >> 1)]) : y[i];
    }
    u = pack8(p);
    v = pack8(q);
}

// Cosine and sine of pair i at position pos, times the amplitude.
__device__ __forceinline__ void turn_of(unsigned long long turns, int pos, float amp, float& c,
                                        float& s) {
    const unsigned long long t = static_cast<unsigned long long>(static_cast<uint32_t>(pos)) * turns;
    const float half_turns = static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f;
    sincospif(half_turns, &s, &c);
    c *= amp;
    s *= amp;
}

// One head's 8 pairs of this lane: normed over the D / 16 lanes of the head, weighted, rotated.
template <int D>
__device__ __forceinline__ void norm_turn(float* x, float* y, bool norm, const float* wx,
                                          const float* wy, float eps, const float* c,
                                          const float* s) {
    if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
        for (int o = 1; o < D / 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(fmaf(ss, 1.0f / D, eps));
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
}

template <int D>
__device__ __forceinline__ void load_weight(const void* w, const HeadLane<D>& l, bool pairs, float* wx,
                                            float* wy) {
    if (w == nullptr) return;
    const uint4* v = static_cast<const uint4*>(w);
    to_pairs(v[l.a], v[l.b], pairs, wx, wy);
}

struct HeadRows {
    const uint4* in;
    uint4* out;
    int64_t in_stride, out_stride;      // 16-byte vectors between tokens
    int heads;
};

// Heads [h0, h1) of one row, 512 / D side by side, U passes' loads in flight.
template <int D>
__device__ __forceinline__ void turn_heads(const HeadRows& r, int64_t row, int h0, int h1,
                                           const HeadLane<D>& l, int lane, bool pairs, bool norm,
                                           const float* wx, const float* wy, float eps,
                                           const float* c, const float* s) {
    constexpr int HP = 512 / D, SEGS = D / 8, U = 4;
    const uint4* in = r.in + row * r.in_stride;
    uint4* out = r.out + row * r.out_stride;
    const int mine = lane / (D / 16);
    for (int h = h0; h < h1; h += U * HP) {
        uint4 u[U], v[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int at = h + i * HP + mine;
            if (at < h1) {
                u[i] = in[at * SEGS + l.a];
                v[i] = in[at * SEGS + l.b];
            } else {
                u[i] = v[i] = make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (h + i * HP >= h1) break;                     // the same for the whole warp
            const int at = h + i * HP + mine;
            float x[8], y[8];
            to_pairs(u[i], v[i], pairs, x, y);
            norm_turn<D>(x, y, norm, wx, wy, eps, c, s);
            uint4 p, q;
            from_pairs(x, y, pairs, p, q);
            if (at < h1) {
                out[at * SEGS + l.a] = p;
                out[at * SEGS + l.b] = q;
            }
        }
    }
}

// A warp takes a row, or one of `parts` parts of its heads when there are few rows.
template <int D>
__global__ void __launch_bounds__(128)
    qk_rope_kernel(se_rope rope, const int32_t* pos, int rows, int parts, HeadRows q, HeadRows k) {
    pdl_wait();
    pdl_trigger();
    constexpr int HP = 512 / D;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int row = static_cast<int>(w / parts), part = static_cast<int>(w % parts);
    if (row >= rows) return;
    const int at = pos[row];
    if (at < 0) return;
    const bool pairs = rope.layout == SE_ROPE_PAIRS;
    const HeadLane<D> l(lane, rope.rot_dim, rope.layout);
    float c[8], s[8], wx[8], wy[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
        if (l.turns)
            turn_of(reinterpret_cast<const unsigned long long*>(rope.turns)[8 * l.j + i], at,
                    rope.amplitude, c[i], s[i]);
    }
    // passes of HP heads: queries first, then keys
    const int nq = (q.heads + HP - 1) / HP, n = nq + (k.heads + HP - 1) / HP;
    const int p0 = static_cast<int>((int64_t)n * part / parts);
    const int p1 = static_cast<int>((int64_t)n * (part + 1) / parts);
    if (p0 < nq) {
        load_weight<D>(rope.q_weight, l, pairs, wx, wy);
        turn_heads<D>(q, row, p0 * HP, min(q.heads, p1 * HP), l, lane, pairs,
                      rope.q_weight != nullptr, wx, wy, rope.eps, c, s);
    }
    if (p1 > nq) {
        load_weight<D>(rope.k_weight, l, pairs, wx, wy);
        turn_heads<D>(k, row, (max(p0, nq) - nq) * HP, min(k.heads, (p1 - nq) * HP), l, lane, pairs,
                      rope.k_weight != nullptr, wx, wy, rope.eps, c, s);
    }
}

// Append of packed rows with the rotation in front.  Pieces as in the plain append: a warp takes the
// rows of one sequence in one page for one KV head (512 / D rows side by side), rotates the keys,
// writes keys and values and folds the rounded keys into the page's summary, which it owns.  The block's
// other units are its rows' queries.  The cosines of the block's 16 rows are made once, in shared
// memory.
template <int D>
__global__ void __launch_bounds__(128)
    rope_append_chunk_kernel(se_paged_kv kv, se_rope rope, HeadRows q, const uint4* k_new,
                             const uint4* v_new, int64_t row_stride, se_chunk ck, int batch, int parts,
                             int* status) {
    constexpr int SEGS = D / 8, RP = 512 / D, IT = kPage / RP, HALF = D / 2;
    __shared__ __align__(16) float s_cos[kPage * 2 - 1][HALF], s_sin[kPage * 2 - 1][HALF];
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
    // a piece that begins in the block's 16 rows may reach 15 rows past them
    const int half = rope.rot_dim / 2;
    for (int i = threadIdx.x; i < (2 * kPage - 1) * half; i += blockDim.x) {
        const int r = i / half, at = first + r < ck.max_tokens ? ck.pos[first + r] : -1;
        float c = 1.f, s = 0.f;
        if (at >= 0)
            turn_of(reinterpret_cast<const unsigned long long*>(rope.turns)[i % half], at,
                    rope.amplitude, c, s);
        s_cos[r][i % half] = c;
        s_sin[r][i % half] = s;
    }
    __syncthreads();
    const bool pairs = rope.layout == SE_ROPE_PAIRS;
    const HeadLane<D> l(lane, rope.rot_dim, rope.layout);
    float c[8], s[8], wx[8], wy[8];
    auto load_turns = [&](int r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = l.turns ? s_cos[r][8 * l.j + i] : 1.f;
            s[i] = l.turns ? s_sin[r][8 * l.j + i] : 0.f;
        }
    };
    const int rp = lane / (D / 16);
    uint4* K = static_cast<uint4*>(kv.k);
    uint4* V = static_cast<uint4*>(kv.v);
    uint4* M = static_cast<uint4*>(kv.meta);
    const int n_kv = __popc(pieces.lead) * H, n_q = q.heads > 0 ? kPage * parts : 0;
    const int nw = (blockDim.x >> 5) * gridDim.y;
    for (int u = warp + (blockDim.x >> 5) * blockIdx.y; u < n_kv + n_q; u += nw) {
        if (u >= n_kv) {
            const int r = (u - n_kv) / parts, part = (u - n_kv) % parts, t = first + r;
            if (t >= ck.max_tokens || ck.pos[t] < 0) continue;
            const int n = (q.heads + RP - 1) / RP;
            const int p0 = n * part / parts, p1 = n * (part + 1) / parts;
            load_turns(r);
            load_weight<D>(rope.q_weight, l, pairs, wx, wy);
            turn_heads<D>(q, t, p0 * RP, min(q.heads, p1 * RP), l, lane, pairs,
                          rope.q_weight != nullptr, wx, wy, rope.eps, c, s);
            continue;
        }
        const int h = u % H;
        const Piece pc = piece_at(pieces, u / H, lane);
        const int r0 = pc.f - 1;                             // the piece's first row in the block
        const int64_t src = (int64_t)(first + r0) * row_stride + h * SEGS;
        uint4 ka[IT], kb[IT], va[IT], vb[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = i * RP + rp;
            ka[i] = kb[i] = make_uint4(0, 0, 0, 0);
            if ((pc.rows >> r) & 1) {
                ka[i] = k_new[src + r * row_stride + l.a];
                kb[i] = k_new[src + r * row_stride + l.b];
                va[i] = v_new[src + r * row_stride + l.a];
                vb[i] = v_new[src + r * row_stride + l.b];
            }
        }
        const int64_t m0 =
            ((((int64_t)pc.seq0 * kv.max_pages_per_seq + pc.pos0 / kPage) * H + h) * 2) * SEGS;
        const bool fold = pc.pos0 % kPage != 0;
        load_weight<D>(rope.k_weight, l, pairs, wx, wy);
        const int64_t dst =
            (((int64_t)(pc.slot0 / kPage) * H + h) * kPage + pc.slot0 % kPage) * SEGS;
        Bf8 mn[2], mx[2];
#pragma unroll
        for (int e = 0; e < 8; ++e)              // none yet: min and max pass a NaN over
            mn[0].x[e] = mx[0].x[e] = mn[1].x[e] = mx[1].x[e] = CUDART_NAN_F;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = i * RP + rp;
            if (i * RP >= 32 - __clz(pc.rows)) break;        // the same for the whole warp
            const bool there = (pc.rows >> r) & 1;
            load_turns(min(r0 + r, 2 * kPage - 2));
            float x[8], y[8];
            to_pairs(ka[i], kb[i], pairs, x, y);
            norm_turn<D>(x, y, rope.k_weight != nullptr, wx, wy, rope.eps, c, s);
            uint4 p, p2;
            from_pairs(x, y, pairs, p, p2);
            if (there) {
                K[dst + r * SEGS + l.a] = p;
                K[dst + r * SEGS + l.b] = p2;
                V[dst + r * SEGS + l.a] = va[i];
                V[dst + r * SEGS + l.b] = vb[i];
                const Bf8 f[2] = {unpack8(p), unpack8(p2)};
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        mn[g].x[e] = fminf(mn[g].x[e], f[g].x[e]);
                        mx[g].x[e] = fmaxf(mx[g].x[e], f[g].x[e]);
                    }
            }
        }
        if (M == nullptr) continue;
#pragma unroll
        for (int o = D / 16; o < 32; o <<= 1)
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    mn[g].x[e] = fminf(mn[g].x[e], __shfl_xor_sync(0xffffffffu, mn[g].x[e], o));
                    mx[g].x[e] = fmaxf(mx[g].x[e], __shfl_xor_sync(0xffffffffu, mx[g].x[e], o));
                }
        if (rp == 0) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int64_t at = m0 + (g ? l.b : l.a);
                if (fold) {
                    const Bf8 a = unpack8(M[at]), b = unpack8(M[at + SEGS]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        mn[g].x[e] = fminf(a.x[e], mn[g].x[e]);
                        mx[g].x[e] = fmaxf(b.x[e], mx[g].x[e]);
                    }
                }
                M[at] = pack8(mn[g]);
                M[at + SEGS] = pack8(mx[g]);
            }
        }
    }
}

HeadRows head_rows(const HeadArgs& a) {
    return HeadRows{static_cast<const uint4*>(a.in), static_cast<uint4*>(a.out), a.in_stride / 8,
                    a.out_stride / 8, a.heads};
}

}  // namespace

cudaError_t launch_qk_rope(const se_rope& rope, const int32_t* pos, int rows, int head_dim,
                           const HeadArgs& q, const HeadArgs& k, cudaStream_t s) {
    const int hp = 512 / head_dim;
    const int passes = (q.heads + hp - 1) / hp + (k.heads + hp - 1) / hp;
    if (rows == 0 || passes == 0) return cudaSuccess;
    // few rows: their heads are spread over warps until the GPU has four a scheduler
    const int parts = std::max(1, std::min(passes, 16 * num_sms() / rows));
    const int64_t warps = (int64_t)rows * parts;
    const dim3 grid(static_cast<unsigned>((warps + 3) / 4));
    if (head_dim == 128)
        return launch_pdl(qk_rope_kernel<128>, grid, dim3(128), 0, s, rope, pos, rows, parts,
                          head_rows(q), head_rows(k));
    return launch_pdl(qk_rope_kernel<64>, grid, dim3(128), 0, s, rope, pos, rows, parts, head_rows(q),
                      head_rows(k));
}

cudaError_t launch_rope_append_chunk(const se_paged_kv& kv, const se_rope& rope, const HeadArgs& q,
                                     const void* k_new, const void* v_new, int64_t row_stride,
                                     const se_chunk& ck, int batch, int* status, cudaStream_t s) {
    const int blocks = (ck.max_tokens + kPage - 1) / kPage;
    if (blocks == 0) return cudaSuccess;
    // few rows: more blocks share one group of 16, down to one unit a warp
    const int hp = 512 / kv.head_dim, passes = std::max(1, (q.heads + hp - 1) / hp);
    const int parts = std::max(1, std::min(passes, num_sms() / blocks));
    const int most = kPage * (kv.num_kv_heads + (q.heads > 0 ? parts : 0));
    const int share = std::max(1, std::min(4 * num_sms() / blocks, (most + 3) / 4));
    const dim3 grid(blocks, share);
    const uint4* k = static_cast<const uint4*>(k_new);
    const uint4* v = static_cast<const uint4*>(v_new);
    if (kv.head_dim == 128)
        return launch_pdl(rope_append_chunk_kernel<128>, grid, dim3(128), 0, s, kv, rope,
                          head_rows(q), k, v, row_stride / 8, ck, batch, parts, status);
    return launch_pdl(rope_append_chunk_kernel<64>, grid, dim3(128), 0, s, kv, rope, head_rows(q), k,
                      v, row_stride / 8, ck, batch, parts, status);
}

}  // namespace se
