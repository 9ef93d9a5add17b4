// Drafted tokens against the target's probabilities (se_draft_verify): which of them stay,
// and the token that is drawn behind them.  Draft d with u q(d) < p(d) stays; behind the
// first refused one the next token comes from max(0, p - q), which leaves every token
// distributed as p.
//
// One row of the vocabulary per sequence is read (two where a draft was refused): HBM
// bound, a sum and a search.  A draw compares a running sum of up to millions of weights
// with a random part of the whole: sums in fp32 would move it over a border in about one of
// 30 draws over 128K tokens.  So a weight is p - q with its rounding error beside it (exact
// together), a lane's sum of 32 weights carries its error in a second word, and from there
// on sums are integers in units of 2^-58, the same in any order: the row is cut into tiles
// of 1024 that any warp of any block may sum, and the last block of a sequence finds the
// tile and in it the token.  Two weights at once in packed fp32: 5 operations a weight of p
// alone, 9 with q (one by one 41.4 us for the 39.9 below).  A row whose weights come to little
// (hardly any is left of p beside q, or the row is no distribution) would lose them below those
// units: its last block makes the sums again, with the weights scaled by a power of two.
// Up to eight blocks of a sequence are a cluster, whose first block gets the sums in shared
// memory; more (a large vocabulary, few sequences) meet over a counter in memory (one
// sequence of 32,000 tokens: 0.8 us more).
// 256 sequences over 131,072 tokens (about 1.6 rows each) take 39.9 us, 5.3 TB/s: 78% of the
// copy rate; the rest is three latencies before a block knows its row, blocks with two rows
// beside blocks with one, and the last sequences' search.  In bf16 1.5 rows each take 34.6 us,
// one of p alone 25.4: instructions a weight, not bytes.  Every weight made a 64-bit integer 122
// us; two waves of blocks 52; rows through a ring in shared memory 4 us more.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace se {
namespace {

constexpr int kTile = 1024;                  // weights of a tile
constexpr int kMaxBatch = 8192;
constexpr size_t kSumsAt = 256 + kMaxBatch * sizeof(int);   // counters of the sequences before it
constexpr float kBelowOne = 0x1.fffffep-1f;

using u64 = unsigned long long;

__device__ __forceinline__ uint64_t sub_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Two sums side by side (packed fp32), each in two words: s + lo is exact but for lo's own
// rounding.
struct Sum {
    uint64_t s = 0, lo = 0;
    __device__ __forceinline__ void add(uint64_t d) {        // each within [0, 1]
        lo = add_f32x2(lo, lost(d));
    }
    // Adds p - q, q at most p.
    __device__ __forceinline__ void add(uint64_t p, uint64_t q) {
        const uint64_t d = sub_f32x2(p, q);
        const uint64_t e = sub_f32x2(sub_f32x2(p, d), q);    // what the difference lost
        lo = add_f32x2(lo, add_f32x2(lost(d), e));
    }
    // In units of 2^-58 (each s up to 16).
    __device__ __forceinline__ u64 units() const {
        float a, b, c, d;
        f32x2_split(s, a, b);
        f32x2_split(lo, c, d);
        return units(a, c) + units(b, d);
    }
    static __device__ __forceinline__ u64 units(float s, float lo) {
        return __float2ull_rz(s * 0x1p58f) + static_cast<u64>(__float2ll_rz(lo * 0x1p58f));
    }

  private:
    // Adds d to s; what that lost.
    __device__ __forceinline__ uint64_t lost(uint64_t d) {
        const uint64_t t = add_f32x2(s, d), b = sub_f32x2(t, s);
        const uint64_t x = add_f32x2(sub_f32x2(s, sub_f32x2(t, b)), sub_f32x2(d, b));
        s = t;
        return x;
    }
};

template <typename T>
__device__ __forceinline__ float value(const T* p);
template <>
__device__ __forceinline__ float value<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float value<uint16_t>(const uint16_t* p) {
    return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
template <typename T>
__device__ __forceinline__ void widen(uint4 w, float* x) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
    if (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(a[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf_lo(a[i]);
            x[2 * i + 1] = bf_hi(a[i]);
        }
    }
}

// A row of the vocabulary: of p, of q (NULL: none is taken off), the token without weight
// (-1: none), and the power of two that all weights are multiplied with.
template <typename T>
struct Row {
    const T* p;
    const T* q;
    int vocab, without;
    int lead;                    // elements between the 16-byte boundary below p and p
    float scale;
};

// Vector c (16 bytes, on the boundaries) of `from`, the row's p or q; places outside the row
// get 0.
template <typename T>
__device__ __forceinline__ uint4 load_vector(const Row<T>& r, const T* from, int c) {
    constexpr int N = 16 / sizeof(T);
    const int v0 = c * N - r.lead;
    if (v0 >= 0 && v0 + N <= r.vocab) return __ldcs(reinterpret_cast<const uint4*>(from + v0));
    uint32_t a[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (v0 + e >= 0 && v0 + e < r.vocab) {
            const uint32_t x = __float_as_uint(value<T>(from + v0 + e));
            if (sizeof(T) == 4)
                a[e & 3] = x;
            else
                a[e / 2] |= (x >> 16) << (16 * (e & 1));
        }
    return make_uint4(a[0], a[1], a[2], a[3]);
}
// Vector c's values of p within [0, 1] (NaN: 0), scaled, 0 for the token without weight.
template <typename T, bool SCALED>
__device__ __forceinline__ void p_terms(const Row<T>& r, int c, uint4 p, float* x) {
    constexpr int N = 16 / sizeof(T);
    widen<T>(p, x);
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = SCALED ? __saturatef(x[e]) * r.scale : __saturatef(x[e]);
    const int at = r.without < 0 ? -1 : r.without + r.lead - c * N;
    if (at >= 0 && at < N)
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e == at) x[e] = 0.f;
}
// What q takes off each of them: at most all.
template <typename T, bool SCALED>
__device__ __forceinline__ void q_terms(const Row<T>& r, uint4 q, const float* x, float* y) {
    constexpr int N = 16 / sizeof(T);
    widen<T>(q, y);
#pragma unroll
    for (int e = 0; e < N; ++e)
        y[e] = fminf(SCALED ? fmaxf(y[e], 0.f) * r.scale : fmaxf(y[e], 0.f), x[e]);
}

__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The sum of tile k of the row, in every lane: up to eight vectors a lane in flight.  SCALED:
// `some` is set where this lane sees a weight, however small.
template <typename T, bool BOTH, bool SCALED>
__device__ __forceinline__ u64 tile_sum_of(const Row<T>& r, int k, int lane, bool& some) {
    constexpr int N = 16 / sizeof(T), C = kTile / N / 32, V = BOTH ? 4 : C;
    Sum sum;
#pragma unroll 1
    for (int i0 = 0; i0 < C; i0 += V) {
        const int c = k * (kTile / N) + i0 * 32 + lane;
        uint4 p[V], q[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = load_vector(r, r.p, c + i * 32);
            if (BOTH) q[i] = load_vector(r, r.q, c + i * 32);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float x[N], y[N];
            p_terms<T, SCALED>(r, c + i * 32, p[i], x);
            if (BOTH) q_terms<T, SCALED>(r, q[i], x, y);
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                if (SCALED)
                    some |= BOTH ? x[e] > y[e] || x[e + 1] > y[e + 1] : x[e] > 0.f || x[e + 1] > 0.f;
                if (BOTH)
                    sum.add(f32x2(x[e], x[e + 1]), f32x2(y[e], y[e + 1]));
                else
                    sum.add(f32x2(x[e], x[e + 1]));
            }
        }
    }
    return warp_sum(sum.units());
}
template <typename T, bool SCALED>
__device__ __forceinline__ u64 tile_sum(const Row<T>& r, int k, int lane, bool& some) {
    return r.q != nullptr ? tile_sum_of<T, true, SCALED>(r, k, lane, some)
                          : tile_sum_of<T, false, SCALED>(r, k, lane, some);
}

// Exclusive block-wide sum of one value per thread; *total receives the sum.  All threads
// call it, with two buffers in turn (the values read last must not be written by the next
// call).
__device__ __forceinline__ u64 block_sum_before(u64 x, u64* tmp, u64* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    u64 y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    if (lane == 31) tmp[warp] = y;
    __syncthreads();
    u64 before = y - x, all = 0;
    for (int w = 0; w < nw; ++w) {
        const u64 t = tmp[w];
        before += w < warp ? t : 0;
        all += t;
    }
    *total = all;
    return before;
}

// floor(u * total) for u in [0, 1): u is a whole number m < 2^24 times 2^-s.
__device__ __forceinline__ u64 part_of(float u, u64 total) {
    u = fminf(fmaxf(u, 0.f), kBelowOne);
    const uint32_t bits = __float_as_uint(u);
    const int e = bits >> 23;
    const u64 m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const int s = e ? 150 - e : 149;                      // at least 24
    const u64 lo = m * total, hi = __umul64hi(m, total);
    return s < 64 ? (hi << (64 - s)) | (lo >> s) : s < 128 ? hi >> (s - 64) : 0;
}

// How far sums are off: a lane's sum of a tile by less than four units where it is cut to them,
// those of a row (2^22 tokens, 32 a lane) by 2^19 units, 2^-39; the second words' own rounding is
// less than 2^-40 of the sum (16 terms of up to 2^-24 of it, or twice that with q's, each
// added with 2^-24 of their sum).  Together below 2^-38 of a row that sums to 1.  A sum
// below 2^-16 is made again, scaled so that the true one stays below 2^-2; scaled it passes
// 2^-16, or the scale is the last: there the smallest fp32 number is 2^17 units, nothing is cut,
// and a sum of 0 is one of no weights.
constexpr u64 kSmall = 1ull << 42;
constexpr int kMaxShift = 108;
__device__ __forceinline__ int next_shift(int shift, u64 total) {      // (at least 13 more)
    return min(kMaxShift, shift + 56 - (64 - __clzll(static_cast<long long>(total + (1u << 19)))));
}

constexpr int kBlocks = 4;                   // blocks an SM
constexpr int kCluster = 8;                  // blocks of a cluster, at most

template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(256, kBlocks)
    draft_verify_kernel(const T* probs, const T* draft, int64_t row_stride, int vocab, int tiles,
                        const int32_t* tokens, const float* accept_u, const float* sample_u,
                        const int32_t* start, const int32_t* pos, int max_tokens,
                        int32_t* n_accepted, int32_t* next_token, int32_t* keep, int* ws) {
    constexpr int N = 16 / sizeof(T);
    __shared__ int s_stay, s_token, s_last, s_tile;
    __shared__ u64 s_rest;
    __shared__ u64 tmp[3][8];
    extern __shared__ __align__(16) u64 s_sums[];            // [tiles] (CLUSTER)
    if (CLUSTER) cluster_arrive();
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float draw_u = sample_u[b];
    int r0 = start[b], r1 = start[b + 1];
    const bool bad = r0 < 0 || r1 < r0 || r1 > max_tokens;
    const int drafts = bad ? 0 : r1 - r0 - 1;
    const int first_pos = !bad && r0 < r1 ? pos[r0] : -1;
    // (the first 32 drafts come with the position: one latency less)
    int d = -1;
    float u = 0.f;
    auto load_drafts = [&](int i0) {
        if (warp == 0 && i0 + lane < drafts) {
            d = tokens[r0 + i0 + lane + 1];
            u = accept_u[r0 + i0 + lane + 1];
        }
    };
    load_drafts(0);
    if (CLUSTER) cluster_wait();                             // (all blocks have begun)
    if (first_pos < 0) {                                     // the same in every block of the sequence
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            if (bad) flag(ws, SE_DEV_BAD_LENGTH);
            n_accepted[b] = 0;
            next_token[b] = keep[b] = -1;
        }
        return;
    }
    // which drafts stay: every block finds out for itself
    if (warp == 0) {
        int stay = drafts, refused = -1;
        for (int i0 = 0; i0 < drafts; i0 += 32) {
            if (i0 > 0) load_drafts(i0);
            bool out = false;
            if (i0 + lane < drafts) {
                const int64_t t = r0 + i0 + lane;
                out = true;
                if (d >= 0 && d < vocab) {
                    const double x = fminf(fmaxf(u, 0.f), kBelowOne);
                    const double p = value<T>(probs + t * row_stride + d);
                    const double q = draft ? value<T>(draft + t * row_stride + d) : 1.0;
                    out = !(x * q < p);
                }
            }
            const uint32_t m = __ballot_sync(0xffffffffu, out);
            if (m != 0) {
                stay = i0 + __ffs(m) - 1;
                refused = __shfl_sync(0xffffffffu, d, __ffs(m) - 1);
                break;
            }
        }
        if (lane == 0) {
            s_stay = stay;
            s_token = refused;
        }
    }
    __syncthreads();
    const int stay = s_stay, refused = s_token;              // (the refused draft, if one is)
    const bool outside = stay < drafts && (refused < 0 || refused >= vocab);
    const int64_t at = (r0 + stay) * row_stride;
    Row<T> row;
    row.p = probs + at;
    row.q = stay < drafts && draft != nullptr ? draft + at : nullptr;
    row.vocab = vocab;
    row.without = stay < drafts && draft == nullptr && !outside ? refused : -1;
    row.lead = static_cast<int>(reinterpret_cast<uintptr_t>(row.p) % 16 / sizeof(T));
    row.scale = 1.f;
    u64* sums = reinterpret_cast<u64*>(reinterpret_cast<char*>(ws) + kSumsAt) + (int64_t)b * tiles;
    const int nw = blockDim.x >> 5;
    bool some = false;
    for (int k = blockIdx.x * nw + warp; k < tiles; k += gridDim.x * nw) {
        const u64 sum = tile_sum<T, false>(row, k, lane, some);
        if (lane == 0) {
            if (CLUSTER)
                cluster_poke(s_sums + k, 0, sum);
            else
                sums[k] = sum;
        }
    }
    // the sequence's last block goes on; of a cluster the first
    int* arrived = ws + 64 + b;
    if (CLUSTER) {
        cluster_sync();
        if (blockIdx.x != 0) return;
    } else {
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) s_last = atomicAdd(arrived, 1) == static_cast<int>(gridDim.x) - 1;
        __syncthreads();
        if (!s_last) return;
        __threadfence();
    }
    auto sum_of = [&](int k) { return CLUSTER ? s_sums[k] : __ldcg(sums + k); };
    // a thread's run of tiles, so that one scan serves any number of them
    const int per = (tiles + blockDim.x - 1) / blockDim.x;
    const int k0 = min(static_cast<int>(threadIdx.x) * per, tiles), k1 = min(k0 + per, tiles);
    u64 total = 0, ahead = 0, held = 0;
    int shift = 0;
    for (int round = 0;; ++round) {
        held = 0;
        for (int k = k0; k < k1; ++k) held += sum_of(k);
        ahead = block_sum_before(held, tmp[round & 1], &total);
        if (total >= kSmall) break;
        if (shift < kMaxShift) {
            shift = next_shift(shift, total);
        } else if (total == 0 && (row.q != nullptr || row.without >= 0)) {
            // nothing is left of p beside q: drawn from p
            row.q = nullptr;
            row.without = -1;
            shift = 0;
        } else {
            break;
        }
        row.scale = __int_as_float((127 + shift) << 23);
        some = false;
        for (int k = warp; k < tiles; k += nw) {
            const u64 sum = tile_sum<T, true>(row, k, lane, some);
            if (lane == 0) *(CLUSTER ? s_sums + k : sums + k) = sum;
        }
        if (!__syncthreads_or(some)) shift = kMaxShift;      // no scale finds a weight
    }
    if (threadIdx.x == 0) {
        if (!CLUSTER) *arrived = 0;
        if (outside) flag(ws, SE_DEV_BAD_INDEX);
        if (total == 0) flag(ws, SE_DEV_BAD_VALUE);
        n_accepted[b] = stay;
        keep[b] = first_pos + 1 + stay;
        next_token[b] = total == 0 ? -1 : vocab - 1;
    }
    if (total == 0) return;
    const u64 want = part_of(draw_u, total);             // the first token whose sum passes it
    if (threadIdx.x == 0) s_tile = tiles;
    __syncthreads();
    if (ahead <= want && want < ahead + held) {
        int k = k0;
        for (u64 w; k < k1 - 1 && ahead + (w = sum_of(k)) <= want; ++k) ahead += w;
        s_tile = k;
        s_rest = want - ahead;
    }
    __syncthreads();
    if (s_tile == tiles) return;
    // in the tile: a vector a thread
    u64 w[N], sum = 0;
    const int c = s_tile * (kTile / N) + threadIdx.x;
    if (threadIdx.x < kTile / N) {
        float x[N], y[N];
        p_terms<T, true>(row, c, load_vector(row, row.p, c), x);
        if (row.q != nullptr) q_terms<T, true>(row, load_vector(row, row.q, c), x, y);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float q = row.q != nullptr ? y[e] : 0.f, d = x[e] - q;
            // (less than a unit counts as one: a tile that was chosen has a token with weight)
            w[e] = Sum::units(d, (x[e] - d) - q);
            if (w[e] == 0 && d > 0.f) w[e] = 1;
            sum += w[e];
        }
    }
    u64 part;
    ahead = block_sum_before(sum, tmp[2], &part);
    // (the weights one by one may end before the tile's sum, by up to a unit each: then it is the last)
    const u64 rest = part == 0 ? 0 : min(s_rest, part - 1);
    if (sum > 0 && ahead <= rest && rest < ahead + sum) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (ahead <= rest && rest < ahead + w[e]) next_token[b] = c * N - row.lead + e;
            ahead += w[e];
        }
    }
}

}  // namespace

int draft_verify_max_batch() { return kMaxBatch; }

// (rows may begin off a 16-byte boundary: up to 7 places more)
static int verify_tiles(int vocab) { return (vocab + 7 + kTile - 1) / kTile; }

size_t draft_verify_ws_bytes(int batch, int vocab) {
    return (kSumsAt + (size_t)batch * verify_tiles(vocab) * sizeof(u64) + 255) & ~(size_t)255;
}

cudaError_t launch_draft_verify(const void* probs, const void* draft, int64_t row_stride,
                                int prob_dtype, int vocab, const int32_t* tokens,
                                const float* accept_u, const float* sample_u, const se_chunk& ck,
                                int batch, int32_t* n_accepted, int32_t* next_token, int32_t* keep,
                                int* ws, cudaStream_t s) {
    const int tiles = verify_tiles(vocab);
    // a block's eight warps have a tile each at least; one wave of blocks
    const int split = std::max(1, std::min((tiles + 7) / 8, kBlocks * num_sms() / batch));
    const dim3 grid(split, batch);
    auto run = [&](auto kernel, auto type, int cluster) {
        using T = decltype(type);
        return launch_cluster(kernel, grid, dim3(256), cluster ? tiles * sizeof(u64) : 0, cluster, s,
                              static_cast<const T*>(probs), static_cast<const T*>(draft), row_stride,
                              vocab, tiles, tokens, accept_u, sample_u, (const int32_t*)ck.start,
                              (const int32_t*)ck.pos, ck.max_tokens, n_accepted, next_token, keep, ws);
    };
    if (prob_dtype == 1)
        return split <= kCluster ? run(draft_verify_kernel<float, true>, float(), split)
                                 : run(draft_verify_kernel<float, false>, float(), 0);
    return split <= kCluster ? run(draft_verify_kernel<uint16_t, true>, uint16_t(), split)
                             : run(draft_verify_kernel<uint16_t, false>, uint16_t(), 0);
}

}  // namespace se
