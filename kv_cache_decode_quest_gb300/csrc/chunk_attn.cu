// Attention of a chunk of new tokens over a paged cache (se_chunk_attn).
//
// Rows (token, query head of the KV head's group) of one (sequence, KV head)
// share its keys; 16 rows at a time walk the keys page by page with a running
// maximum and sum (online softmax, fp32): per page, 16 x 16 scores, then
// O <- O * exp(m_old - m_new) + P V.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace se {
namespace {

constexpr int kRows = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
    se_paged_kv kv;
    se_chunk ck;
    int batch;
    ChunkAttnArgs a;
    int* status;
};

__device__ __forceinline__ int chunk_start(const Params& p, int b, bool& bad) {
    const int s = p.ck.start[b];
    if (s < 0 || s > p.ck.max_tokens) bad = true;
    return min(max(s, 0), p.ck.max_tokens);
}

// Row blocks of sequence b are numbered from floor(start[b] * G / 16) + b on:
// each sequence has at most as many as the next one's first number leaves.
template <int D>
__global__ void __launch_bounds__(128) chunk_attn_simple_kernel(const Params p) {
    constexpr int DT = D / 8;                       // head_dim elements per thread
    __shared__ float qs[kRows][D + 1], ks[kPage][D + 1], vs[kPage][D], ps[kRows][kPage];
    const int H = p.kv.num_kv_heads, G = p.a.Hq / H;
    const int h = blockIdx.y;
    bool bad = false;
    int lo = 0, hi = p.batch;                        // last b whose first number is <= blockIdx.x
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        const long long first = (long long)chunk_start(p, mid, bad) * G / kRows + mid;
        if (first <= (long long)blockIdx.x) lo = mid;
        else hi = mid;
    }
    const int b = lo;
    const int s0 = chunk_start(p, b, bad), s1 = chunk_start(p, b + 1, bad);
    if (s1 < s0) bad = true;
    const long long blk = (long long)blockIdx.x - ((long long)s0 * G / kRows + b);
    const long long row0 = blk * kRows, rows = (long long)max(0, s1 - s0) * G;
    const int cap = p.kv.max_pages_per_seq * kPage;
    int L = p.kv.ctx_len[b];
    if (L < 0 || L > cap) {
        bad = true;
        L = L < 0 ? 0 : cap;
    }
    if (bad && threadIdx.x == 0) flag(p.status, SE_DEV_BAD_LENGTH);
    if (blk < 0 || row0 >= rows) return;
    const int p0 = p.ck.pos[s0];
    const int r = threadIdx.x / 8, c = threadIdx.x % 8;
    const uint16_t* Q = static_cast<const uint16_t*>(p.a.q);
    for (int i = threadIdx.x; i < kRows * D; i += blockDim.x) {
        const long long row = min(row0 + i / D, rows - 1);
        const int64_t t = s0 + row / G;
        qs[i / D][i % D] = __uint_as_float(
            (uint32_t)Q[t * p.a.q_stride + (h * G + row % G) * D + i % D] << 16);
    }
    const long long my = min(row0 + r, rows - 1);
    const int pos = p0 < 0 ? -1 : p0 + static_cast<int>(my / G);
    if (pos >= L && p0 >= 0 && c == 0) flag(p.status, SE_DEV_BAD_LENGTH);
    float m = -INFINITY, l = 0.f, o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = 0.f;
    const int last = p0 < 0 ? -1 : p0 + static_cast<int>(min(row0 + kRows - 1, rows - 1) / G);
    const int keys = min(L, last + 1);
    const int first_pos = p0 < 0 ? -1 : p0 + static_cast<int>(row0 / G);
    for (int pg = 0; pg * kPage < keys; ++pg) {
        // pages that no row of the block sees
        if (p.a.window && pg * kPage >= p.a.sink && pg * kPage + kPage - 1 <= first_pos - p.a.window)
            continue;
        const int phys = p.kv.block_table[(int64_t)b * p.kv.max_pages_per_seq + pg];
        if (phys < 0 || phys >= p.kv.num_pages) {
            if (threadIdx.x == 0) flag(p.status, SE_DEV_BAD_INDEX);
            continue;
        }
        const int valid = min(kPage, L - pg * kPage);
        const int64_t base = ((int64_t)phys * H + h) * kPage * D;
        const uint16_t* K = static_cast<const uint16_t*>(p.kv.k) + base;
        const uint16_t* V = static_cast<const uint16_t*>(p.kv.v) + base;
        __syncthreads();
        for (int i = threadIdx.x; i < kPage * D; i += blockDim.x) {
            ks[i / D][i % D] = __uint_as_float((uint32_t)K[i] << 16);
            vs[i / D][i % D] = i / D < valid ? __uint_as_float((uint32_t)V[i] << 16) : 0.f;
        }
        __syncthreads();
        float s2[2], mx = m;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int j = c + 8 * e, key = pg * kPage + j;
            float x = 0.f;
            for (int d = 0; d < D; ++d) x = fmaf(qs[r][d], ks[j][d], x);
            const bool see = key <= pos && key < L &&
                             (p.a.window == 0 || key > pos - p.a.window || key < p.a.sink);
            s2[e] = see ? x * p.a.scale * kLog2e : -INFINITY;
            mx = fmaxf(mx, s2[e]);
        }
#pragma unroll
        for (int w = 1; w < 8; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float ref = mx == -INFINITY ? 0.f : mx;
        const float corr = exp2f(m - ref);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float w = exp2f(s2[e] - ref);
            ps[r][c + 8 * e] = w;
            sum += w;
        }
#pragma unroll
        for (int w = 1; w < 8; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        l = l * corr + sum;
        m = mx;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < DT; ++i) {
            float x = o[i] * corr;
            for (int j = 0; j < kPage; ++j) x = fmaf(ps[r][j], vs[j][c + 8 * i], x);
            o[i] = x;
        }
        __syncwarp();
    }
    if (row0 + r >= rows) return;
    const int64_t t = s0 + my / G;
    const int64_t oh = t * p.a.Hq + h * G + my % G;
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < DT; ++i) {
        if (p.a.out_dtype == 1)
            static_cast<float*>(p.a.out)[oh * D + c + 8 * i] = o[i] * inv;
        else
            static_cast<uint16_t*>(p.a.out)[oh * D + c + 8 * i] = to_bf16_bits(o[i] * inv);
    }
    if (p.a.lse && c == 0) p.a.lse[oh] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

size_t chunk_attn_ws_bytes(int, int, int, int, int) { return 256; }

cudaError_t launch_chunk_attn(const se_paged_kv& kv, const se_chunk& ck, int batch,
                              const ChunkAttnArgs& a, void* ws, cudaEvent_t ev_begin,
                              cudaEvent_t ev_end, cudaStream_t s) {
    Params p{kv, ck, batch, a, static_cast<int*>(ws)};
    const int G = a.Hq / kv.num_kv_heads;
    const int64_t blocks = (int64_t)ck.max_tokens * G / kRows + batch;
    const dim3 grid(static_cast<unsigned>(blocks), kv.num_kv_heads);
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
    if (kv.head_dim == 128) chunk_attn_simple_kernel<128><<<grid, 128, 0, s>>>(p);
    else chunk_attn_simple_kernel<64><<<grid, 128, 0, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (ev_end && (e = record(ev_end)) != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace se
