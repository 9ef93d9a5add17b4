// What the kernels over page tables share: block-wide sums of lengths that come from the device, and
// the block that finishes last.
#pragma once

#include "common.cuh"

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

}  // namespace
}  // namespace se
