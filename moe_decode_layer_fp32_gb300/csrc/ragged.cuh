// Work of requests of different lengths, shared out evenly without the host knowing them.
#pragma once

#include "block.h"

namespace moe {

// x / y for 0 <= x, 0 < y; 64-bit division only where it must be.
__device__ __forceinline__ long long div_u(long long x, long long y) {
    if (((unsigned long long)(x | y) >> 32) == 0) return (uint32_t)x / (uint32_t)y;
    return x / y;
}

// A stretch of the line in which all requests' units lie end to end: `n` of them from unit `at` of
// request `b` on, which walks forward with them.
struct Stretch {
    int b;
    long long at, n;
    template <class Count>
    __device__ __forceinline__ void skip(long long units, Count count) {
        at += units;
        n -= units;
        if (n <= 0) return;
        for (long long c = count(b); at >= c; c = count(b)) {
            at -= c;
            ++b;
        }
    }
};

template <int THREADS>
struct LineShared {
    long long wsum[THREADS / 32], at;
    int b;
};

// The block's share of the line: of the first shares(total) blocks of the grid each has an equal one, the
// others nothing (n 0).  All threads call it; count(b) >= 0 is the number of units of request b.
template <int THREADS, class Count, class Shares>
__device__ Stretch line_share(int B, Count count, Shares shares, LineShared<THREADS>& sh, long long& total) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // inclusive scan of t over the threads; `all` gets the block's sum
    auto scan = [&](long long t, long long& all) {
        long long incl = t;
        __syncwarp();
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) sh.wsum[warp] = incl;
        __syncthreads();
        all = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) incl += sh.wsum[w];
            all += sh.wsum[w];
        }
        return incl;
    };
    long long have = tid < B ? count(tid) : 0, sum = 0, all;
    long long incl = scan(have, all);
    total = all;
    if (B > THREADS) {
        long long mine = 0, rest;
        for (int b = THREADS + tid; b < B; b += THREADS) mine += count(b);
        __syncthreads();
        scan(mine, rest);
        total += rest;
    }
    const long long blocks = min((long long)gridDim.x, shares(total));
    Stretch s = {0, 0, 0};
    if (blockIdx.x >= blocks || total == 0) return s;
    const long long start = div_u((long long)blockIdx.x * total, blocks), end = div_u(((long long)blockIdx.x + 1) * total, blocks);
    s.n = end - start;
    for (int b0 = 0;;) {
        const long long before = sum + incl - have;
        if (start >= before && start < sum + incl) {
            sh.b = b0 + tid;
            sh.at = start - before;
        }
        sum += all;
        if (start < sum) break;       // the same for all threads
        b0 += THREADS;
        have = b0 + tid < B ? count(b0 + tid) : 0;
        __syncthreads();
        incl = scan(have, all);
    }
    __syncthreads();
    s.b = sh.b;
    s.at = sh.at;
    return s;
}

}  // namespace moe
