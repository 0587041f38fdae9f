// The pages of the cache that the new token's attention reads: per channel the least and greatest key
// of a page (bounds), from them a bound on what a page can score (scores), and the best pages (select).
#include <algorithm>
#include <climits>

#include <math_constants.h>

#include "ragged.cuh"

namespace moe {

namespace {

// Tokens of request b that the block table has room for.
__device__ __forceinline__ int tokens_of(const PageArgs& a, int b) {
    const int n = max(a.seq_lens[b], 0);
    return (int)min((long long)n, (long long)a.max_pages * a.page_size);
}
// Pages of n tokens, without a sum that may pass 2^31.
__device__ __forceinline__ int pages_of(int n, int page_size) { return n > 0 ? (n - 1) / page_size + 1 : 0; }
__device__ __forceinline__ void report_lengths(const PageArgs& a) {
    if (blockIdx.x != 0 || !a.status) return;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x)
        if ((long long)a.seq_lens[b] > (long long)a.max_pages * a.page_size) set_status(a.status, MOE_ERR_DEVICE);
}

// ---- bounds -------------------------------------------------------------------
//
// A page's rows are read once and the least and greatest of a channel come out: memory bounds it, or a
// few trips to it for the pages of a few new tokens.  A unit is 16 bytes of a head's row and all rows of a
// page, so that a thread needs nothing of another; where there are fewer units than threads, up to 8
// threads share the rows of a unit and meet in shared memory.
constexpr int kBoundsThreads = 256;
constexpr int kBoundsParts = 8;
constexpr int kBoundsBlocks = 4;            // per SM
constexpr int kBoundsAhead = 8;             // rows in flight per thread

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t*>(&v); }

// The least and greatest of 16 bytes of a row so far.  E4M3 codes are compared as the upper bytes of bf16 numbers,
// which are in the same order (sign and magnitude; no code is a NaN there): a word's codes are two pairs.
template <bool F8>
struct Extremes {
    static constexpr int N = F8 ? 8 : 4;
    uint32_t lo[N], hi[N];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            lo[i] = F8 ? 0x7f007f00u : 0x7f807f80u;
            hi[i] = F8 ? 0xff00ff00u : 0xff80ff80u;
        }
    }
    __device__ __forceinline__ void take(int i, uint32_t l, uint32_t h) {
        lo[i] = as_u32(__hmin2_nan(as_bf162(lo[i]), as_bf162(l)));
        hi[i] = as_u32(__hmax2_nan(as_bf162(hi[i]), as_bf162(h)));
    }
    __device__ __forceinline__ void add(uint4 v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F8) {
                const uint32_t odd = w[i] & 0xff00ff00u, even = (w[i] << 8) & 0xff00ff00u;
                take(2 * i, even, even);
                take(2 * i + 1, odd, odd);
            } else {
                take(i, w[i], w[i]);
            }
        }
    }
    __device__ __forceinline__ uint4 packed(const uint32_t (&e)[N]) const {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F8) w[i] = e[2 * i] >> 8 | e[2 * i + 1];
            else w[i] = e[i];
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void join(uint4 l, uint4 h) {
        Extremes o;
        o.clear();
        o.add(l);
        Extremes p;
        p.clear();
        p.add(h);
#pragma unroll
        for (int i = 0; i < N; ++i) take(i, o.lo[i], p.hi[i]);
    }
};

template <bool F8>
__global__ void __launch_bounds__(kBoundsThreads, kBoundsBlocks) page_bounds_kernel(const __grid_constant__ BoundsArgs a) {
    constexpr int kElems = F8 ? 16 : 8;      // of 16 bytes
    __shared__ LineShared<kBoundsThreads> sh;
    __shared__ uint4 meet[2][kBoundsThreads];
    pdl_allow_dependents();
    pdl_wait_primary();
    report_lengths(a);
    const int P = a.page_size, heads = a.c.heads, vecs = a.c.head_dim / kElems, tid = threadIdx.x;
    const long long columns = (long long)heads * vecs;       // of a page
    auto first_page = [&](int b) { return a.first ? max(a.first[b], 0) / P : 0; };
    auto count = [&](int b) {
        const int n = tokens_of(a, b);
        if (a.first && a.first[b] >= n) return 0ll;
        return (pages_of(n, P) - first_page(b)) * columns;
    };
    long long total;
    int parts = 1;
    auto shares = [&](long long t) {
        while (parts < kBoundsParts && parts < P && t * parts * 2 <= (long long)gridDim.x * kBoundsThreads) parts *= 2;
        return (t * parts + kBoundsThreads - 1) / kBoundsThreads;
    };
    Stretch s = line_share<kBoundsThreads>(a.B, count, shares, sh, total);
    const int wide = kBoundsThreads / parts, part = tid / wide, me = tid - part * wide;
    for (long long left = s.n; left > 0; left -= wide) {
        Stretch mine = s;
        if (me < left) mine.skip(me, count);
        Extremes<F8> e;
        e.clear();
        bool good = me < left;
        char* to = nullptr;
        if (good) {
            const long long at = div_u(mine.at, columns);
            const int v = (int)(mine.at - at * columns), g = v / vecs, col = first_page(mine.b) + (int)at;
            const int page = a.table[mine.b * a.table_ld + col];
            if (page < 0 || page >= a.c.num_pages) {
                if (a.status) set_status(a.status, MOE_ERR_DEVICE);
                good = false;
            } else {
                const uint32_t rows = min(P, tokens_of(a, mine.b) - col * P);
                const long long size = F8 ? 1 : 2;
                const char* from = static_cast<const char*>(a.c.k) +
                                   (page * a.c.k_page_stride + g * a.c.k_head_stride + (v - g * vecs) * kElems) * size;
                to = static_cast<char*>(a.bounds) + (((long long)page * heads + g) * 2 * a.c.head_dim + (v - g * vecs) * kElems) * size;
                for (uint32_t r = part; r < rows; r += kBoundsAhead * parts) {
                    uint4 w[kBoundsAhead];
                    // the last row again instead of those beyond it
#pragma unroll
                    for (int i = 0; i < kBoundsAhead; ++i)
                        w[i] = *reinterpret_cast<const uint4*>(from + min(r + i * parts, rows - 1u) * a.c.k_slot_stride * size);
#pragma unroll
                    for (int i = 0; i < kBoundsAhead; ++i) e.add(w[i]);
                }
            }
        }
        if (parts > 1) {
            __syncthreads();
            meet[0][tid] = e.packed(e.lo);
            meet[1][tid] = e.packed(e.hi);
            __syncthreads();
            for (int p = 1; part == 0 && p < parts; ++p) e.join(meet[0][p * wide + me], meet[1][p * wide + me]);
        }
        if (good && part == 0) {
            *reinterpret_cast<uint4*>(to) = e.packed(e.lo);
            *reinterpret_cast<uint4*>(to + a.c.head_dim * (F8 ? 1 : 2)) = e.packed(e.hi);
        }
        s.skip(wide, count);
    }
}

// ---- scores -------------------------------------------------------------------
//
// sum over the heads h of a group of sum_d max(q_hd lo_d, q_hd hi_d) is one product of length 2 D,
//   sum_d (sum_h min(q_hd, 0)) lo_d + (sum_h max(q_hd, 0)) hi_d,
// as lo <= hi: two additions and multiplications per value read, and memory bounds it.  Units are
// (request, key-value head, page); a warp takes a run of them, the sums of q in its registers, L lanes to a
// page's 2 D values and 8 pages under way per lane.
constexpr int kScoreThreads = 256;
constexpr int kScorePages = 8;              // of a lane at a time

template <bool F8, int L, int VL>
__global__ void __launch_bounds__(kScoreThreads, 2) page_scores_kernel(const __grid_constant__ ScoresArgs a) {
    constexpr int E = F8 ? 16 : 8, kWarps = kScoreThreads / 32, kSide = 32 / L, kBatch = kScorePages * kSide;
    __shared__ LineShared<kScoreThreads> sh;
    pdl_allow_dependents();
    pdl_wait_primary();
    report_lengths(a);
    const int heads = a.c.heads, D = a.c.head_dim, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int side = lane / L, at0 = lane % L, vecs = 2 * D / E;
    auto pages = [&](int b) { return pages_of(tokens_of(a, b), a.page_size); };
    auto count = [&](int b) { return (long long)pages(b) * heads; };
    long long total;
    Stretch s = line_share<kScoreThreads>(a.B, count, [&](long long t) { return (t + kWarps * kBatch - 1) / (kWarps * kBatch); }, sh, total);
    // the warp's part, in whole batches
    const long long per = ((s.n + kWarps - 1) / kWarps + kBatch - 1) / kBatch * kBatch, whole = s.n;
    s.skip(min(warp * per, whole), count);
    s.n = min(per, whole - warp * per);
    while (s.n > 0) {
        const int b = s.b, np = pages(b), g = (int)div_u(s.at, np);
        int col = (int)(s.at - (long long)g * np);
        const int end = (int)min((long long)np, col + s.n);
        // the sums of q that go with the lane's values
        float q[VL][E];
        const float ks = a.c.k_scale ? a.c.k_scale[g] : 1.0f;
#pragma unroll
        for (int v = 0; v < VL; ++v) {
            const int vec = at0 + v * L, d = vec * E;
            const bool low = d < D;
#pragma unroll
            for (int e = 0; e < E; ++e) q[v][e] = 0.0f;
            for (int h = 0; vec < vecs && h < a.group; ++h) {
                const long long i = b * a.q_bs + (g * a.group + h) * a.q_hs + (low ? d : d - D);
#pragma unroll
                for (int j = 0; j < E; j += 8) {
                    float f[8];
                    load8_f32(a.q, a.q_dt, i + j, f);
                    // NaN goes into both
#pragma unroll
                    for (int e = 0; e < 8; ++e) q[v][j + e] += (low ? f[e] > 0.0f : f[e] < 0.0f) ? 0.0f : f[e];
                }
            }
        }
        const int32_t* row = a.table + b * a.table_ld;
        float* out = a.scores + ((long long)b * heads + g) * a.max_pages;
        auto ids = [&](int c) { return lane < kBatch && c + lane < end ? max(row[c + lane], -1) : INT_MIN; };
        int id = ids(col);
        s.skip(end - col, count);
        for (; col < end; col += kBatch) {
            const int next = ids(col + kBatch);
            if (id != INT_MIN && (id < 0 || id >= a.c.num_pages)) {
                if (a.status) set_status(a.status, MOE_ERR_DEVICE);
                id = -1;
            }
            __syncwarp();
            uint4 w[kScorePages][VL];
#pragma unroll
            for (int u = 0; u < kScorePages; ++u) {
                const int page = __shfl_sync(0xffffffffu, id, u * kSide + side);
                const char* from = static_cast<const char*>(a.bounds) + ((long long)page * heads + g) * vecs * 16;
#pragma unroll
                for (int v = 0; v < VL; ++v) {
                    const int vec = at0 + v * L;
                    w[u][v] = page >= 0 && vec < vecs ? reinterpret_cast<const uint4*>(from)[vec] : make_uint4(0, 0, 0, 0);
                }
            }
            float sum[kScorePages];
#pragma unroll
            for (int u = 0; u < kScorePages; ++u) {
                sum[u] = 0.0f;
#pragma unroll
                for (int v = 0; v < VL; ++v) {
                    if constexpr (F8) {
                        const uint32_t x[4] = {w[u][v].x, w[u][v].y, w[u][v].z, w[u][v].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 l = unpack_e4m3x2<false>(x[i]), h = unpack_e4m3x2<true>(x[i]);
                            sum[u] = fmaf(q[v][4 * i], l.x, sum[u]);
                            sum[u] = fmaf(q[v][4 * i + 1], l.y, sum[u]);
                            sum[u] = fmaf(q[v][4 * i + 2], h.x, sum[u]);
                            sum[u] = fmaf(q[v][4 * i + 3], h.y, sum[u]);
                        }
                    } else {
                        float f[8];
                        unpack_bf16x8(w[u][v], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum[u] = fmaf(q[v][e], f[e], sum[u]);
                    }
                }
            }
            // Sums over the L lanes of a page: at the three widest steps a lane keeps half of its pages and
            // hands on the others, then all lanes of a page add up.
            int mine = 0;
#pragma unroll
            for (int n = kScorePages / 2, o = L / 2; n > 0; n /= 2, o /= 2) {
                const bool up = lane & o;
                mine += up ? n : 0;
#pragma unroll
                for (int u = 0; u < kScorePages / 2; ++u) {
                    if (u >= n) continue;
                    const float give = up ? sum[u] : sum[u + n], keep = up ? sum[u + n] : sum[u];
                    sum[u] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            }
            float total_q = sum[0];
#pragma unroll
            for (int o = L / 16; o > 0; o /= 2) total_q += __shfl_xor_sync(0xffffffffu, total_q, o);
            const int at = mine * kSide + side, known = __shfl_sync(0xffffffffu, id, at);
            if (lane % (L / 8) == 0 && known != INT_MIN) out[col + at] = known < 0 ? -CUDART_INF_F : total_q * ks;
            id = next;
        }
    }
}

// ---- select -------------------------------------------------------------------
//
// One block per (request, key-value head).  Scores become whole numbers of the same order, forced pages the
// greatest; the `keep`-th greatest is found digit by digit (8 bits each, from the highest bit in which two of
// them differ), and the pages above it, with the first ones equal to it, are written in order.
constexpr int kSelectThreads = 256;
constexpr int kSelectKeys = 8192;           // kept in shared memory; the others are read again

// Scores in ascending order; NaN above all, -0 like 0.
__device__ __forceinline__ uint32_t key_of(float s) {
    if (s != s) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(s + 0.0f);
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(kSelectThreads) page_select_kernel(const __grid_constant__ SelectArgs a) {
    constexpr int kWarps = kSelectThreads / 32;
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ uint32_t hist[256], found[2];
    __shared__ uint32_t ends[2][kWarps];
    __shared__ long long wsum[kWarps];
    pdl_allow_dependents();
    pdl_wait_primary();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, unit = blockIdx.x, b = unit / a.heads, keep = a.keep;
    const int n = tokens_of(a, b), pages = pages_of(n, a.page_size), kept = min(keep, pages);
    const float* scores = a.scores + (long long)unit * a.max_pages;
    const int32_t* row = a.table + b * a.table_ld;
    int32_t* out = a.tables + (long long)unit * keep;
    if (tid == 0) {
        // whole pages but for the last one, if that is among them
        a.lens[unit] = pages <= keep ? n : kept * a.page_size;
    }
    for (int i = kept + tid; i < keep; i += kSelectThreads) out[i] = -1;
    if (pages <= keep) {
        for (int i = tid; i < pages; i += kSelectThreads) out[i] = row[i];
        return;
    }
    auto key_at = [&](int i) {
        return i < a.sinks || i >= pages - a.recent ? 0xffffffffu : key_of(scores[i]);
    };
    uint32_t low = 0xffffffffu, high = 0u;
    for (int i = tid; i < pages; i += kSelectThreads) {
        const uint32_t k = key_at(i);
        if (i < a.cached) keys[i] = k;
        low = min(low, k);
        high = max(high, k);
    }
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) {
        ends[0][warp] = low;
        ends[1][warp] = high;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        low = min(low, ends[0][w]);
        high = max(high, ends[1][w]);
    }
    auto key = [&](int i) { return i < a.cached ? keys[i] : key_at(i); };
    // The keys in question agree with `value` above bit `bits`; `need` of the greatest of them are wanted.
    int bits = 32 - __clz(low ^ high);
    uint32_t value = bits == 32 ? 0u : high >> bits << bits, need = keep;
    while (bits > 0) {
        const int take = min(bits, 8), shift = bits - take;
        hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < pages; i += kSelectThreads) {
            const uint32_t k = key(i);
            if (bits == 32 || (k ^ value) >> bits == 0) atomicAdd(hist + (k >> shift & ((1u << take) - 1u)), 1u);
        }
        __syncthreads();
        // keys of this digit or a greater one, thread 0 at the greatest digit
        const uint32_t mine = hist[255 - tid];
        uint32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) ends[0][warp] = incl;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (w < warp) incl += ends[0][w];
        if (incl >= need && incl - mine < need) {
            found[0] = 255 - tid;
            found[1] = incl - mine;
        }
        __syncthreads();
        value |= found[0] << shift;
        need -= found[1];
        bits = shift;
    }
    // `need` pages of key `value`, the first ones, and all above; a thread has a run of an odd
    // number of pages (bank conflicts), and writes behind what the threads before it do
    const int run = (pages + kSelectThreads - 1) / kSelectThreads | 1, i0 = min(tid * run, pages), i1 = min(i0 + run, pages);
    long long mine = 0;                     // pages above, and in the upper half pages equal
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = key(i);
        mine += k > value ? 1ll : k == value ? 1ll << 32 : 0ll;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp) incl += wsum[w];
    uint32_t above = (uint32_t)(incl - mine), equal = (uint32_t)((incl - mine) >> 32);
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = key(i);
        if (k > value || (k == value && equal < need)) {
            out[above + min(equal, need)] = row[i];
            if (i == pages - 1) a.lens[unit] = n - (pages - keep) * a.page_size;
        }
        above += k > value;
        equal += k == value;
    }
}

template <bool F8, int L, int VL>
cudaError_t launch_scores_as(const ScoresArgs& a, cudaStream_t s) {
    return launch_pdl(page_scores_kernel<F8, L, VL>, dim3((unsigned)(2 * device_sm_count())), dim3(kScoreThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_page_bounds(const BoundsArgs& a, cudaStream_t s) {
    auto kern = a.c.dtype == MOE_DTYPE_FP8_E4M3 ? page_bounds_kernel<true> : page_bounds_kernel<false>;
    return launch_pdl(kern, dim3((unsigned)(kBoundsBlocks * device_sm_count())), dim3(kBoundsThreads), 0, s, a);
}

cudaError_t launch_page_scores(const ScoresArgs& a, cudaStream_t s) {
    const int D = a.c.head_dim;
    if (a.c.dtype == MOE_DTYPE_FP8_E4M3)
        return D <= 64 ? launch_scores_as<true, 8, 1>(a, s) : D <= 128 ? launch_scores_as<true, 16, 1>(a, s) : launch_scores_as<true, 32, 1>(a, s);
    return D <= 32 ? launch_scores_as<false, 8, 1>(a, s)
           : D <= 64 ? launch_scores_as<false, 16, 1>(a, s)
           : D <= 128 ? launch_scores_as<false, 32, 1>(a, s) : launch_scores_as<false, 32, 2>(a, s);
}

cudaError_t launch_page_select(const SelectArgs& args, cudaStream_t s) {
    SelectArgs a = args;
    a.cached = std::min(a.max_pages, kSelectKeys);
    return launch_pdl(page_select_kernel, dim3((unsigned)(a.B * a.heads)), dim3(kSelectThreads), (size_t)a.cached * 4, s, a);
}

}  // namespace moe
