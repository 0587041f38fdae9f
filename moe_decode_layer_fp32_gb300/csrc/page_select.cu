// The pages of the cache that the new token's attention reads: per channel the least and greatest key
// of a page (bounds), from them a bound on what a page can score (scores), and the best pages (select).
#include <algorithm>
#include <climits>
#include <type_traits>

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
//
// Measured: 7 x 16383 tokens of 8 heads of 128 in pages of 64 (242 MB in bf16) 41 us, 6.0 TB/s, and E4M3 23, 5.3;
// 33 requests with a new token each 4.4. With 16 or 4 rows in flight and 2 or 6 blocks per SM 40 and 45 us (E4M3 26 and
// 32), 4 blocks 41 (E4M3 26); without sharing, 128 new tokens of one head 9.2 instead of 5.2.
constexpr int kBoundsThreads = 256;
constexpr int kBoundsParts = 8;
constexpr int kBoundsBlocks = 3;            // per SM
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
// as lo <= hi: an addition and a multiplication per value read, and memory bounds it if the instructions
// per value are few.  So the tensor cores multiply: 8 or 16 pages are the rows of an MMA, and its columns the sums of q
// as three terms of bf16 (of f16 next to E4M3 bounds, which it holds: the E4M3 form of mma.sync is two f16 ones and
// conversions of both operands), 24 bits of them and more.
// A lane reads 16 bytes of its page at a time, in any order of d, as a dot product does not mind it.
// Every warp works alone on a run of batches of one or several heads, with the rows of the next batches on their way
// into shared memory; where a head begins the warp forms its terms of q meanwhile.
//
// Measured, 128 requests of 0 to 32768 tokens in pages of 32, 56 / 8 heads of 128: E4M3 (112 MB) 26 us, bf16 (221 MB) 46; a
// request of 2048 pages, 16 / 4 heads 5.4. About 5 us of that are launch, lengths, shares, page numbers and first
// rows, the rest streams at 5.2 to 5.4 TB/s; other numbers of stages or blocks per SM change 3 %. Ruled out: a
// page's values to 16 lanes with fp32 multiply-adds 59 us (E4M3); the terms formed by a block instead of a warp 38 to 48;
// all heads of a page in one block 46 to 57; a bulk copy per page 30 when these copies took 32 (it is issued one lane after
// another); pieces copied in the order in which they are read (64 bytes a page and instruction) 5 % slower; a page read in
// the place of one that a batch does not have, the same for all warps, 31.5.
constexpr int kScoreThreads = 128;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kScoreSetup = 1;              // what the terms of q cost, in batches

// 4 JC pieces of 16 bytes: a page's 2 D values, rounded up.  U: 8 U pages are a batch.
template <bool F8, int JC>
struct Scores {
    static constexpr int E = F8 ? 16 : 8, MC = E / 4;        // values of a piece, and its MMAs
    static constexpr int U = JC >= 8 ? 1 : 8 / JC;
    static constexpr int kBatch = 8 * U;
    static constexpr int kValues = 4 * JC * E;
    static constexpr int V = kValues > 256 ? kValues / 32 : 8;   // of a lane, in the terms of q
    // B fragments of q: for each MMA the words of three terms, 4 lanes, 2 words
    static constexpr int kWords = JC * MC * 24;
    static constexpr int kStage = U * JC * 512;              // a warp's
    static constexpr int kStages = 3;
    static constexpr int kWarpBytes = kStages * kStage + kWords * 4;
    static constexpr int kSmem = kScoreWarps * kWarpBytes;
    static constexpr int kBlocksPerSm = JC >= 16 ? 2 : JC >= 8 ? 3 : 4;
    static_assert(kBatch <= 32, "a lane's page");
    static_assert(kBlocksPerSm * (kSmem + 1280) <= 228 * 1024, "blocks that run at once");
};

// max(x, 0) of two bf16 and of an fp32; NaN stays NaN.
__device__ __forceinline__ uint32_t relu_bf16x2(uint32_t x) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0u));
    return r;
}
__device__ __forceinline__ float relu_f32(float x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(0.0f));
    return r;
}

template <bool F8, int JC>
__global__ void __launch_bounds__(kScoreThreads, (Scores<F8, JC>::kBlocksPerSm)) page_scores_kernel(const __grid_constant__ ScoresArgs a) {
    using K = Scores<F8, JC>;
    constexpr int E = K::E, U = K::U, kBatch = K::kBatch, V = K::V;
    extern __shared__ __align__(16) char smem[];
    __shared__ LineShared<kScoreThreads> sh;
    const int heads = a.c.heads, D = a.c.head_dim, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pieces = 2 * D / E;
    char* ring = smem + warp * K::kWarpBytes;
    uint32_t* frag = reinterpret_cast<uint32_t*>(ring + K::kStages * K::kStage);
    pdl_allow_dependents();
    pdl_wait_primary();
    report_lengths(a);
    auto pages = [&](int b) { return pages_of(tokens_of(a, b), a.page_size); };
    auto batches = [&](int np) { return np > 0 ? (np - 1) / kBatch + 1 : 0; };
    // a head's batches, and what its queries cost before the first one
    auto count = [&](int b) {
        const int nb = batches(pages(b));
        return nb > 0 ? (long long)(nb + kScoreSetup) * heads : 0;
    };
    long long total;
    // a batch to each warp at least
    Stretch s = line_share<kScoreThreads>(a.B, count, [&](long long t) { return (t + kScoreWarps - 1) / kScoreWarps; }, sh, total);
    // the warp's part
    const long long from_unit = s.n * warp / kScoreWarps, to_unit = s.n * (warp + 1) / kScoreWarps;
    s.skip(from_unit, count);
    struct Walk {
        int b, g, np, nb;
        int n, last;              // the head's batches of the run
        long long left;           // units of the run behind this head
    };
    auto take = [&](Walk& w, int r) {
        const int units = (int)min((long long)(w.nb + kScoreSetup - r), w.left);
        w.left -= units;
        w.n = max(r - kScoreSetup, 0);
        w.last = max(r + units - kScoreSetup, 0);
    };
    // to the run's next head with batches
    auto next_head = [&](Walk& w) {
        do {
            if (w.left <= 0) return false;
            if (++w.g == heads) {
                w.g = 0;
                do w.np = pages(++w.b);
                while (w.np == 0);
                w.nb = batches(w.np);
            }
            take(w, 0);
        } while (w.n >= w.last);
        return true;
    };
    Walk here = {s.b, 0, 0, 0, 0, 0, to_unit - from_unit};
    if (here.left <= 0) return;
    here.np = pages(here.b);
    here.nb = batches(here.np);
    here.g = (int)div_u(s.at, here.nb + kScoreSetup);
    take(here, (int)(s.at - (long long)here.g * (here.nb + kScoreSetup)));
    if (here.n >= here.last && !next_head(here)) return;
    // ---- the copies, kStages - 1 batches ahead
    Walk ahead = here;
    bool more = true;
    int stage_in = 0;
    const uint32_t place = smem_u32(ring);
    const long long page_bytes = (long long)heads * pieces * 16;
    auto ask = [&]() {
        const int col = ahead.n * kBatch + lane;
        return lane < kBatch && col < ahead.np ? max(a.table[ahead.b * a.table_ld + col], -1) : INT_MIN;
    };
    int id_next = ask(), ids[K::kStages - 1];      // pages of the batches under way, a lane each (INT_MIN: none, -1: no such)
    auto feed = [&](int& id) {
        id = INT_MIN;
        if (!more) return;
        id = id_next;
        const int g = ahead.g;
        if (++ahead.n >= ahead.last) more = next_head(ahead);
        if (more) id_next = ask();
        if (id != INT_MIN && (id < 0 || id >= a.c.num_pages)) {
            if (a.status) set_status(a.status, MOE_ERR_DEVICE);
            id = -1;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < U * JC; ++i) {
            // A page that is not there stays what the stage has (nobody looks at its sum; reads of some page instead
            // of it, the same for all warps, took 13.4 us for 128 requests of one page, and 5.4 without). Pieces behind the
            // last one are that one: they meet terms of 0.
            const int at = (i * 32 + lane) / (4 * JC), piece = (i * 32 + lane) % (4 * JC);
            const int page = __shfl_sync(0xffffffffu, id, at);
            if (page < 0) continue;
            const char* from = static_cast<const char*>(a.bounds) + page * page_bytes + ((long long)g * pieces + min(piece, pieces - 1)) * 16;
            cp_async16_to(place + stage_in * K::kStage + (at * 4 * JC + (piece ^ (at & 1) << 2)) * 16, from);
        }
        stage_in = stage_in + 1 == K::kStages ? 0 : stage_in + 1;
    };
#pragma unroll
    for (int i = 0; i < K::kStages - 1; ++i) {
        feed(ids[i]);
        cp_async_commit();
    }
    // ---- the products
    // the columns of terms; those behind the last have it again, and count for nothing
    const uint32_t* mine = frag + min(lane / 4, 2) * 8 + lane % 4 * 2;
    int stage = 0;
    do {
        // the sums of q: V of the 2 D values to a lane, eight query heads' loads together (the type is asked outside the
        // loop); the lower side's with its sign turned
        float q[V] = {};
        auto add = [&](auto dt) {
            constexpr bool BF = decltype(dt)::value == MOE_DTYPE_BF16;
            constexpr int N = BF ? 1 : 2;
#pragma unroll
            for (int v = 0; v < V; v += 8) {
                const int d = lane * V + v;
                const uint32_t turn = d < D ? BF ? 0x80008000u : 0x80000000u : 0u;
                const char* from = static_cast<const char*>(a.q) + (here.b * a.q_bs + here.g * a.group * a.q_hs + (d < D ? d : d - D)) * (2 * N);
                for (int h0 = 0; d < 2 * D && h0 < a.group; h0 += 8) {
                    uint4 w[8][N];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int c = 0; c < N; ++c)
                            w[k][c] = h0 + k < a.group ? reinterpret_cast<const uint4*>(from + (h0 + k) * a.q_hs * (2 * N))[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int c = 0; c < N; ++c) {
                            const uint32_t x[4] = {w[k][c].x ^ turn, w[k][c].y ^ turn, w[k][c].z ^ turn, w[k][c].w ^ turn};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if constexpr (BF) {
                                    const uint32_t y = relu_bf16x2(x[i]);
                                    q[v + 2 * i] += __uint_as_float(y << 16);
                                    q[v + 2 * i + 1] += __uint_as_float(y & 0xffff0000u);
                                } else {
                                    q[v + c * 4 + i] += relu_f32(__uint_as_float(x[i]));
                                }
                            }
                        }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) q[v + e] = d < D ? -q[v + e] : q[v + e];
            }
        };
        if (a.q_dt == MOE_DTYPE_BF16) add(std::integral_constant<int, MOE_DTYPE_BF16>());
        else add(std::integral_constant<int, MOE_DTYPE_F32>());
        float back = a.c.k_scale ? a.c.k_scale[here.g] : 1.0f, turn_back = 1.0f;
        if constexpr (F8) {
            // a power of two brings the greatest between 2^14 and 2^15: f16 holds it, and three terms 2^-38 of it
            float most = 0.0f;
#pragma unroll
            for (int e = 0; e < V; ++e) most = fmaxf(most, fabsf(q[e]));
            __syncwarp();
            const uint32_t e = __reduce_max_sync(0xffffffffu, __float_as_uint(most)) >> 23, up = min(268 - e, 253u);
            // on one side of 1 both, they stay two factors: their product may be no normal number, and the score one
            const float down = __uint_as_float((254 - up) << 23);
            if ((down < 1.0f) == (back < 1.0f)) turn_back = down;
            else back *= down;
#pragma unroll
            for (int v = 0; v < V; ++v) q[v] *= __uint_as_float(up << 23);
        }
        __syncwarp();       // the terms of the head before have been read
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            const int at = lane * V + v, piece = at / E;
            if (at >= K::kValues) break;
            uint32_t* to = frag + (piece / 4 * K::MC + at % E / 4) * 24 + piece % 4 * 2 + at % 4 / 2;
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                if constexpr (F8) {
                    const uint32_t w = pack_f16x2(q[v], q[v + 1]);
                    const float2 have = unpack_f16x2(w);
                    to[t * 8] = w;
                    q[v] -= have.x;
                    q[v + 1] -= have.y;
                } else {
                    to[t * 8] = pack_hi(q[v], q[v + 1]);
                    q[v] -= bf16_trunc(q[v]);
                    q[v + 1] -= bf16_trunc(q[v + 1]);
                }
            }
        }
        __syncwarp();
        float* out = a.scores + ((long long)here.b * heads + here.g) * a.max_pages;
        for (; here.n < here.last; ++here.n) {
            cp_async_wait<K::kStages - 2>();
            __syncwarp();          // all lanes' pieces are there, and the stage before has been read
            const int had = ids[0];
#pragma unroll
            for (int i = 0; i + 2 < K::kStages; ++i) ids[i] = ids[i + 1];
            feed(ids[K::kStages - 2]);
            cp_async_commit();
            const char* rows = ring + stage * K::kStage + lane / 4 * JC * 64 + lane % 4 * 16;
            const int odd = lane / 4 % 2 * 64;
            stage = stage + 1 == K::kStages ? 0 : stage + 1;
            constexpr int G = (U + 1) / 2;          // 16 pages each
            float c[G][2][4] = {};                  // two chains of additions
#pragma unroll
            for (int j = 0; j < JC; ++j) {
                uint4 y[2 * G] = {};
#pragma unroll
                for (int u = 0; u < U; ++u) y[u] = *reinterpret_cast<const uint4*>(rows + u * JC * 512 + j * 64 + (j % 2 ? -odd : odd));
#pragma unroll
                for (int i = 0; i < K::MC; ++i) {
                    const uint2 f = *reinterpret_cast<const uint2*>(mine + (j * K::MC + i) * 24);
#pragma unroll
                    for (int k = 0; k < G; ++k) {
                        const uint4 y0 = y[2 * k], y1 = y[2 * k + 1];
                        const uint32_t x0[4] = {y0.x, y0.y, y0.z, y0.w}, x1[4] = {y1.x, y1.y, y1.z, y1.w};
                        if constexpr (F8)
                            mma_f16(c[k][i % 2], e4m3x2_to_f16x2<false>(x0[i]), U > 1 ? e4m3x2_to_f16x2<false>(x1[i]) : 0u,
                                    e4m3x2_to_f16x2<true>(x0[i]), U > 1 ? e4m3x2_to_f16x2<true>(x1[i]) : 0u, f.x, f.y);
                        else
                            mma_bf16(c[k][i % 2], x0[2 * i], x1[2 * i], x0[2 * i + 1], x1[2 * i + 1], f.x, f.y);
                    }
                }
            }
            // lane 4 p has page p's (and 8 + p's) sums of the first two terms, its neighbour that of the third
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float(&c0)[4] = c[u / 2][0];
                const float(&c1)[4] = c[u / 2][1];
                const float first = c0[u % 2 * 2] + c1[u % 2 * 2], second = c0[u % 2 * 2 + 1] + c1[u % 2 * 2 + 1];
                const float found = first + (second + __shfl_down_sync(0xffffffffu, first, 1));
                const int at = u * 8 + lane / 4, known = __shfl_sync(0xffffffffu, had, at);
                if (lane % 4 == 0 && known != INT_MIN) out[here.n * kBatch + at] = known < 0 ? -CUDART_INF_F : (F8 ? found * turn_back : found) * back;
            }
        }
    } while (next_head(here));
    cp_async_wait<0>();
}

// ---- select -------------------------------------------------------------------
//
// One block per (request, key-value head).  Scores become whole numbers of the same order, forced pages the
// greatest.  The last one wanted of the others lies among fewer and fewer keys: those that agree with it in a digit
// (8 bits each, from the highest bit in which two of them differ), until they are few enough to be compared with one
// another.  The pages above it, with the first ones equal to it, are written in order.  Trips to memory, barriers and
// chains of instructions bound it: a thread has up to 8 keys in registers from one trip, a warp consecutive ones.
// (Keys in shared memory and four digits: 8.5 instead of 5.6 us for 4 heads of 2048 pages, 17 instead of 12.1 for
// 1024 heads of up to as many.)
constexpr int kSelectItems = 8;             // keys of a thread; more pages go in turns, read again each time
constexpr int kSelectGroup = 2;             // and those that are gone through without a branch
constexpr int kSelectRank = 128;            // keys that are compared with one another

// Keys of no page, and of a forced one.
constexpr uint32_t kNone = 0u, kForced = 0xffffffffu;
// Scores in ascending order; NaN above all, -0 like 0.
__device__ __forceinline__ uint32_t key_of(float s) { return s != s ? kForced - 1 : ordered_key(s); }

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) page_select_kernel(const __grid_constant__ SelectArgs a) {
    constexpr int kWarps = THREADS / 32, kTurn = THREADS * kSelectItems;
    __shared__ __align__(16) uint32_t list[kSelectRank];
    __shared__ uint32_t hist[256], found[4];
    // two arrays: with all the others' keys equal no barrier lies between the last read of `ends` and the counts
    __shared__ uint32_t ends[2][kWarps], counts[2][kWarps];
    pdl_allow_dependents();
    pdl_wait_primary();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, unit = blockIdx.x, b = unit / a.heads, keep = a.keep;
    const int n = tokens_of(a, b), pages = pages_of(n, a.page_size), kept = min(keep, pages);
    const float* scores = a.scores + (long long)unit * a.max_pages;
    const int32_t* row = a.table + b * a.table_ld;
    int32_t* out = a.tables + (long long)unit * keep;
    // whole pages but for the last one, if that is among them
    if (tid == 0) a.lens[unit] = pages <= keep ? n : kept * a.page_size;
    for (int i = kept + tid; i < keep; i += THREADS) out[i] = -1;
    if (pages <= keep) {
        for (int i = tid; i < pages; i += THREADS) out[i] = row[i];
        return;
    }
    // A turn's pages from `base` on, equally many of them in a row to each warp: item j of the thread is page first + 32 j.
    uint32_t k[kSelectItems];
    int first = 0, items = 0;
    auto load = [&](int base) {
        items = (min(pages - base, kTurn) + THREADS - 1) / THREADS;
        first = base + warp * 32 * items + lane;
        const int end = min(pages, base + kTurn);
        float f[kSelectItems];
#pragma unroll
        for (int j = 0; j < kSelectItems; ++j) f[j] = j < items && first + 32 * j < end ? scores[first + 32 * j] : 0.0f;
#pragma unroll
        for (int j = 0; j < kSelectItems; ++j) {
            if (j % kSelectGroup == 0 && j >= items) break;
            const int i = first + 32 * j;
            k[j] = j >= items || i >= end ? kNone : i < a.sinks || i >= pages - a.recent ? kForced : key_of(f[j]);
        }
    };
    const bool turns = pages > kTurn;
    // f() for every turn, with its keys
    auto each = [&](auto f) {
        for (int base = 0; base < pages; base += kTurn) {
            if (turns) load(base);
            f();
        }
    };
    if (!turns) load(0);
    uint32_t low = kForced, high = 0u;      // of the others
    each([&] {
#pragma unroll
        for (int j = 0; j < kSelectItems; ++j) {
            if (j % kSelectGroup == 0 && j >= items) break;
            if (k[j] == kNone || k[j] == kForced) continue;
            low = min(low, k[j]);
            high = max(high, k[j]);
        }
    });
    __syncwarp();
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) {
        ends[0][warp] = low;
        ends[1][warp] = high;
    }
    if (tid < 256) hist[tid] = 0;
    if (tid == 0) found[3] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        low = min(low, ends[0][w]);
        high = max(high, ends[1][w]);
    }
    // The `candidates` keys in question agree with `value` from bit `bits` on; `need` of the greatest of them are wanted.
    const int must = a.sinks + a.recent;
    int bits = must < keep ? 32 - __clz(low ^ high) : 0;
    uint32_t value = must == keep ? kForced - 1 : bits == 32 ? 0u : high >> bits << bits, need = keep - must, candidates = pages - must;
    auto in_question = [&](uint32_t key) { return key != kNone && key != kForced && (bits == 32 || (key ^ value) >> bits == 0); };
    while (bits > 0 && candidates > kSelectRank) {
        const int take = min(bits, 8), shift = bits - take;
        each([&] {
#pragma unroll
            for (int j = 0; j < kSelectItems; ++j) {
                if (j % kSelectGroup == 0 && j >= items) break;
                if (in_question(k[j])) atomicAdd(hist + (k[j] >> shift & ((1u << take) - 1u)), 1u);
            }
        });
        __syncthreads();
        // one warp looks for the digit, 8 to a lane, the greatest ones in lane 0
        if (warp == 0) {
            uint32_t h[8], mine = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] = hist[255 - 8 * lane - i];
                hist[255 - 8 * lane - i] = 0;
                mine += h[i];
            }
            uint32_t above = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, above, o);
                if (lane >= o) above += u;
            }
            above -= mine;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (above < need && above + h[i] >= need) {
                    found[0] = 255 - 8 * lane - i;
                    found[1] = above;
                    found[2] = h[i];
                }
                above += h[i];
            }
        }
        __syncthreads();
        value |= found[0] << shift;
        need -= found[1];
        candidates = found[2];
        bits = shift;
    }
    if (bits > 0) {
        each([&] {
            uint32_t in[kSelectItems], all = 0, at = 0;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kSelectItems; ++j) {
                if (j % kSelectGroup == 0 && j >= items) break;
                in[j] = __ballot_sync(0xffffffffu, in_question(k[j]));
                all += __popc(in[j]);
            }
            if (lane == 0 && all) at = atomicAdd(found + 3, all);
            at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
            for (int j = 0; j < kSelectItems; ++j) {
                if (j % kSelectGroup == 0 && j >= items) break;
                if (in[j] >> lane & 1u) list[at + __popc(in[j] & ((1u << lane) - 1u))] = k[j];
                at += __popc(in[j]);
            }
        });
        __syncthreads();
        if (warp * 32 < (int)candidates) {
            const uint32_t mine = tid < (int)candidates ? list[tid] : kNone;
            uint32_t greater = 0, equal = 0;
            for (uint32_t i = 0; i < candidates; i += 4) {
                const uint4 o = *reinterpret_cast<const uint4*>(list + i);
                const uint32_t other[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    greater += i + e < candidates && other[e] > mine;
                    equal += i + e < candidates && other[e] == mine;
                }
            }
            if (tid < (int)candidates && greater < need && greater + equal >= need) {
                found[0] = mine;           // the same for all that are equal
                found[1] = greater;
            }
        }
        __syncthreads();
        value = found[0];
        need -= found[1];
    }
    // `need` pages of key `value`, the first ones, and all above: a warp writes behind what the warps before it do
    uint32_t above = 0, equal = 0;          // in the turns before
    each([&] {
        int32_t entry[kSelectItems];
        uint32_t more[kSelectItems], same[kSelectItems], n_more = 0, n_same = 0;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kSelectItems; ++j) {
            if (j % kSelectGroup == 0 && j >= items) break;
            entry[j] = k[j] >= value && k[j] != kNone ? row[first + 32 * j] : 0;
            more[j] = __ballot_sync(0xffffffffu, k[j] > value);
            same[j] = __ballot_sync(0xffffffffu, k[j] == value);
            n_more += __popc(more[j]);
            n_same += __popc(same[j]);
        }
        if (turns) __syncthreads();         // the counts before have been read
        if (lane == 0) {
            counts[0][warp] = n_more;
            counts[1][warp] = n_same;
        }
        __syncthreads();
        uint32_t up = above, eq = equal;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            above += counts[0][w];
            equal += counts[1][w];
            if (w < warp) {
                up += counts[0][w];
                eq += counts[1][w];
            }
        }
        const uint32_t before = (1u << lane) - 1u;
#pragma unroll
        for (int j = 0; j < kSelectItems; ++j) {
            if (j % kSelectGroup == 0 && j >= items) break;
            const uint32_t e = eq + __popc(same[j] & before);
            if ((more[j] >> lane & 1u) || ((same[j] >> lane & 1u) && e < need)) {
                out[up + __popc(more[j] & before) + min(e, need)] = entry[j];
                if (first + 32 * j == pages - 1) a.lens[unit] = n - (pages - keep) * a.page_size;
            }
            up += __popc(more[j]);
            eq += __popc(same[j]);
        }
    });
}

template <bool F8, int JC>
cudaError_t launch_scores_as(const ScoresArgs& a, cudaStream_t s) {
    using K = Scores<F8, JC>;
    static std::atomic<uint64_t> done;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(page_scores_kernel<F8, JC>), K::kSmem, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(page_scores_kernel<F8, JC>, dim3((unsigned)(K::kBlocksPerSm * device_sm_count())), dim3(kScoreThreads),
                      K::kSmem, s, a);
}

}  // namespace

cudaError_t launch_page_bounds(const BoundsArgs& a, cudaStream_t s) {
    auto kern = a.c.dtype == MOE_DTYPE_FP8_E4M3 ? page_bounds_kernel<true> : page_bounds_kernel<false>;
    return launch_pdl(kern, dim3((unsigned)(kBoundsBlocks * device_sm_count())), dim3(kBoundsThreads), 0, s, a);
}

cudaError_t launch_page_scores(const ScoresArgs& a, cudaStream_t s) {
    const int D = a.c.head_dim;
    if (a.c.dtype == MOE_DTYPE_FP8_E4M3)
        return D <= 64 ? launch_scores_as<true, 2>(a, s) : D <= 128 ? launch_scores_as<true, 4>(a, s) : launch_scores_as<true, 8>(a, s);
    return D <= 32 ? launch_scores_as<false, 2>(a, s)
           : D <= 64 ? launch_scores_as<false, 4>(a, s)
           : D <= 128 ? launch_scores_as<false, 8>(a, s) : launch_scores_as<false, 16>(a, s);
}

cudaError_t launch_page_select(const SelectArgs& a, cudaStream_t s) {
    const int blocks = a.B * a.heads;
    // More than 2048 pages: blocks that have them all in a turn (or many of them), but no more threads than the SMs hold at
    // once.  4 heads of 8192 pages 20.5, 14.5 and 10.4 us with 256, 512 and 1024 threads, 256 heads of 4096 18.7, 9.9
    // and 18.6, 1024 heads of up to 2048 13.4, 22.3 with 256 and 512.
    const int sms = device_sm_count();
    if (a.max_pages > 512 * kSelectItems && blocks <= sms)
        return launch_pdl(page_select_kernel<1024>, dim3((unsigned)blocks), dim3(1024), 0, s, a);
    if (a.max_pages > 256 * kSelectItems && blocks <= 2 * sms)
        return launch_pdl(page_select_kernel<512>, dim3((unsigned)blocks), dim3(512), 0, s, a);
    return launch_pdl(page_select_kernel<256>, dim3((unsigned)blocks), dim3(256), 0, s, a);
}

}  // namespace moe
