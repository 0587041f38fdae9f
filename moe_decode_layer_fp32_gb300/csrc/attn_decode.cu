// Attention of one new token per request over the paged cache.
//
// Mathematics.  For a head with scores s_j and values v_j a part of the keys is
// summed up by (m, l, o): m = max s_j, l = sum e^(s_j - m), o = sum e^(s_j - m) v_j;
// two parts join as m = max(m1, m2), l = l1 e^(m1 - m) + l2 e^(m2 - m), o alike, and
// the result is o / l.  Scores are kept in base 2 (s log2 e), so that every
// exponential is one exp2.
//
// Split.  The cache is read once and there are 4 to 16 multiply-adds per value
// read: memory bounds it, so the keys of all (request, key-value head) units are
// laid end to end in tiles, every CTA takes an equal run of them whatever the
// requests' lengths, and the parts of a unit that several CTAs share go through
// the workspace: the CTA that finishes last joins them, in an order that does not
// depend on which one that is.
//
// In a CTA every warp works alone on its own keys of a tile (its own cp.async ring,
// running maximum and sum); the warps join only where a unit ends.  All query heads
// of a key-value head share its rows: they are the rows of the 16-row MMA tile.
// With up to 8 heads the other 8 rows hold the second term of each value: q (when
// fp32) and the weights p enter as sums of two or three terms of the cache's
// 16-bit type (f16 for E4M3, which holds its values), which keeps them to 16 bits and
// more at no cost in MMAs; bf16 queries over an E4M3 cache as two E4M3 terms.
//
// Measured: 1 x 131071 keys of 8 heads of 128, bf16 (537 MB) 87 us, 6.1 TB/s; 128
// requests of 1 to 4096 keys, bf16 137 us, 6.3 TB/s, and E4M3 95 us, 4.6 TB/s: there the
// chains of dependent instructions bound it, about 750 for a warp's 32 keys, which a scheduler's two
// warps (255 registers each) issue at 0.35 a clock (105 us with a mask or shift more per conversion).
// Two CTAs per SM with a ring of three stages beat three with two (64 x 2048 keys: bf16 91 and 98 us,
// E4M3 58 and 66) and tiles of 16 keys (E4M3 69).
//
// Beyond 128 columns o, the scores and q do not fit the registers (124 to 960 bytes of spills) and a bf16
// cache leaves one CTA to an SM: 64 x 2048 keys of 4 heads of 256, 16 query heads, bf16 102 us (77 % of
// the cache's bytes at the copy rate), fp32 q 264, over E4M3 90 and 73.  More than 8 query heads of a key-value head
// are one unit of 16 rows up to 128 columns without extra terms; otherwise every 8 of them are a unit of
// their own and read the keys again: 64 / 4 heads of 128, bf16 54 us, fp32 q 92, over E4M3 49 and 59.
#include <algorithm>

#include <math_constants.h>

#include "block.h"

namespace moe {

namespace {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kAttnMaxCtas = 320;          // bounds the workspace
constexpr int kJoinMost = 24;              // parts joined by one CTA; more go in groups of kJoinGroup first
constexpr int kJoinGroup = 16;
// What a tile and the beginning and end of a unit cost.  Unit costs of 1, 3, 5 and 8: 204, 137, 136, 136 us
// for 128 ragged bf16 requests in order of length, 134, 92, 94, 98 for E4M3 with a cap, 10.2, 10.1, 10.8,
// 12.0 for one request of 777 keys.
constexpr int kTileCost = 2, kUnitCost = 3;
// The fast tanh is off by 2^-22 of the cap: up to 256, 2^-14 of a weight, where a bf16 output is rounded to
// 2^-9.  Larger caps take the kernel of fp32 outputs, with tanhf (64 x 2048 keys, bf16 91 and 94 us, E4M3 60
// and 60; with 16 heads to a key-value head, which that kernel takes in two parts, 96 and 181, 88 and 110).
constexpr float kFastCap = 256.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A 16 x 32 by 32 x 8, E4M3 into fp32.
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bytes, or zeros where size is 0 (src is then not read).
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, uint32_t size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
// 2^x to about 2^-22 relative; results below 2^-126 become 0.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// tanh(x) = 1 - 2 / (1 + e^2x), to about 2^-22 of 1 (not of small results).  Large x: the division
// gives 0 from a divisor of 2^126 on, an infinite one included; NaN stays NaN.
__device__ __forceinline__ float tanh_fast(float x) {
    return 1.0f - __fdividef(2.0f, 1.0f + exp2_fast(2.0f * kLog2e * x));
}
// bf16 parts by truncation: p = hi + rest exactly, rest of p's sign.
__device__ __forceinline__ float bf16_trunc(float p) { return __uint_as_float(__float_as_uint(p) & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_hi(float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632); }

// Where a CTA (or one of its warps) stands.
struct Cursor {
    int b, unit, tile, tiles, first, n;
    int last;                              // tiles of the unit that begin before the run's end
    const int32_t* row;                    // the request's row of the block table
    long long base;                        // where the unit begins in the line of all units
};
// Of a unit of so many tiles.
__device__ __forceinline__ int span_of(int tiles) { return tiles > 0 ? kTileCost * tiles + kUnitCost : 0; }
// Tiles of the cursor's unit that begin before position p.
__device__ __forceinline__ int tiles_before(const Cursor& c, long long p) {
    const long long n = p - c.base - kUnitCost;
    return n <= 0 ? 0 : (int)min((n + kTileCost - 1) / kTileCost, (long long)c.tiles);
}
// Whether the cursor's tile is one of the run.
__device__ __forceinline__ bool inside(const Cursor& c) { return c.tile < c.last; }

// x / y for 0 <= x, 0 < y; 64-bit division only where it must be.
__device__ __forceinline__ long long div_u(long long x, long long y) {
    if (((unsigned long long)(x | y) >> 32) == 0) return (uint32_t)x / (uint32_t)y;
    return x / y;
}
// CTA k of `ctas` <= total takes the tiles from k total / ctas on.
struct Share {
    long long ctas, total;
    __device__ Share(long long c, long long t) : ctas(c), total(t) {}
    __device__ long long start(long long k) const { return div_u(k * total, ctas); }
    // the largest k with start(k) <= u
    __device__ int cta_of(long long u) const { return (int)div_u((u + 1) * ctas - 1, total); }
};

// DP: head_dim rounded up to 64, 128 or 256.  F8: E4M3 cache.  ROWS: query heads of a
// unit, 8 or 16.  EX: fp32 queries or output, or a large cap: terms keep 22 bits or more.
template <int DP, bool F8, int ROWS, bool EX>
struct Attn {
    static constexpr int kElem = F8 ? 1 : 2;
    static constexpr int kPitch = DP * kElem;                        // bytes of a row in shared memory
    static constexpr int KT = kPitch <= 128 ? 32 : 16;               // keys of a warp's tile
    static constexpr int kTileBytes = KT * kPitch;                   // K or V
    static constexpr int kTileShift = KT == 32 ? 7 : 6;
    static constexpr int kTileKeys = KT * kAttnWarps;
    static_assert(kTileKeys == 1 << kTileShift, "tiles counted by a shift");
    static constexpr uint32_t kAllKeys = KT == 32 ? 0xffffffffu : (1u << (KT % 32)) - 1u;
    static constexpr int kChunks = kPitch / 16;                      // 16-byte chunks of a row
    static constexpr int kRowsPerIter = 32 / kChunks;
    // bf16 queries over an E4M3 cache: q is two E4M3 terms (4 bits each, its 8) and the codes of K go
    // into the MMA as they are
    static constexpr bool kQ8 = F8 && !EX;
    static constexpr int kQTerms = EX ? (F8 ? 2 : 3) : kQ8 ? 2 : 1;
    static constexpr int kPTerms = EX && !F8 ? 3 : 2;
    static constexpr int kSteps = kQ8 ? DP / 32 : DP / 16;           // MMAs of q . k along d
    static constexpr int kVElems = F8 ? (DP >= 128 ? 16 : 8) : 8;    // columns a thread takes of a V row at once
    static constexpr int kWindows = DP / (8 * kVElems);
    static constexpr int kAccs = DP / 8;                             // n8 tiles of o
    // The running maximum is replaced only when the new one passes it by more than 2^kSlack:
    // until then weights may be up to that, and o needs no rescaling (which most tiles
    // would, for the sake of one of their heads).  p in f16 is scaled to use its range: 2^7
    // at the maximum, 2^15 with the slack.
    static constexpr float kSlack = 8.0f;
    static constexpr float kLeast = 0x1p-126f;                       // bf16's least normal number, and two of it
    static constexpr uint32_t kLeast2 = 0x00800080u;
    static constexpr float kPShift = F8 ? 7.0f : 0.0f;
    static constexpr int kCtasPerSm = kTileBytes > 4096 ? 1 : 2;
    static constexpr int kStages = 3;
    static constexpr size_t kRing = (size_t)kAttnWarps * kStages * 2 * kTileBytes;
    static constexpr int kQBytes = ROWS * DP * (EX ? 4 : 2);         // a unit's query rows
    static constexpr size_t kSmem = kRing + 2 * kQBytes;
    static_assert(ROWS * DP * 4 <= 2 * kTileBytes, "a warp's o fits the stage it read last");
    static constexpr int kPartFloats = ROWS * (DP + 2);
    static_assert(ROWS == 8 || (ROWS == 16 && !EX), "16 heads only without extra terms");

    // Byte offset of chunk `ch` of row `r` in a K or V tile; the chunks of a
    // 128-byte line are permuted so that the readers below (8 rows x 4 chunks of K, 4
    // rows of one parity x 2 chunks of V) hit distinct banks.
    __device__ static __forceinline__ uint32_t at_k(int r, int ch) {
        if constexpr (kPitch == 64) return (r >> 1) * 128 + ((((r & 1) * 4 + ch) ^ (2 * ((r >> 1) & 3))) << 4);
        return r * kPitch + ((ch ^ ((r & 1) << 2)) << 4);
    }
    __device__ static __forceinline__ uint32_t at_v(int r, int ch) {
        if constexpr (kPitch == 64) return at_k(r, ch);
        return r * kPitch + ((ch ^ (r & 6)) << 4);
    }
    // The lane's offsets within a stage, from which every address of a tile is a constant away.
    struct Lane {
        uint32_t k[2];     // reads K row lane / 4, chunk lane % 4, and the chunk 4 further on (in the permuted order)
        uint32_t v[2];     // reads V row 2 (lane % 4) [+ 1], its chunk (8-byte piece) lane / 4
        uint32_t wk, wv;   // writes row lane / kChunks, chunk lane % kChunks
        __device__ __forceinline__ explicit Lane(int lane) {
            const int row = lane / 4, col = lane % 4;
            k[0] = at_k(row, col);
            k[1] = kChunks > 4 ? at_k(row, 4 + col) : k[0];
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * col + e;
                v[e] = kTileBytes + (kVElems * kElem == 16 ? at_v(r, row) : at_v(r, row / 2) + (row % 2) * 8);
            }
            wk = at_k(lane / kChunks, lane % kChunks);
            wv = kTileBytes + at_v(lane / kChunks, lane % kChunks);
        }
    };

    __device__ static __forceinline__ void set_request(const AttnArgs& a, Cursor& c) {
        int n = max(a.seq_lens[c.b], 0);
        n = (int)min((long long)n, (long long)a.max_pages * a.c.page_size);
        c.n = n;
        c.first = a.window > 0 ? max(0, n - a.window) : 0;
        c.tiles = ((n - c.first - 1) >> kTileShift) + 1;     // without a sum that may pass 2^31; 0 for no keys
        c.row = a.table + c.b * a.table_ld;
    }
    // To the next tile; where none begins before `end`, to none of the run.
    __device__ static __forceinline__ void advance(const AttnArgs& a, int units, long long end, Cursor& c) {
        if (++c.tile < c.tiles) return;
        c.base += span_of(c.tiles);
        c.tile = 0;
        c.last = 0;
        if (c.base >= end) return;
        if (++c.unit == units) {
            c.unit = 0;
            do {
                ++c.b;
                set_request(a, c);
            } while (c.tiles == 0);
        }
        c.last = tiles_before(c, end);
    }
    // Page and slot of the key that lane `lane` looks after in the warp's tile; page -1: none.
    __device__ static __forceinline__ int2 place_of(const AttnArgs& a, const Cursor& c, int warp, int lane) {
        // unsigned: the end of the last tile may lie beyond 2^31
        const uint32_t at = (uint32_t)c.first + (uint32_t)c.tile * kTileKeys + warp * KT + lane;
        if (!inside(c) || lane >= KT || at >= (uint32_t)c.n) return make_int2(-1, 0);
        const int key = (int)at;
        const int col = a.page_shift >= 0 ? key >> a.page_shift : key / a.c.page_size;
        const int page = c.row[col];
        if (page < 0 || page >= a.c.num_pages) {
            set_status(a.status, MOE_ERR_DEVICE);
            return make_int2(-1, 0);
        }
        return make_int2(page, key - col * a.c.page_size);
    }
    // Start the copies of the warp's K and V rows of tile c into a stage; returns the
    // mask of the keys that count.  The rows of the others become zeros.
    __device__ static __forceinline__ uint32_t issue(const AttnArgs& a, const Cursor& c, int2 place, int nsub, int lane,
                                                     const Lane& ln, uint32_t stage) {
        const int g = nsub == 1 ? c.unit : c.unit / nsub;
        const uint32_t mask = __ballot_sync(0xffffffffu, place.x >= 0);
        if (mask == 0u) return 0u;   // nobody reads the stage
        // offsets in 16-byte steps: 32 bits of them unless a cache tensor passes 64 GB
        long long ko = 0, vo = 0;
        if (place.x >= 0) {
            ko = (place.x * a.c.k_page_stride + place.y * a.c.k_slot_stride + g * a.c.k_head_stride) / (16 / kElem);
            vo = (place.x * a.c.v_page_stride + place.y * a.c.v_slot_stride + g * a.c.v_head_stride) / (16 / kElem);
        }
        const int ch = lane % kChunks, r0 = lane / kChunks;
        const uint32_t in = ch * 16 < a.c.head_dim * kElem ? 16u : 0u;
        const char* kb = static_cast<const char*>(a.c.k) + ch * 16;
        const char* vb = static_cast<const char*>(a.c.v) + ch * 16;
        // row i kRowsPerIter + r0: the permutations differ from row r0's by a constant per i
        auto copy = [&](int i, long long o, long long p, uint32_t size) {
            const int r = i * kRowsPerIter;
            const uint32_t fk = kPitch == 512 ? (r & 1) << 6 : 0, fv = kPitch > 64 ? (r & 6) << 4 : 0;
            cp_async16_zfill(stage + (ln.wk ^ fk) + r * kPitch, kb + o * 16, size);
            cp_async16_zfill(stage + ((ln.wv - kTileBytes) ^ fv) + kTileBytes + r * kPitch, vb + p * 16, size);
        };
        if (mask == kAllKeys && !a.far) {
#pragma unroll
            for (int i = 0; i < KT / kRowsPerIter; ++i) {
                const int r = i * kRowsPerIter + r0;
                const uint32_t o = __shfl_sync(0xffffffffu, (uint32_t)ko, r), p = __shfl_sync(0xffffffffu, (uint32_t)vo, r);
                copy(i, o, p, in);
            }
        } else {
#pragma unroll
            for (int i = 0; i < KT / kRowsPerIter; ++i) {
                const int r = i * kRowsPerIter + r0;
                const long long o = __shfl_sync(0xffffffffu, ko, r), p = __shfl_sync(0xffffffffu, vo, r);
                copy(i, o, p, (mask >> r) & 1u ? in : 0u);
            }
        }
        return mask;
    }

    struct State {
        uint32_t q[kQTerms][ROWS / 8][kSteps][2];   // terms of q: A fragments of the thread's row(s)
        float qf[ROWS / 8];                         // factor of the accumulated score (base 2)
        float m[ROWS / 8], l[ROWS / 8];
        float o[kAccs][4];
    };

    __device__ static __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
        if constexpr (F8) mma_f16(c, a0, a1, a2, a3, b0, b1);
        else mma_bf16(c, a0, a1, a2, a3, b0, b1);
    }

    // Copies of a unit's query rows into shared memory, as they are.
    __device__ static __forceinline__ void fetch_q(const AttnArgs& a, const Cursor& c, int nsub, char* dst) {
        const int g = c.unit / nsub, sub = c.unit % nsub;
        const int es = a.q_dt == MOE_DTYPE_BF16 ? 2 : 4, per_row = a.c.head_dim * es / 16;   // 16-byte words
        const long long base = c.b * a.q_bs + (g * a.group + sub * ROWS) * a.q_hs;
        const int rows = min(ROWS, a.group - sub * ROWS);
        for (int i = threadIdx.x; i < rows * per_row; i += kAttnThreads) {
            const int r = i / per_row, w = i - r * per_row;
            cp_async16(dst + r * DP * es + w * 16, static_cast<const char*>(a.q) + (base + r * a.q_hs) * es + w * 16);
        }
        cp_async_commit();
    }
    // The unit's query rows: the thread holds rows lane / 4 (and + 8), elements
    // 8 (lane % 4) + {0..7} of every 32 (bf16), 16 (lane % 4) + {0..15} of every 64 (E4M3): the order
    // in which it reads K rows; a dot product does not mind the order.
    __device__ static void load_q(const AttnArgs& a, const Cursor& c, int nsub, int lane, const char* src, State& st) {
        const int g = c.unit / nsub, sub = c.unit % nsub;
        const float ks = a.c.k_scale ? a.c.k_scale[g] : 1.0f;
        constexpr int E = F8 ? 16 : 8, J = DP / (4 * E);
#pragma unroll
        for (int rr = 0; rr < ROWS / 8; ++rr) {
            const int row = rr * 8 + lane / 4;
            const bool have = sub * ROWS + row < a.group;
            float f[J][E];
            float mx = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int h = 0; h < E / 8; ++h) {
                    const int d0 = j * 4 * E + (lane % 4) * E + h * 8;
                    float v[8] = {};
                    if (have && d0 < a.c.head_dim) load8_f32(src, a.q_dt, row * DP + d0, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        f[j][h * 8 + e] = v[e];
                        mx = fmaxf(mx, fabsf(v[e]));
                    }
                }
            float back = 1.0f;
            if constexpr (F8) {
                // f16 terms: the row is scaled by a power of two to at most 2^8
                __syncwarp();
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                int e = 0;
                if (mx > 0.0f && mx < CUDART_INF_F) frexpf(mx, &e);
                e = min(8 - e, 126);             // 8 - e >= -120: both factors are normal numbers
                const float up = ldexpf(1.0f, e);
                back = ldexpf(1.0f, -e);
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < E; ++i) f[j][i] *= up;
            }
            st.qf[rr] = a.scale * (ks * back);   // in this order: a small scale of k goes with a large q
            if constexpr (kQ8) {
                // E4M3 has no infinity: a head with one gets NaN
                if (mx == CUDART_INF_F) st.qf[rr] = CUDART_NAN_F;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float* u = &f[s / 2][(s % 2) * 8 + h * 4];
                            const uint32_t w = pack_e4m3x4(u[0], u[1], u[2], u[3]);
                            const float2 lo = unpack_e4m3x2<false>(w), hi = unpack_e4m3x2<true>(w);
                            u[0] = (u[0] - lo.x) * 16.0f;
                            u[1] = (u[1] - lo.y) * 16.0f;
                            u[2] = (u[2] - hi.x) * 16.0f;
                            u[3] = (u[3] - hi.y) * 16.0f;
                            st.q[t][rr][s][h] = w;
                        }
            }
#pragma unroll
            for (int t = 0; t < (kQ8 ? 0 : kQTerms); ++t)
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const int j = s / (E / 4) % J, i = (s % (E / 4)) * 4;
                    uint32_t w[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float &u = f[j][i + 2 * h], &v = f[j][i + 2 * h + 1];
                        if constexpr (F8) {
                            w[h] = pack_f16x2(u, v);
                            const float2 r = unpack_f16x2(w[h]);
                            u -= r.x;
                            v -= r.y;
                        } else {
                            w[h] = pack_hi(u, v);
                            u -= bf16_trunc(u);
                            v -= bf16_trunc(v);
                        }
                    }
                    st.q[t][rr][s][0] = w[0];
                    st.q[t][rr][s][1] = w[1];
                }
            st.m[rr] = -CUDART_INF_F;
            st.l[rr] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kAccs; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[i][e] = 0.0f;
    }

    // One tile: scores, running maximum, weights, o.
    __device__ static __forceinline__ void tile(const AttnArgs& a, State& st, uint32_t stage, const Lane& ln, uint32_t mask, int lane) {
        constexpr int NT = KT / 8;
        const int col = lane % 4;
        float s[NT][ROWS / 8][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // c: first terms (rows 0-7) and second terms or heads 8-15 (rows 8-15); c2: third terms
            float c[4] = {}, c2[4] = {};
#pragma unroll
            for (int j = 0; j < kChunks / 4; ++j) {
                // row 8 nt + lane / 4, chunk 4 j + lane % 4
                const uint4 k4 = lds128(stage + ln.k[j & 1] + nt * 8 * kPitch + (j >> 1) * 128);
                const uint32_t w[4] = {k4.x, k4.y, k4.z, k4.w};
                if constexpr (kQ8) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t(&q0)[2] = st.q[0][0][j * 2 + i];
                        const uint32_t(&q1)[2] = st.q[1][0][j * 2 + i];
                        if constexpr (ROWS == 16) {
                            const uint32_t(&r0)[2] = st.q[0][1][j * 2 + i];
                            const uint32_t(&r1)[2] = st.q[1][1][j * 2 + i];
                            mma_e4m3(c, q0[0], r0[0], q0[1], r0[1], w[2 * i], w[2 * i + 1]);
                            mma_e4m3(c2, q1[0], r1[0], q1[1], r1[1], w[2 * i], w[2 * i + 1]);
                        } else {
                            mma_e4m3(c, q0[0], q1[0], q0[1], q1[1], w[2 * i], w[2 * i + 1]);
                        }
                    }
                    continue;
                }
                constexpr int SJ = F8 ? 4 : 2;
#pragma unroll
                for (int i = 0; i < SJ; ++i) {
                    const int step = j * SJ + i;
                    uint32_t b0, b1;
                    if constexpr (F8) {
                        b0 = e4m3x2_to_f16x2<false>(w[i]);
                        b1 = e4m3x2_to_f16x2<true>(w[i]);
                    } else {
                        b0 = w[2 * i];
                        b1 = w[2 * i + 1];
                    }
                    const uint32_t* q0 = st.q[0][0][step];
                    if constexpr (ROWS == 16) {
                        const uint32_t* q1 = st.q[0][1][step];
                        mma(c, q0[0], q1[0], q0[1], q1[1], b0, b1);
                    } else if constexpr (kQTerms == 1) {
                        mma(c, q0[0], 0u, q0[1], 0u, b0, b1);
                    } else {
                        const uint32_t* q1 = st.q[1][0][step];
                        mma(c, q0[0], q1[0], q0[1], q1[1], b0, b1);
                        if constexpr (kQTerms == 3) {
                            const uint32_t* q2 = st.q[2][0][step];
                            mma(c2, q2[0], 0u, q2[1], 0u, b0, b1);
                        }
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[nt][0][e] = c[e];
                if constexpr (kQ8) {
                    s[nt][0][e] = fmaf(ROWS == 16 ? c2[e] : c[2 + e], 0.0625f, c[e]);
                    if constexpr (ROWS == 16) s[nt][1][e] = fmaf(c2[2 + e], 0.0625f, c[2 + e]);
                } else if constexpr (ROWS == 16) s[nt][1][e] = c[2 + e];
                // an infinite first term stands: the others' products with it may be NaN
                else if (kQTerms > 1 && fabsf(c[e]) < CUDART_INF_F) s[nt][0][e] = c[e] + (c[2 + e] + c2[e]);
            }
        }
        uint32_t pf[kPTerms][NT][ROWS / 8];   // weights as A fragments: keys 2 col, + 1 of each n8 tile
#pragma unroll
        for (int rr = 0; rr < ROWS / 8; ++rr) {
            float mx = -CUDART_INF_F;
            if (a.softcap > 0.0f) {
                const float f = st.qf[rr] / a.softcap, cap = a.softcap * kLog2e;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        s[nt][rr][e] = cap * (EX ? tanhf(s[nt][rr][e] * f) : tanh_fast(s[nt][rr][e] * f));
            } else {
                const float f = st.qf[rr] * kLog2e;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) s[nt][rr][e] *= f;
            }
            if (mask != kAllKeys) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (!((mask >> (nt * 8 + 2 * col + e)) & 1u)) s[nt][rr][e] = -CUDART_INF_F;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(s[nt][rr][0], s[nt][rr][1]));
            __syncwarp();
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const bool raise = mx > st.m[rr] + kSlack;       // also from -inf
            if (__any_sync(0xffffffffu, raise)) {
                // rows that stay as they are have the factor 1
                const float corr = raise ? exp2_fast(st.m[rr] - mx) : 1.0f;
                if (raise) st.m[rr] = mx;
                st.l[rr] *= corr;
#pragma unroll
                for (int i = 0; i < kAccs; ++i) {
                    st.o[i][2 * rr] *= corr;
                    st.o[i][2 * rr + 1] *= corr;
                    if constexpr (ROWS == 8) {
                        st.o[i][2] *= corr;
                        st.o[i][3] *= corr;
                    }
                }
            }
            const float base = (st.m[rr] == -CUDART_INF_F ? 0.0f : st.m[rr]) - kPShift;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p0 = exp2_fast(s[nt][rr][0] - base), p1 = exp2_fast(s[nt][rr][1] - base);
                st.l[rr] += p0 + p1;
#pragma unroll
                for (int t = 0; t < kPTerms; ++t) {
                    if constexpr (F8) {
                        pf[t][nt][rr] = pack_f16x2(p0, p1);
                        const float2 r = unpack_f16x2(pf[t][nt][rr]);
                        p0 -= r.x;
                        p1 -= r.y;
                    } else if (!EX && t == 1) {
                        // 16 heads: both terms go into one sum, so that with an infinite v neither may be 0
                        pf[t][nt][rr] = ROWS == 16 ? pack_bf16x2(fmaxf(p0, kLeast), fmaxf(p1, kLeast)) : pack_bf16x2(p0, p1);
                    } else {
                        pf[t][nt][rr] = pack_hi(p0, p1);
                        p0 -= bf16_trunc(p0);
                        p1 -= bf16_trunc(p1);
                    }
                }
            }
        }
        // o += p v: the thread reads kVElems columns of its 4 keys of each 16 and pairs the
        // keys of a column; column (8 w + n) kVElems + e is column n of MMA tile (w, e)
#pragma unroll
        for (int w = 0; w < kWindows; ++w) {
            float fresh[EX ? kVElems : 1][4];
            if constexpr (EX) {
#pragma unroll
                for (int e = 0; e < kVElems; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) fresh[e][i] = 0.0f;
            }
#pragma unroll
            for (int kg = 0; kg < KT / 16; ++kg) {
                uint32_t v[4][4];   // keys 2 col, + 1, + 8, + 9
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // row 16 kg + 2 col + (i & 1) + 8 (i >> 1), chunk 8 w + lane / 4
                    const uint32_t at = stage + ln.v[i & 1] + (kg * 16 + (i >> 1) * 8) * kPitch + w * 128;
                    if constexpr (kVElems * kElem == 16) {
                        const uint4 u = lds128(at);
                        v[i][0] = u.x; v[i][1] = u.y; v[i][2] = u.z; v[i][3] = u.w;
                    } else {
                        const uint2 u = lds64(at);
                        v[i][0] = u.x; v[i][1] = u.y;
                    }
                }
                const uint32_t (&p0)[ROWS / 8] = pf[0][2 * kg];
                const uint32_t (&p0b)[ROWS / 8] = pf[0][2 * kg + 1];
#pragma unroll
                for (int e = 0; e < kVElems; ++e) {
                    uint32_t b[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (F8) {
                            const uint32_t x = __byte_perm(v[2 * h][e / 4], v[2 * h + 1][e / 4], (e & 2) ? 0x7362 : 0x5140);
                            b[h] = (e & 1) ? e4m3x2_to_f16x2<true>(x) : e4m3x2_to_f16x2<false>(x);
                        } else {
                            b[h] = __byte_perm(v[2 * h][e / 2], v[2 * h + 1][e / 2], (e & 1) ? 0x7632 : 0x5410);
                        }
                    }
                    float (&acc)[4] = EX ? fresh[EX ? e : 0] : st.o[w * kVElems + e];
                    if constexpr (ROWS == 16) {
                        mma(acc, p0[0], p0[1], p0b[0], p0b[1], b[0], b[1]);
                        mma(acc, pf[1][2 * kg][0], pf[1][2 * kg][1], pf[1][2 * kg + 1][0], pf[1][2 * kg + 1][1], b[0], b[1]);
                    } else {
                        mma(acc, p0[0], pf[1][2 * kg][0], p0b[0], pf[1][2 * kg + 1][0], b[0], b[1]);
                        // third terms beside the second ones; the least bf16 instead of 0 leaves the first
                        // terms' sum as it is, next to an infinite v too
                        if constexpr (kPTerms == 3)
                            mma(acc, kLeast2, pf[2][2 * kg][0], kLeast2, pf[2][2 * kg + 1][0], b[0], b[1]);
                    }
                }
            }
            if constexpr (EX) {
                // the tensor cores cut their sums to 24 bits instead of rounding: a tile's sum is
                // added to o with a rounded fp32 addition, so that the cuts do not add up
#pragma unroll
                for (int e = 0; e < kVElems; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) st.o[w * kVElems + e][i] += fresh[e][i];
            }
        }
    }

    struct Shared {
        float m[kAttnWarps][ROWS], l[kAttnWarps][ROWS];
        uint32_t mask[kAttnWarps][kStages];
        long long wsum[kAttnWarps];
        int found_b, last;
        long long found_pre;
    };

    // Result of a row: o / l, its value scale, and the log of the sum.
    __device__ static __forceinline__ void finish(const AttnArgs& a, int b, int g, int sub, int row, int c4, float4 o,
                                                  float m, float l) {
        const int r = sub * ROWS + row;
        if (r >= a.group || c4 * 4 >= a.c.head_dim) return;
        const int h = g * a.group + r;
        const float vs = a.c.v_scale ? a.c.v_scale[g] : 1.0f;
        // l == 0: no key counted
        const float inv = l == 0.0f ? 0.0f : vs / l;
        const long long i = b * a.o_bs + h * a.o_hs + c4 * 4;
        if (a.o_dt == MOE_DTYPE_BF16)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + i) =
                make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + i) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (a.lse && c4 == 0)
            a.lse[(long long)b * a.q_heads + h] = l == 0.0f ? -CUDART_INF_F : (m + log2f(l) - kPShift) * kLn2;
    }

    __device__ static __forceinline__ void axpy4(float4& acc, float f, float4 v) {
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
    }
    // 2^(m - top) for a part's maximum (0 for a part without keys)
    __device__ static __forceinline__ float weight_of(float m, float top) {
        return m == -CUDART_INF_F ? 0.0f : exp2f(m - top);
    }

    // The warps' results (sh.m, sh.l, and o of warp w at base + w * stride) become one: the unit's
    // result, or the part `to`.
    __device__ static void combine(const AttnArgs& a, const Cursor& c, int nsub, const char* base, int stride, Shared& sh,
                                   float* to) {
        const int g = c.unit / nsub, sub = c.unit % nsub;
        __syncthreads();
#pragma unroll 2
        for (int it = threadIdx.x; it < ROWS * (DP / 4); it += kAttnThreads) {
            const int row = it / (DP / 4), c4 = it % (DP / 4);
            float top = -CUDART_INF_F, l = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, sh.m[w][row]);
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float f = weight_of(sh.m[w][row], top);
                // a NaN sum has no maximum: it stays NaN
                l = fmaf(sh.l[w][row] != sh.l[w][row] ? 1.0f : f, sh.l[w][row], l);
                axpy4(o, f, reinterpret_cast<const float4*>(base + w * stride)[row * (DP / 4) + (c4 ^ (row & 7))]);
            }
            if (to) {
                reinterpret_cast<float4*>(to)[row * (DP / 4) + c4] = o;
                if (c4 == 0) {
                    to[ROWS * DP + row] = top;
                    to[ROWS * DP + ROWS + row] = l;
                }
            } else {
                finish(a, c.b, g, sub, row, c4, o, top, l);
            }
        }
        __syncthreads();
    }

    // Join what the warps have of a unit.  A warp's o goes to the stage that it read last
    // (base + warp * stride).
    __device__ static void merge(const AttnArgs& a, const Cursor& c, int nsub, State& st, char* base, int stride, Shared& sh,
                                 float* to) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int rr = 0; rr < ROWS / 8; ++rr) {
            float l = st.l[rr];
            __syncwarp();
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if (lane % 4 == 0) {
                sh.m[warp][rr * 8 + lane / 4] = st.m[rr];
                sh.l[warp][rr * 8 + lane / 4] = l;
            }
        }
        float4* mine = reinterpret_cast<float4*>(base + warp * stride);
#pragma unroll
        for (int w = 0; w < kWindows; ++w)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int colb = (8 * w + 2 * (lane % 4) + i) * kVElems;   // kVElems columns from here
#pragma unroll
                for (int rr = 0; rr < ROWS / 8; ++rr)
#pragma unroll
                    for (int e = 0; e < kVElems; e += 4) {
                        float v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float (&o)[4] = st.o[w * kVElems + e + k];
                            // an infinite sum of first terms stands: a second term may be 0, and its sum NaN
                            v[k] = ROWS == 16 ? o[2 * rr + i] : fabsf(o[i]) < CUDART_INF_F ? o[i] + o[2 + i] : o[i];
                        }
                        const int row = rr * 8 + lane / 4, f4 = (colb + e) / 4;
                        mine[row * (DP / 4) + (f4 ^ (row & 7))] = make_float4(v[0], v[1], v[2], v[3]);
                    }
            }
        combine(a, c, nsub, base, stride, sh, to);
    }

    // Join `count` parts, part_at(0), part_at(1), ..., in that order: a thread has the same elements of
    // all, with the loads of kBatch parts together (one trip to L2 for most units).  `to` may be one
    // of the parts: its maxima and sums are written when all have read them.
    template <class PartAt>
    __device__ static void join(const AttnArgs& a, const Cursor& c, int nsub, int count, PartAt part_at, Shared& sh, float* to) {
        constexpr int kBatch = 8;
        const int g = c.unit / nsub, sub = c.unit % nsub;
#pragma unroll 2
        for (int it = threadIdx.x; it < ROWS * (DP / 4); it += kAttnThreads) {
            const int row = it / (DP / 4), c4 = it % (DP / 4);
            float top = -CUDART_INF_F, l = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int k0 = 0; k0 < count; k0 += kBatch) {
                float pm[kBatch], pl[kBatch];
                float4 po[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    pm[k] = -CUDART_INF_F;
                    pl[k] = 0.0f;
                    po[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (k0 + k < count) {
                        const float* p = part_at(k0 + k);
                        po[k] = __ldcg(reinterpret_cast<const float4*>(p) + it);
                        pm[k] = __ldcg(p + ROWS * DP + row);
                        pl[k] = __ldcg(p + ROWS * DP + ROWS + row);
                    }
                }
                float mx = top;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) mx = fmaxf(mx, pm[k]);
                const float f0 = weight_of(top, mx);
                top = mx;
                // a NaN sum has no maximum: it stays NaN
                l *= l != l ? 1.0f : f0;
                o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const float f = weight_of(pm[k], top);
                    l = fmaf(pl[k] != pl[k] ? 1.0f : f, pl[k], l);
                    axpy4(o, f, po[k]);
                }
            }
            if (to) {
                reinterpret_cast<float4*>(to)[it] = o;
                if (c4 == 0) {
                    sh.m[0][row] = top;
                    sh.l[0][row] = l;
                }
            } else {
                finish(a, c.b, g, sub, row, c4, o, top, l);
            }
        }
        if (to) {
            __syncthreads();
            if (threadIdx.x < ROWS) {
                to[ROWS * DP + threadIdx.x] = sh.m[0][threadIdx.x];
                to[ROWS * DP + ROWS + threadIdx.x] = sh.l[0][threadIdx.x];
            }
            __syncthreads();
        }
    }

    // Whether this CTA is the last of `n` to arrive at the counter (which then is zero
    // again).  What the CTAs wrote before is visible to the last one after it.
    __device__ static bool arrive_last(uint32_t* counter, int n, Shared& sh) {
        __syncthreads();
        if (threadIdx.x == 0) {
            const bool last = atomic_add_acq_rel_gpu(counter, 1u) == (uint32_t)(n - 1);
            if (last) *counter = 0u;
            sh.last = last;
        }
        __syncthreads();
        return sh.last;
    }
};

template <int DP, bool F8, int ROWS, bool EX>
__global__ void __launch_bounds__(kAttnThreads, Attn<DP, F8, ROWS, EX>::kCtasPerSm) attn_kernel(const __grid_constant__ AttnArgs a) {
    using K = Attn<DP, F8, ROWS, EX>;
    extern __shared__ __align__(128) char smem[];
    __shared__ typename K::Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nsub = (a.group + ROWS - 1) / ROWS, units = a.c.heads * nsub;
    pdl_allow_dependents();
    pdl_wait_primary();

    // ---- the run of this CTA.  All units lie end to end, each with kUnitCost for its beginning and
    // end and kTileCost per tile; a CTA has the tiles that begin in its equal part of that.  The
    // part's first request is found with a scan of the requests in blocks of the CTA's threads.
    auto tiles_of = [&](int b) {
        Cursor c;
        c.b = b;
        K::set_request(a, c);
        return c.tiles;
    };
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
        for (int w = 0; w < kAttnWarps; ++w) {
            if (w < warp) incl += sh.wsum[w];
            all += sh.wsum[w];
        }
        return incl;
    };
    const int s0 = tid < a.B ? span_of(tiles_of(tid)) : 0;      // of the first block
    long long sum0, total;
    const long long incl0 = scan((long long)s0 * units, sum0);
    total = sum0;
    if (a.B > kAttnThreads) {
        long long mine = 0;
        for (int b = kAttnThreads + tid; b < a.B; b += kAttnThreads) mine += span_of(tiles_of(b));
        long long rest;
        __syncthreads();
        scan(mine * units, rest);
        total += rest;
    }
    if (blockIdx.x == 0) {
        for (int b = tid; b < a.B; b += kAttnThreads)
            if ((long long)max(a.seq_lens[b], 0) > (long long)a.max_pages * a.c.page_size) set_status(a.status, MOE_ERR_DEVICE);
    }
    // requests without keys
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (tiles_of(b) > 0) continue;
        for (int it = tid; it < units * ROWS * (DP / 4); it += kAttnThreads) {
            const int c4 = it % (DP / 4), row = it / (DP / 4) % ROWS, unit = it / (DP / 4) / ROWS;
            K::finish(a, b, unit / nsub, unit % nsub, row, c4, make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f, 0.0f);
        }
    }
    // parts of at least a whole tile and unit
    const Share share(min((long long)gridDim.x, div_u(total, kTileCost + kUnitCost)), total);
    if (blockIdx.x >= share.ctas) return;
    const long long start = share.start(blockIdx.x), end = share.start(blockIdx.x + 1);
    long long sum = 0, incl = incl0, all = sum0;
    int span = s0, b0 = 0;
    while (true) {
        const long long pre = sum + incl - (long long)span * units;
        if (start >= pre && start < sum + incl) {
            sh.found_b = b0 + tid;
            sh.found_pre = pre;
        }
        sum += all;
        if (start < sum) break;      // the same for all threads
        b0 += kAttnThreads;
        span = b0 + tid < a.B ? span_of(tiles_of(b0 + tid)) : 0;
        __syncthreads();
        incl = scan((long long)span * units, all);
    }
    __syncthreads();
    Cursor c;
    c.b = sh.found_b;
    K::set_request(a, c);
    c.unit = (int)div_u(start - sh.found_pre, span_of(c.tiles));
    c.base = sh.found_pre + (long long)c.unit * span_of(c.tiles);
    c.tile = tiles_before(c, start);
    c.last = tiles_before(c, end);
    if (c.tile == c.tiles) {            // the part begins with the end of a unit
        --c.tile;
        K::advance(a, units, end, c);
    }
    if (!inside(c)) return;

    // ---- pipeline: `ahead` runs K::kStages - 1 tiles in front of `c`
    const uint32_t ring = smem_u32(smem) + warp * K::kStages * 2 * K::kTileBytes;
    const typename K::Lane ln(lane);
    char* q_buf = smem + K::kRing;
    K::fetch_q(a, c, nsub, q_buf);
    Cursor ahead = c;
    int2 place = K::place_of(a, ahead, warp, lane);
    int stage_in = 0;
    auto feed = [&]() {
        if (inside(ahead)) {
            Cursor next = ahead;
            K::advance(a, units, end, next);
            const int2 place_next = K::place_of(a, next, warp, lane);
            const uint32_t mask = K::issue(a, ahead, place, nsub, lane, ln, ring + stage_in * 2 * K::kTileBytes);
            if (lane == 0) sh.mask[warp][stage_in] = mask;
            stage_in = stage_in + 1 == K::kStages ? 0 : stage_in + 1;
            ahead = next;
            place = place_next;
        }
        cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < K::kStages - 1; ++i) feed();

    int stage_out = 0, segment = 0;
    while (inside(c)) {
        // the query rows came with a group of copies before the last kStages - 2
        cp_async_wait<K::kStages - 2>();
        __syncthreads();
        typename K::State st;
        K::load_q(a, c, nsub, lane, q_buf + (segment & 1) * K::kQBytes, st);
        const Cursor seg = c;
        const int count = c.last - c.tile;
        {
            // the next unit's query rows
            Cursor next = c;
            next.tile += count - 1;
            K::advance(a, units, end, next);
            if (inside(next)) K::fetch_q(a, next, nsub, q_buf + (~segment & 1) * K::kQBytes);
        }
        for (int i = 0; i < count; ++i) {
            cp_async_wait<K::kStages - 2>();
            __syncwarp();
            const uint32_t mask = sh.mask[warp][stage_out];
            feed();
            // keys beyond the request (the tail of its last tile) count for nothing
            if (mask) K::tile(a, st, ring + stage_out * 2 * K::kTileBytes, ln, mask, lane);
            stage_out = stage_out + 1 == K::kStages ? 0 : stage_out + 1;
            K::advance(a, units, end, c);
        }
        const int last_stage = stage_out == 0 ? K::kStages - 1 : stage_out - 1;
        const bool whole = seg.tile == 0 && count == seg.tiles;
        // slot of CTA k's part: its first unit, or its last
        auto part_of = [&](int k, bool first) { return a.parts + (size_t)(2 * k + (first ? 0 : 1)) * K::kPartFloats; };
        char* lay = smem + last_stage * 2 * K::kTileBytes;
        constexpr int kStride = K::kStages * 2 * K::kTileBytes;
        K::merge(a, seg, nsub, st, lay, kStride, sh, whole ? nullptr : part_of(blockIdx.x, segment == 0));
        if (!whole) {
            const int c_first = share.cta_of(seg.base + kUnitCost);
            const int c_last = share.cta_of(seg.base + kUnitCost + (long long)kTileCost * (seg.tiles - 1));
            // the unit is the first one of CTA c_first unless that also has the last tile before it
            const bool head = seg.base == 0 || share.start(c_first) > seg.base - kTileCost;
            const int n = c_last - c_first + 1;
            auto part_at = [&](int i) { return part_of(c_first + i, i > 0 || head); };
            uint32_t* done = a.done + (long long)seg.b * units + seg.unit;
            if (n <= kJoinMost) {
                if (K::arrive_last(done, n, sh)) K::join(a, seg, nsub, n, part_at, sh, nullptr);
            } else {
                const int me = (int)blockIdx.x - c_first, g0 = me / kJoinGroup * kJoinGroup, gn = min(kJoinGroup, n - g0);
                if (K::arrive_last(a.group_done + 2 * (c_first + g0) + (g0 > 0 || head ? 0 : 1), gn, sh)) {
                    K::join(a, seg, nsub, gn, [&](int i) { return part_at(g0 + i); }, sh, part_at(g0));
                    const int groups = (n + kJoinGroup - 1) / kJoinGroup;
                    if (K::arrive_last(done, groups, sh))
                        K::join(a, seg, nsub, groups, [&](int i) { return part_at(i * kJoinGroup); }, sh, nullptr);
                }
            }
        }
        ++segment;
    }
    cp_async_wait<0>();
}

int dp_of(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
// Query heads of a unit: 16 where the heads of a key-value head need them and the
// registers hold 16 rows of o and q.
int rows_of(int group, int dp, bool exact) { return group > 8 && dp <= 128 && !exact ? 16 : 8; }

template <int DP, bool F8, int ROWS, bool EX>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    using K = Attn<DP, F8, ROWS, EX>;
    auto kern = attn_kernel<DP, F8, ROWS, EX>;
    static std::atomic<uint64_t> done;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), (int)K::kSmem, done);
    if (e != cudaSuccess) return e;
    static_assert(K::kCtasPerSm * (K::kSmem + sizeof(typename K::Shared) + 1024) <= 228 * 1024, "CTAs that run at once");
    const int grid = std::min(K::kCtasPerSm * device_sm_count(), kAttnMaxCtas);
    return launch_pdl(kern, dim3((unsigned)grid), dim3(kAttnThreads), K::kSmem, s, a);
}

template <int DP, bool F8>
cudaError_t launch_dp(const AttnArgs& a, cudaStream_t s) {
    const bool exact = a.q_dt == MOE_DTYPE_F32 || a.o_dt == MOE_DTYPE_F32 || a.softcap > kFastCap;
    if (exact) return launch<DP, F8, 8, true>(a, s);
    if constexpr (DP <= 128) {
        if (rows_of(a.group, DP, false) == 16) return launch<DP, F8, 16, false>(a, s);
    }
    return launch<DP, F8, 8, false>(a, s);
}

}  // namespace

size_t attn_workspace_bytes(int B, int q_heads, int heads, int head_dim, size_t* done_off, size_t* group_off, size_t* parts_off) {
    // the group counters and the parts come first: their place does not depend on B, so that the
    // counters after them stay zero whatever the calls' batch sizes are
    const int group = q_heads / heads, dp = dp_of(head_dim);
    const size_t floats = (size_t)rows_of(group, dp, false) * (dp + 2);
    *group_off = 512;
    *parts_off = 512 + 2 * kAttnMaxCtas * sizeof(uint32_t);
    *done_off = *parts_off + 2 * kAttnMaxCtas * floats * sizeof(float);
    const size_t total = *done_off + (size_t)B * heads * ((group + 7) / 8) * sizeof(uint32_t);
    return (total + 255) / 256 * 256;   // moe_workspace_init clears whole 16-byte words
}

cudaError_t launch_attn_decode(const AttnArgs& args, cudaStream_t s) {
    AttnArgs a = args;
    const bool f8 = a.c.dtype == MOE_DTYPE_FP8_E4M3;
    a.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (a.c.page_size == 1 << i) a.page_shift = i;
    // bytes up to the last row of either tensor
    auto reach = [&](int64_t page, int64_t slot, int64_t head) {
        return (__int128)page * (a.c.num_pages - 1) + (__int128)slot * (a.c.page_size - 1) + (__int128)head * (a.c.heads - 1);
    };
    const __int128 most = std::max(reach(a.c.k_page_stride, a.c.k_slot_stride, a.c.k_head_stride),
                                   reach(a.c.v_page_stride, a.c.v_slot_stride, a.c.v_head_stride));
    a.far = most * (f8 ? 1 : 2) / 16 > 0xffffffffll;
    switch (dp_of(a.c.head_dim)) {
        case 64: return f8 ? launch_dp<64, true>(a, s) : launch_dp<64, false>(a, s);
        case 128: return f8 ? launch_dp<128, true>(a, s) : launch_dp<128, false>(a, s);
        default: return f8 ? launch_dp<256, true>(a, s) : launch_dp<256, false>(a, s);
    }
}

}  // namespace moe
