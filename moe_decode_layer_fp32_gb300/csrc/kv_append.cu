// Rotary position encoding of q and k, and the new tokens' k, v rows into the
// paged cache.  Element i < rot / 2 of a head turns with element i + rot / 2:
//   a' = a cos - b sin,  b' = b cos + a sin.
//
// HBM bounds many tokens, latency a few.  An item of a head is two vectors of 8 elements, a
// rotated pair or two of the others; a thread has the same item of several heads, so that
// each element is read once and cos, sin once for all heads.  What a token costs is a chain of
// loads (position, then page and cos, sin; rows), so each block has the next token's under
// way while it works on the current one, and looks at nothing in the turn that loads it.
//
// moe_qk_norm_append takes the same way and norms each head of q and k first: u = x / sqrt(mean x^2 + eps) w.
// The threads of a head's items are then a power of two, so that its sum of squares is a few shuffles;
// the weights wait in shared memory.  With positions of several axes each element of cos, sin comes from
// the row of its pair's axis: single words copied into one row, which is read like any other.
//
// Measured, 12345 tokens of 56 + 8 + 8 heads of 128, bf16 into E4M3, half of each head rotated
// (431 MB): 66 us, 6.5 TB/s; a block per token without the copies ahead 86 us.  A page looked at where
// it is loaded 73 us, the units' divisions in the loop 71 us, tokens in two slices 93 us; at 56
// registers instead of 72 (9 blocks per SM instead of 7) 69 us.
#include <algorithm>
#include <climits>
#include <type_traits>

#include <math_constants.h>

#include "block.h"

namespace moe {

namespace {

constexpr int kAppendThreads = 128;
constexpr int kVec = 8;                     // elements of a vector
constexpr int kAppendSmem = 112 * 1024;     // two blocks per SM

// inv: 1 / scale of E4M3 rows (a code is the value times it, within 1 ulp of value / scale).
template <int VEC>
__device__ __forceinline__ void store_vec(void* p, int dt, long long i, const float (&f)[VEC], float inv) {
    if (dt == MOE_DTYPE_FP8_E4M3) {
        uint8_t* b = static_cast<uint8_t*>(p) + i;
        if constexpr (VEC == 8) {
            *reinterpret_cast<uint2*>(b) = make_uint2(pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                                                      pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
        } else {
            b[0] = (uint8_t)__nv_cvt_float_to_fp8(f[0] * inv, __NV_SATFINITE, __NV_E4M3);
        }
    } else if constexpr (VEC == 8) {
        store8(p, dt, i, f);
    } else {
        if (dt == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f[0]);
        else static_cast<float*>(p)[i] = f[0];
    }
}

// What a thread has of every head it takes: elements [i0, + VEC) and (two) [i1, + VEC), turned
// into one another (turn) or left alone.
template <int VEC>
struct Item {
    int i0, i1;
    bool two, turn;
    alignas(16) float cs[VEC], sn[VEC];
    // item i of a head of D elements, whose first 2 half turn
    __device__ __forceinline__ void place(int i, int D, int half) {
        const int pairs = half / VEC, plain = (D - 2 * half) / VEC;
        turn = i < pairs;
        if (turn) {
            i0 = i * VEC;
            i1 = i0 + half;
            two = true;
        } else {
            const int k = i - pairs, k1 = k + (plain + 1) / 2;
            i0 = 2 * half + k * VEC;
            i1 = 2 * half + k1 * VEC;
            two = k1 < plain;
        }
    }
    __device__ __forceinline__ void rotate(float (&x)[VEC], float (&y)[VEC]) const {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float f = x[e], g = y[e];
            x[e] = f * cs[e] - g * sn[e];
            y[e] = g * cs[e] + f * sn[e];
        }
    }
};

// The request's page of a position as the table has it, which may not be one of the pool; -1: none.
// last: the last position that has one (of the rows of cos_sin).
__device__ __forceinline__ int page_of(const AppendArgs& a, int req, int pos, int last) {
    const int col = pos / a.c.page_size;
    return pos < 0 || req < 0 || req >= a.R || col >= a.max_pages || pos > last ? -1 : a.table[req * a.table_ld + col];
}
__device__ __forceinline__ int last_of(const AppendArgs& a) { return a.rot ? a.max_pos - 1 : INT_MAX; }
// With axes the rows of cos_sin are those of the axes' positions, and not looked up by `positions`.
__device__ __forceinline__ int last_of(const QkAppendArgs& a) { return a.rot && !a.axes ? a.max_pos - 1 : INT_MAX; }
__device__ __forceinline__ float weight_at(const void* w, int dt, int i) {
    return !w ? 1.0f : dt == MOE_DTYPE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
}
// 1 / sqrt(v): the fast one and a Newton step (v = 0 and infinity as they are).
__device__ __forceinline__ float inv_sqrt(float v) {
    const float r = rsqrtf(v);
    return v > 0.0f && v < CUDART_INF_F ? r * fmaf(-0.5f * v * r, r, 1.5f) : r;
}
// Items of a head of 16-byte vectors: the pairs that turn, and the others two by two.
__host__ __device__ inline int items_of(int D, int rot) { return rot / 2 / kVec + ((D - rot) / kVec + 1) / 2; }
// Threads of a head.  16 items at most: a head never leaves its warp.
template <bool NORM>
__host__ __device__ inline int span_of(int items) {
    return !NORM ? items : items <= 1 ? 1 : items <= 2 ? 2 : items <= 4 ? 4 : items <= 8 ? 8 : 16;
}

// Any strides, alignment and rotary width: an element at a time (12000 tokens of 32 + 8 + 8 heads, bf16: of 80
// with 40 rotated 102 us, of 96 with 24 rotated 120 us; the vectors below, all rotated, 37 and 38 us).
// Grid: x = token, y = slice of the heads.
template <bool BF>
__global__ void __launch_bounds__(kAppendThreads) kv_append_any_kernel(const __grid_constant__ AppendArgs a) {
    pdl_allow_dependents();
    pdl_wait_primary();
    const int t = blockIdx.x, D = a.c.head_dim, kvh = a.c.heads, heads = a.q_heads + 2 * kvh, pos = a.positions[t];
    const int half = a.rot && pos >= 0 && pos < a.max_pos ? a.rot / 2 : 0;
    const int entry = page_of(a, a.req ? a.req[t] : t, pos, last_of(a)), page = entry < a.c.num_pages ? entry : -1;
    if (pos >= 0 && page < 0 && threadIdx.x == 0 && a.status) set_status(a.status, MOE_ERR_DEVICE);
    const int items = half + (D - 2 * half + 1) / 2, slot = pos - pos / a.c.page_size * a.c.page_size;
    const float* row = a.cos_sin + (long long)pos * a.rot;
    auto load = [&](const void* p, long long i) {
        return BF ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
    };
    for (int i = blockIdx.y * kAppendThreads + threadIdx.x; i < heads * items; i += gridDim.y * kAppendThreads) {
        const int h = i / items, g = h - a.q_heads;
        if (g >= 0 && page < 0) break;
        Item<1> it;
        it.place(i - h * items, D, half);
        const void* src = g < 0 ? a.q : g < kvh ? a.k : a.v;
        const long long o = g < 0 ? t * a.q_ts + h * a.q_hs : g < kvh ? t * a.k_ts + g * a.k_hs : t * a.v_ts + (g - kvh) * a.v_hs;
        float x[1] = {load(src, o + it.i0)}, y[1] = {it.two ? load(src, o + it.i1) : 0.0f};
        if (it.turn && g < kvh) {
            it.cs[0] = row[it.i0];
            it.sn[0] = row[half + it.i0];
            it.rotate(x, y);
        }
        void* dst = g < 0 ? a.q_out : g < kvh ? a.c.k : a.c.v;
        const long long d =
            g < 0 ? t * a.o_ts + h * a.o_hs
            : g < kvh ? page * a.c.k_page_stride + slot * a.c.k_slot_stride + g * a.c.k_head_stride
                      : page * a.c.v_page_stride + slot * a.c.v_slot_stride + (g - kvh) * a.c.v_head_stride;
        const float* scale = g < 0 ? nullptr : g < kvh ? a.c.k_scale : a.c.v_scale;
        const float inv = scale ? 1.0f / scale[g < kvh ? g : g - kvh] : 1.0f;
        const int dt = g < 0 ? a.in_dt : a.c.dtype;
        store_vec<1>(dst, dt, d + it.i0, x, inv);
        if (it.two) store_vec<1>(dst, dt, d + it.i1, y, inv);
    }
}

// The same with norms: a warp to a head, its lanes' items 32 apart.
template <bool BF>
__global__ void __launch_bounds__(kAppendThreads) qk_append_any_kernel(const __grid_constant__ QkAppendArgs a) {
    pdl_allow_dependents();
    pdl_wait_primary();
    constexpr int kMost = 4, kWarps = kAppendThreads / 32;      // items of a lane: 128 pairs of a head at most
    const int t = blockIdx.x, D = a.c.head_dim, kvh = a.c.heads, heads = a.q_heads + 2 * kvh, pos = a.positions[t];
    const int lane = threadIdx.x & 31, half = a.rot / 2, items = half + (D - 2 * half + 1) / 2;
    bool bad = a.rot && !a.axes && pos >= a.max_pos;
    Item<1> it[kMost];
#pragma unroll
    for (int n = 0; n < kMost; ++n) {
        const int i = lane + 32 * n;
        it[n].turn = false;
        if (i < items) it[n].place(i, D, half);
        if (!it[n].turn || pos < 0) continue;
        const int at = a.axes ? a.axis_positions[(long long)a.axis[i] * a.T + t] : pos;
        if (at < 0 || at >= a.max_pos) {
            bad = true;
        } else {
            it[n].cs[0] = a.cos_sin[(long long)at * a.rot + i];
            it[n].sn[0] = a.cos_sin[(long long)at * a.rot + half + i];
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    const bool turn = pos >= 0 && !bad;
    const int entry = bad ? -1 : page_of(a, a.req ? a.req[t] : t, pos, INT_MAX), page = entry < a.c.num_pages ? entry : -1;
    if (pos >= 0 && page < 0 && threadIdx.x == 0 && a.status) set_status(a.status, MOE_ERR_DEVICE);
    const int slot = pos - pos / a.c.page_size * a.c.page_size;
    auto load = [&](const void* p, long long i) {
        return BF ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
    };
    for (int h = blockIdx.y * kWarps + threadIdx.x / 32; h < heads; h += gridDim.y * kWarps) {
        const int g = h - a.q_heads;
        if (g >= 0 && page < 0) break;
        const bool normed = g < kvh;
        const void* src = g < 0 ? a.q : normed ? a.k : a.v;
        const long long o = g < 0 ? t * a.q_ts + h * a.q_hs : normed ? t * a.k_ts + g * a.k_hs : t * a.v_ts + (g - kvh) * a.v_hs;
        float x[kMost][1], y[kMost][1], sum = 0.0f;
#pragma unroll
        for (int n = 0; n < kMost; ++n) {
            const bool on = lane + 32 * n < items;
            x[n][0] = on ? load(src, o + it[n].i0) : 0.0f;
            y[n][0] = on && it[n].two ? load(src, o + it[n].i1) : 0.0f;
            sum += x[n][0] * x[n][0] + y[n][0] * y[n][0];
        }
        const float r = inv_sqrt(warp_sum(sum) / D + a.eps);
        void* dst = g < 0 ? a.q_out : normed ? a.c.k : a.c.v;
        const long long d =
            g < 0 ? t * a.o_ts + h * a.o_hs
            : normed ? page * a.c.k_page_stride + slot * a.c.k_slot_stride + g * a.c.k_head_stride
                     : page * a.c.v_page_stride + slot * a.c.v_slot_stride + (g - kvh) * a.c.v_head_stride;
        const void* w = g < 0 ? a.q_weight : a.k_weight;
        const float* scale = g < 0 ? nullptr : normed ? a.c.k_scale : a.c.v_scale;
        const float inv = scale ? 1.0f / scale[normed ? g : g - kvh] : 1.0f;
        const int dt = g < 0 ? a.in_dt : a.c.dtype;
#pragma unroll
        for (int n = 0; n < kMost; ++n) {
            if (lane + 32 * n >= items) break;
            if (normed) {
                x[n][0] *= r * weight_at(w, a.w_dt, it[n].i0);
                if (it[n].two) y[n][0] *= r * weight_at(w, a.w_dt, it[n].i1);
                if (turn && it[n].turn) it[n].rotate(x[n], y[n]);
            }
            store_vec<1>(dst, dt, d + it[n].i0, x[n], inv);
            if (it[n].two) store_vec<1>(dst, dt, d + it[n].i1, y[n], inv);
        }
    }
}

// 16-byte vectors.  A unit is a token and a slice of its heads, nq of q's and nkv of k's and v's to a
// thread at most; a block takes units blockIdx.x, + gridDim.x, ..., with the next one's rows on
// their way into shared memory (every thread's own vectors into places of its own) while it
// turns and stores the current one's.
// Norms (QkAppendArgs): a head's threads are a power of two (span), the last ones of them without an item.
template <bool BF, class Args>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ Args a, int slices, int nq, int nkv) {
    constexpr bool NORM = std::is_same_v<Args, QkAppendArgs>;
    constexpr int WB = BF ? 16 : 32;                          // bytes of a vector
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, D = a.c.head_dim, kvh = a.c.heads, P = a.c.page_size, n = nq + nkv;
    const int items = items_of(D, a.rot), span = span_of<NORM>(items), lanes = kAppendThreads / span, hl = tid / span;
    const bool on = !NORM || tid - hl * span < items;
    float* turns = reinterpret_cast<float*>(smem + 4 * n * kAppendThreads * WB);   // [2][rot], behind the rows
    float* inv = turns + 2 * a.rot;                           // [2 kvh] 1 / scale of E4M3 rows
    float* weights = inv + (2 * kvh + 3) / 4 * 4;             // [2][D] of q and k
    Item<kVec> it;
    it.place(on ? tid - hl * span : 0, D, a.rot / 2);
    pdl_allow_dependents();
    pdl_wait_primary();
    for (int i = tid; i < 2 * kvh; i += kAppendThreads) {
        const float* scale = i < kvh ? a.c.k_scale : a.c.v_scale;
        inv[i] = scale ? 1.0f / scale[i < kvh ? i : i - kvh] : 1.0f;
    }
    bool with_axes = false;
    int axis[2] = {0, 0};      // of the words tid, + 128 of a row of cos, sin
    if constexpr (NORM) {
        for (int i = tid; i < 2 * D; i += kAppendThreads) weights[i] = weight_at(i < D ? a.q_weight : a.k_weight, a.w_dt, i < D ? i : i - D);
        with_axes = a.axes > 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int w = tid + j * kAppendThreads, half = a.rot / 2;
            if (w < a.rot) axis[j] = a.axis[w < half ? w : w - half];
        }
    }
    const int last = last_of(a);
    // the thread's heads of a slice: from here on, lanes apart
    auto first_q = [&](int slice) { return hl < lanes ? slice * nq * lanes + hl : a.q_heads; };
    auto first_kv = [&](int slice) { return hl < lanes ? slice * nkv * lanes + hl : 2 * kvh; };
    auto place = [&](int buf, int s, int k) { return smem + (((buf * n + s) * 2 + k) * kAppendThreads + tid) * WB; };
    auto copy = [&](char* dst, const void* p, long long i) {
        const char* src = static_cast<const char*>(p) + i * (BF ? 2 : 4);
        cp_async16(dst, src);
        if constexpr (!BF) cp_async16(dst + 16, src + 16);
    };
    // whether a row of cos, sin that the token needs is not there (with axes, seen by some of the threads)
    auto fetch = [&](int buf, int t, int slice, int pos, const int (&at)[2]) {
        bool bad = false;
        for (int s = 0, h = first_q(slice); on && s < nq && h < a.q_heads; ++s, h += lanes) {
            const long long o = t * a.q_ts + h * a.q_hs;
            copy(place(buf, s, 0), a.q, o + it.i0);
            if (it.two) copy(place(buf, s, 1), a.q, o + it.i1);
        }
        for (int s = nq, h = first_kv(slice); on && pos >= 0 && s < n && h < 2 * kvh; ++s, h += lanes) {
            const bool k = h < kvh;
            const void* p = k ? a.k : a.v;
            const long long o = k ? t * a.k_ts + h * a.k_hs : t * a.v_ts + (h - kvh) * a.v_hs;
            copy(place(buf, s, 0), p, o + it.i0);
            if (it.two) copy(place(buf, s, 1), p, o + it.i1);
        }
        if (with_axes) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int w = tid + j * kAppendThreads;
                if (w >= a.rot || pos < 0) continue;
                if (at[j] < 0 || at[j] >= a.max_pos) bad = true;
                else cp_async4(turns + buf * a.rot + w, a.cos_sin + (long long)at[j] * a.rot + w);
            }
        } else if (pos >= 0 && pos < a.max_pos) {
            for (int w = tid * 4; w < a.rot; w += kAppendThreads * 4)
                cp_async16(turns + buf * a.rot + w, a.cos_sin + (long long)pos * a.rot + w);
        }
        cp_async_commit();
        return bad;
    };
    // the axes' positions of the thread's words
    auto places = [&](int t, int (&at)[2]) {
        if constexpr (NORM) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (with_axes && t < a.T && tid + j * kAppendThreads < a.rot) at[j] = a.axis_positions[(long long)axis[j] * a.T + t];
        }
    };
    // this unit, the next and the one after it
    const int dt = gridDim.x / slices, ds = gridDim.x % slices;
    auto advance = [&](int& t, int& slice) {
        t += dt;
        slice += ds;
        if (slice >= slices) {
            slice -= slices;
            ++t;
        }
    };
    auto position = [&](int t) { return t < a.T ? a.positions[t] : -1; };
    auto request = [&](int t) { return a.req && t < a.T ? a.req[t] : t; };
    int t = blockIdx.x / slices, slice = blockIdx.x % slices, t1 = t, slice1 = slice;
    advance(t1, slice1);
    int t2 = t1, slice2 = slice1;
    // what is loaded in one turn of the loop is looked at in the next
    int pos = position(t), pos1 = position(t1), req1 = request(t1), entry = page_of(a, request(t), pos, last), at[2], at1[2];
    places(t, at);
    places(t1, at1);
    bool bad = fetch(0, t, slice, pos, at);
    for (int buf = 0; t < a.T; buf ^= 1) {
        cp_async_wait<0>();
        // the turns are there, and nobody reads the other half's any more
        bool lost = false;
        if (with_axes) lost = __syncthreads_or(bad);
        else __syncthreads();
        if (t1 < a.T) bad = fetch(buf ^ 1, t1, slice1, pos1, at1);
        advance(t2, slice2);
        places(t2, at1);
        const int entry1 = page_of(a, req1, pos1, last), pos2 = position(t2), req2 = request(t2);
        const int page = entry < a.c.num_pages && !lost ? entry : -1;
        // padding and tokens without a row in cos_sin: q is not turned
        const bool turn = it.turn && pos >= 0 && (with_axes ? !lost : pos < a.max_pos);
        if (turn) {
            const float* row = turns + buf * a.rot + it.i0;
#pragma unroll
            for (int e = 0; e < kVec; e += 4) {
                *reinterpret_cast<float4*>(it.cs + e) = *reinterpret_cast<const float4*>(row + e);
                *reinterpret_cast<float4*>(it.sn + e) = *reinterpret_cast<const float4*>(row + a.rot / 2 + e);
            }
        }
        if (pos >= 0 && page < 0 && tid == 0 && a.status) set_status(a.status, MOE_ERR_DEVICE);
        const int slot = pos - pos / P * P;
        const long long krow = (long long)page * a.c.k_page_stride + slot * a.c.k_slot_stride, vrow = page * a.c.v_page_stride + slot * a.c.v_slot_stride;
        float x[kVec], y[kVec];
        auto get = [&](int s) {
            load8_f32(place(buf, s, 0), BF ? MOE_DTYPE_BF16 : MOE_DTYPE_F32, 0, x);
            load8_f32(place(buf, s, 1), BF ? MOE_DTYPE_BF16 : MOE_DTYPE_F32, 0, y);
        };
        auto norm = [&](const float* w) {
            if constexpr (NORM) {
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    x[e] = on ? x[e] : 0.0f;
                    y[e] = on && it.two ? y[e] : 0.0f;
                    sum += x[e] * x[e] + y[e] * y[e];
                }
                // the threads of a head are neighbours in a warp
                const uint32_t group = ((1u << span) - 1u) << (tid % 32 / span * span);
                for (int o = span / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(group, sum, o);
                const float r = inv_sqrt(sum / D + a.eps);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    x[e] *= r * w[it.i0 + e];
                    if (it.two) y[e] *= r * w[it.i1 + e];
                }
            }
        };
        for (int s = 0, h = first_q(slice); s < nq && h < a.q_heads; ++s, h += lanes) {
            get(s);
            norm(weights);
            if (!on) continue;
            if (turn) it.rotate(x, y);
            const long long d = t * a.o_ts + h * a.o_hs;
            store8(a.q_out, a.in_dt, d + it.i0, x);
            if (it.two) store8(a.q_out, a.in_dt, d + it.i1, y);
        }
        for (int s = nq, h = first_kv(slice); page >= 0 && s < n && h < 2 * kvh; ++s, h += lanes) {
            get(s);
            const bool k = h < kvh;
            if (k) norm(weights + D);
            if (!on) continue;
            if (turn && k) it.rotate(x, y);
            void* p = k ? a.c.k : a.c.v;
            const long long d = k ? krow + h * a.c.k_head_stride : vrow + (h - kvh) * a.c.v_head_stride;
            store_vec<kVec>(p, a.c.dtype, d + it.i0, x, inv[h]);
            if (it.two) store_vec<kVec>(p, a.c.dtype, d + it.i1, y, inv[h]);
        }
        t = t1;
        slice = slice1;
        t1 = t2;
        slice1 = slice2;
        pos = pos1;
        entry = entry1;
        pos1 = pos2;
        req1 = req2;
    }
}

template <class Args>
cudaError_t launch(const Args& a, cudaStream_t s) {
    constexpr bool NORM = std::is_same_v<Args, QkAppendArgs>;
    const bool bf = a.in_dt == MOE_DTYPE_BF16;
    const int sms = device_sm_count(), heads = a.q_heads + 2 * a.c.heads;
    // 16-byte vectors where every offset is a multiple of 8 elements (and units and scales are
    // no more than the kernel's integers and shared memory take)
    auto m8 = [](long long v) { return v % 8 == 0; };
    const bool vec8 = a.rot % 16 == 0 && m8(a.k_ts) && m8(a.k_hs) && m8(a.v_ts) && m8(a.v_hs) && m8(a.q_ts) &&
                      m8(a.q_hs) && m8(a.o_ts) && m8(a.o_hs) &&
                      (((uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.q | (uintptr_t)a.q_out | (uintptr_t)a.cos_sin) & 15) == 0 &&
                      a.c.heads <= 8192 && (long long)a.T * heads <= 1 << 30;
    // Few tokens: slices of the heads, until the blocks fill the GPU or a thread has one head.
    if (!vec8) {
        const int most = NORM ? (heads + 3) / 4 : (heads * ((a.c.head_dim + 1) / 2) + kAppendThreads - 1) / kAppendThreads;
        const int slices = std::max(1, std::min({most, 8 * sms / a.T, 65535}));
        const dim3 grid((unsigned)a.T, (unsigned)slices);
        if constexpr (NORM) return launch_pdl(bf ? qk_append_any_kernel<true> : qk_append_any_kernel<false>, grid, dim3(kAppendThreads), 0, s, a);
        else return launch_pdl(bf ? kv_append_any_kernel<true> : kv_append_any_kernel<false>, grid, dim3(kAppendThreads), 0, s, a);
    }
    const int lanes = kAppendThreads / span_of<NORM>(items_of(a.c.head_dim, a.rot));
    const int most_q = (a.q_heads + lanes - 1) / lanes, most_kv = (2 * a.c.heads + lanes - 1) / lanes;
    int slices = std::max(1, std::min(std::max(most_q, most_kv), 8 * sms / a.T)), nq, nkv;
    size_t smem;
    for (;; ++slices) {      // whole tokens where two units of them fit in shared memory
        nq = (most_q + slices - 1) / slices;
        nkv = (most_kv + slices - 1) / slices;
        smem = (size_t)4 * (nq + nkv) * kAppendThreads * (bf ? 16 : 32) + (2 * a.rot + 2 * a.c.heads) * 4;
        if (NORM) smem += (2 * a.c.head_dim + 3) * 4;
        if (smem <= (size_t)kAppendSmem || nq + nkv <= 2) break;
    }
    auto kern = bf ? kv_append_kernel<true, Args> : kv_append_kernel<false, Args>;
    static std::atomic<uint64_t> done[2], blocks[2];
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kAppendSmem, done[bf]);
    int per_sm = 0;
    if (e == cudaSuccess) e = blocks_per_sm(reinterpret_cast<const void*>(kern), kAppendThreads, smem, blocks[bf], &per_sm);
    if (e != cudaSuccess) return e;
    const int grid = std::min(a.T * slices, per_sm * sms);
    return launch_pdl(kern, dim3((unsigned)grid), dim3(kAppendThreads), smem, s, a, slices, nq, nkv);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s) { return launch(a, s); }
cudaError_t launch_qk_norm_append(const QkAppendArgs& a, cudaStream_t s) { return launch(a, s); }

}  // namespace moe
