// Root-mean-square norm of every head of q and k, rotary position encoding by positions of one or
// several axes, and the new tokens' k, v rows into the paged cache:
//   u = x / sqrt(mean x^2 + eps) w,  u_i' = u_i cos - u_j sin,  u_j' = u_j cos + u_i sin,  j = i + rot / 2.
//
// HBM bounds many tokens if the instructions per value are few, latency a few tokens.  The way through memory
// is the append's without norms: a thread has the same two vectors of several heads, blocks walk over
// the tokens with the next one's rows on their way into shared memory.  The threads of a head are a power
// of two, so that its sum of squares is a few shuffles.  The weights and cos, sin become one set of factors per
// token and thread, so that a pair costs two multiplications and two multiply-adds, and one more of each
// of its values with 1 / sqrt; two heads at a time hide one another's shuffles.  With several axes every element
// of cos, sin comes from the row of its pair's axis: single words copied into one row, which is read like any other.
//
// Measured, 12345 tokens of 56 + 8 + 8 heads of 128, bf16 into E4M3, half of each head rotated by three axes (430 MB):
// 77 us, 5.6 TB/s (with one axis 76; the append without norms 67). Latency bounds it: at 16 warps per SM the schedulers issue
// at 57 % of the clocks and wait for instructions with a fixed latency and for shuffles and shared memory otherwise. One head at a time 86 us, the append's kernel with plain multiplications 104; at 102 registers
// instead of 117 (5 blocks per SM instead of 4) 89. 12345 tokens of 32 + 8 + 8 heads: of 64 34 us (blocks of 128 threads
// 46 before, and 43 of 64), of 80 62 (5 of 8 threads have an item; 6 heads of 5 threads to a warp, with sums one
// thread after another, 64), of 80 with 40 rotated, in vectors of 4, 67 (an element at a time 240).
#include <algorithm>

#include <math_constants.h>

#include "append.cuh"

namespace moe {

namespace {

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

// Any strides, alignment and rotary width: an element at a time, a warp to a head, its lanes' items 32 apart.
// Grid: x = token, y = slice of the heads.
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
        const float r = inv_sqrt(fmaf(warp_sum(sum), 1.0f / D, a.eps));
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

// Items of a head of vectors of `vec` elements: the pairs that turn, and the others two by two; and its threads.
__host__ __device__ inline int items_of(int D, int rot, int vec) { return rot / 2 / vec + ((D - rot) / vec + 1) / 2; }
__host__ __device__ inline int span_of(int items) {
    int span = 1;
    while (span < items) span *= 2;
    return span;       // 32 at most: a head never leaves its warp
}

__device__ __forceinline__ void cp_async8(void* dst_smem, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst_smem)), "l"(src) : "memory");
}

// Vectors of VEC elements.  A unit is a token and a slice of its heads, nq of q's and nkv of k's and v's to a
// thread at most; a block takes units blockIdx.x, + gridDim.x, ..., with the next one's rows on their way into
// shared memory (every thread's own vectors into places of its own) while it works on the current one's.
template <bool BF, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS) qk_append_kernel(const __grid_constant__ QkAppendArgs a, int slices, int nq, int nkv) {
    constexpr int WB = VEC * (BF ? 2 : 4), N = VEC / 2;       // bytes of a vector, its pairs of neighbours
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, D = a.c.head_dim, kvh = a.c.heads, P = a.c.page_size, n = nq + nkv, half = a.rot / 2;
    const int items = items_of(D, a.rot, VEC), span = span_of(items), lanes = THREADS / span, hl = tid / span;
    const bool on = tid - hl * span < items;                  // has an item
    float* turns = reinterpret_cast<float*>(smem + 4 * n * THREADS * WB);   // [2][rot], behind the rows
    float* weights = turns + 2 * a.rot;                       // [2][D] of q and k
    float* inv = weights + 2 * D;                             // [2 kvh] 1 / scale of E4M3 rows
    Item<VEC> it;
    it.place(on ? tid - hl * span : 0, D, half);
    auto place = [&](int buf, int s, int k) { return smem + (((buf * n + s) * 2 + k) * THREADS + tid) * WB; };
    // vectors that the thread does not have are zeros: they add nothing to a sum
    for (int i = 0; i < 2 * n; ++i)
        for (int k = 0; k < 2; ++k)
            if (!on || (k && !it.two))
                for (int w = 0; w < WB; w += 8) *reinterpret_cast<uint2*>(place(0, i, k) + w) = make_uint2(0, 0);
    pdl_allow_dependents();
    pdl_wait_primary();
    for (int i = tid; i < 2 * D; i += THREADS) weights[i] = weight_at(i < D ? a.q_weight : a.k_weight, a.w_dt, i < D ? i : i - D);
    for (int i = tid; i < 2 * kvh; i += THREADS) {
        const float* scale = i < kvh ? a.c.k_scale : a.c.v_scale;
        inv[i] = scale ? 1.0f / scale[i < kvh ? i : i - kvh] : 1.0f;
    }
    const bool with_axes = a.axes > 0;
    constexpr int W = 256 / THREADS;
    int axis[W] = {};          // of the words tid, + THREADS, ... of a row of cos, sin
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const int w = tid + j * THREADS;
        if (w < a.rot) axis[j] = a.axis[w < half ? w : w - half];
    }
    const int last = last_of(a);
    const uint32_t group = (span == 32 ? 0xffffffffu : (1u << span) - 1u) << (tid % 32 / span * span);
    const float inv_d = 1.0f / D;
    // the thread's heads of a slice: from here on, lanes apart
    auto first_q = [&](int slice) { return slice * nq * lanes + hl; };
    auto first_kv = [&](int slice) { return slice * nkv * lanes + hl; };
    constexpr int kSize = BF ? 2 : 4;
    const long long q_step = lanes * a.q_hs * kSize, o_step = lanes * a.o_hs * kSize;     // bytes from a head of the thread to the next
    const int apart = (it.i1 - it.i0) * kSize;
    auto copy = [&](char* dst, const char* src) {
        if constexpr (WB == 8) cp_async8(dst, src);
        else cp_async16(dst, src);
        if constexpr (WB == 32) cp_async16(dst + 16, src + 16);
    };
    // whether a row of cos, sin that the token needs is not there (with axes, seen by some of the threads)
    auto fetch = [&](int buf, int t, int slice, int pos, const int (&at)[W]) {
        bool bad = false;
        const int q1 = on ? min(a.q_heads, first_q(slice) + nq * lanes) : 0, kv1 = on && pos >= 0 ? min(2 * kvh, first_kv(slice) + nkv * lanes) : 0;
        char* to = place(buf, 0, 0);
        const char* src = static_cast<const char*>(a.q) + (t * a.q_ts + first_q(slice) * a.q_hs + it.i0) * kSize;
        for (int h = first_q(slice); h < q1; h += lanes, to += 2 * THREADS * WB, src += q_step) {
            copy(to, src);
            if (it.two) copy(to + THREADS * WB, src + apart);
        }
        to = place(buf, nq, 0);
        for (int h = first_kv(slice); h < kv1; h += lanes, to += 2 * THREADS * WB) {
            const bool k = h < kvh;
            src = static_cast<const char*>(k ? a.k : a.v) + ((k ? t * a.k_ts + h * a.k_hs : t * a.v_ts + (h - kvh) * a.v_hs) + it.i0) * kSize;
            copy(to, src);
            if (it.two) copy(to + THREADS * WB, src + apart);
        }
        if (with_axes) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int w = tid + j * THREADS;
                if (w >= a.rot || pos < 0) continue;
                if (at[j] < 0 || at[j] >= a.max_pos) bad = true;
                else cp_async4(turns + buf * a.rot + w, a.cos_sin + (long long)at[j] * a.rot + w);
            }
        } else if (pos >= 0 && pos < a.max_pos) {
            for (int w = tid * 4; w < a.rot; w += THREADS * 4)
                cp_async16(turns + buf * a.rot + w, a.cos_sin + (long long)pos * a.rot + w);
        }
        cp_async_commit();
        return bad;
    };
    // the axes' positions of the thread's words
    auto places = [&](int t, int (&at)[W]) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (with_axes && t < a.T && tid + j * THREADS < a.rot) at[j] = a.axis_positions[(long long)axis[j] * a.T + t];
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
    int pos = position(t), pos1 = position(t1), req1 = request(t1), entry = page_of(a, request(t), pos, last), at[W], at1[W];
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
        if (pos >= 0 && page < 0 && tid == 0 && a.status) set_status(a.status, MOE_ERR_DEVICE);
        // a value's factors: x' = x xx + y yx, y' = y yy + x xy
        float2 xx[N], yx[N], yy[N], xy[N];
        auto factors = [&](const float* w) {
            const float* row = turns + buf * a.rot + it.i0;
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                const float4 u = *reinterpret_cast<const float4*>(w + it.i0 + 2 * e);
                const float4 v = *reinterpret_cast<const float4*>(w + (it.two ? it.i1 : it.i0) + 2 * e);
                xx[e] = make_float2(u.x, u.y);
                xx[e + 1] = make_float2(u.z, u.w);
                yy[e] = make_float2(v.x, v.y);
                yy[e + 1] = make_float2(v.z, v.w);
            }
            if (turn) {
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const float4 c = *reinterpret_cast<const float4*>(row + 2 * e), s = *reinterpret_cast<const float4*>(row + half + 2 * e);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 cc = k ? make_float2(c.z, c.w) : make_float2(c.x, c.y), ss = k ? make_float2(s.z, s.w) : make_float2(s.x, s.y);
                        xy[e + k] = fmul2(xx[e + k], ss);
                        yx[e + k] = fmul2(yy[e + k], make_float2(-ss.x, -ss.y));
                        xx[e + k] = fmul2(xx[e + k], cc);
                        yy[e + k] = fmul2(yy[e + k], cc);
                    }
                }
            }
        };
        auto get = [&](const char* from, float2 (&x)[N], float2 (&y)[N]) {
#pragma unroll
            for (int k = 0; k < 2; ++k, from += THREADS * WB) {
                float2(&f)[N] = k ? y : x;
                if constexpr (BF && VEC == 8) {
                    unpack_bf16x8_f2(*reinterpret_cast<const uint4*>(from), f);
                } else if constexpr (BF) {
                    const uint2 v = *reinterpret_cast<const uint2*>(from);
                    f[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
                    f[1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
                } else {
#pragma unroll
                    for (int e = 0; e < N; e += 2) {
                        const float4 v = *reinterpret_cast<const float4*>(from + 8 * e);
                        f[e] = make_float2(v.x, v.y);
                        f[e + 1] = make_float2(v.z, v.w);
                    }
                }
            }
        };
        // H heads at once, so that one's shuffles and conversions wait beside the other's
        auto norm = [&](auto& x, auto& y) {
            constexpr int H = sizeof(x) / sizeof(float2[N]);
            float all[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                float2 sum = fmul2(x[h][0], x[h][0]);
#pragma unroll
                for (int e = 1; e < N; ++e) sum = ffma2(x[h][e], x[h][e], sum);
#pragma unroll
                for (int e = 0; e < N; ++e) sum = ffma2(y[h][e], y[h][e], sum);
                all[h] = sum.x + sum.y;
            }
#pragma unroll
            for (int o = 16; o > 0; o /= 2)
                if (o < span) {
#pragma unroll
                    for (int h = 0; h < H; ++h) all[h] += __shfl_xor_sync(group, all[h], o);
                }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float r = inv_sqrt(fmaf(all[h], inv_d, a.eps));
                const float2 rr = make_float2(r, r);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float2 f = x[h][e], g = y[h][e];
                    x[h][e] = fmul2(f, xx[e]);
                    y[h][e] = fmul2(g, yy[e]);
                    if (turn) {
                        x[h][e] = ffma2(g, yx[e], x[h][e]);
                        y[h][e] = ffma2(f, xy[e], y[h][e]);
                    }
                    x[h][e] = fmul2(x[h][e], rr);
                    y[h][e] = fmul2(y[h][e], rr);
                }
            }
        };
        auto put = [&](void* p, int type, long long d, const float2 (&x)[N], const float2 (&y)[N], float scale) {
            if (!on) return;
            store_vec<VEC>(p, type, d + it.i0, reinterpret_cast<const float(&)[VEC]>(x), scale);
            if (it.two) store_vec<VEC>(p, type, d + it.i1, reinterpret_cast<const float(&)[VEC]>(y), scale);
        };
        const int q1 = min(a.q_heads, first_q(slice) + nq * lanes), kv1 = page >= 0 ? min(2 * kvh, first_kv(slice) + nkv * lanes) : 0;
        constexpr int kPass = 2 * THREADS * WB, kType = BF ? MOE_DTYPE_BF16 : MOE_DTYPE_F32;
        const char* from = place(buf, 0, 0);
        factors(weights);
        int h = first_q(slice);
        char* to = static_cast<char*>(a.q_out) + (t * a.o_ts + h * a.o_hs) * kSize;
        for (; h + lanes < q1; h += 2 * lanes, from += 2 * kPass, to += 2 * o_step) {
            float2 x[2][N], y[2][N];
            get(from, x[0], y[0]);
            get(from + kPass, x[1], y[1]);
            norm(x, y);
            put(to, kType, 0, x[0], y[0], 1.0f);
            put(to + o_step, kType, 0, x[1], y[1], 1.0f);
        }
        if (h < q1) {
            float2 x[1][N], y[1][N];
            get(from, x[0], y[0]);
            norm(x, y);
            put(to, kType, 0, x[0], y[0], 1.0f);
        }
        from = place(buf, nq, 0);
        const int slot = pos - pos / P * P;
        const long long krow = (long long)page * a.c.k_page_stride + slot * a.c.k_slot_stride, vrow = page * a.c.v_page_stride + slot * a.c.v_slot_stride;
        if (first_kv(slice) < min(kv1, kvh)) factors(weights + D);
        for (int h = first_kv(slice); h < kv1; h += lanes, from += kPass) {
            const bool k = h < kvh;
            float2 x[1][N], y[1][N];
            get(from, x[0], y[0]);
            if (k) norm(x, y);
            put(k ? a.c.k : a.c.v, a.c.dtype, k ? krow + h * a.c.k_head_stride : vrow + (h - kvh) * a.c.v_head_stride, x[0], y[0], inv[h]);
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

template <bool BF, int VEC, int THREADS>
cudaError_t launch_as(const QkAppendArgs& a, cudaStream_t s) {
    const int sms = device_sm_count(), lanes = THREADS / span_of(items_of(a.c.head_dim, a.rot, VEC));
    const int most_q = (a.q_heads + lanes - 1) / lanes, most_kv = (2 * a.c.heads + lanes - 1) / lanes;
    // Few tokens: slices of the heads, until the blocks fill the GPU or a thread has one head.
    int slices = std::max(1, std::min(std::max(most_q, most_kv), 8 * sms / a.T)), nq, nkv;
    size_t smem;
    for (;; ++slices) {      // whole tokens where two units of them fit in shared memory
        nq = (most_q + slices - 1) / slices;
        nkv = (most_kv + slices - 1) / slices;
        smem = (size_t)4 * (nq + nkv) * THREADS * VEC * (BF ? 2 : 4) + (2 * a.rot + 2 * a.c.head_dim + 2 * a.c.heads) * 4;
        if (smem <= (size_t)kAppendSmem || nq + nkv <= 2) break;
    }
    auto kern = qk_append_kernel<BF, VEC, THREADS>;
    static std::atomic<uint64_t> done, blocks;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kAppendSmem, done);
    int per_sm = 0;
    if (e == cudaSuccess) e = blocks_per_sm(reinterpret_cast<const void*>(kern), THREADS, smem, blocks, &per_sm);
    if (e != cudaSuccess) return e;
    const int grid = std::min(a.T * slices, per_sm * sms);
    return launch_pdl(kern, dim3((unsigned)grid), dim3(THREADS), smem, s, a, slices, nq, nkv);
}

// Blocks of 64 threads where 128 would take all heads of q in one turn, and tokens are more than blocks of 128 at once:
// half the instructions that every warp spends on a token as such.  12345, 2000, 800 and 600 tokens of 16 + 4 + 4 heads of 64
// in bf16 28.6, 8.1, 5.5 and 5.5 us with 64 threads, 43.5, 10.2, 6.4 and 4.7 with 128; a token 4.5 and 4.0.  2000 tokens, bf16, with 64
// and 128: 32 heads of 64 9.0 and 10.8, 16 of 80 9.7 and 11.8, of 128 4 heads 8.6 and 11.4, 16 9.7 and 12.1, 8 of 256 11.0 and 12.5; fp32: 16
// of 64 8.9 and 10.6, 8 of 128 9.8 and 11.8, 16 of 80 12.8 and 13.3, of 128 15.2 and 15.1, 8 of 256 15.6 and 15.5, but 32 of 64 14.4 and 13.2.
template <bool BF, int VEC>
cudaError_t launch(const QkAppendArgs& a, cudaStream_t s) {
    const bool narrow = a.T > 4 * device_sm_count() && a.q_heads * span_of(items_of(a.c.head_dim, a.rot, VEC)) <= 128;
    return narrow ? launch_as<BF, VEC, 64>(a, s) : launch_as<BF, VEC, 128>(a, s);
}

}  // namespace

cudaError_t launch_qk_norm_append(const QkAppendArgs& a, cudaStream_t s) {
    const bool bf = a.in_dt == MOE_DTYPE_BF16;
    const int heads = a.q_heads + 2 * a.c.heads, size = bf ? 2 : 4;
    // Vectors of 8 or 4 elements where every offset is a multiple of them (and units and scales are no more than the
    // kernel's integers and shared memory take)
    auto fits = [&](int vec) {
        const long long strides = a.k_ts | a.k_hs | a.v_ts | a.v_hs | a.q_ts | a.q_hs | a.o_ts | a.o_hs;
        const uintptr_t p = (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.q | (uintptr_t)a.q_out;
        return a.rot % (2 * vec) == 0 && strides % vec == 0 && p % std::min(vec * size, 16) == 0 && ((uintptr_t)a.cos_sin & 15) == 0 &&
               a.c.heads <= 8192 && (long long)a.T * heads <= 1 << 30;
    };
    if (fits(8)) return bf ? launch<true, 8>(a, s) : launch<false, 8>(a, s);
    if (fits(4)) return bf ? launch<true, 4>(a, s) : launch<false, 4>(a, s);
    const int slices = std::max(1, std::min({(heads + 3) / 4, 8 * device_sm_count() / a.T, 65535}));
    return launch_pdl(bf ? qk_append_any_kernel<true> : qk_append_any_kernel<false>, dim3((unsigned)a.T, (unsigned)slices),
                      dim3(kAppendThreads), 0, s, a);
}

}  // namespace moe
