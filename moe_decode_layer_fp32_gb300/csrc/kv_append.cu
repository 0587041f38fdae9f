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
// Measured, 12345 tokens of 56 + 8 + 8 heads of 128, bf16 into E4M3, half of each head rotated
// (431 MB): 66 us, 6.5 TB/s; a block per token without the copies ahead 86 us.  A page looked at where
// it is loaded 73 us, the units' divisions in the loop 71 us, tokens in two slices 93 us; at 56
// registers instead of 72 (9 blocks per SM instead of 7) 69 us.
#include <algorithm>

#include "append.cuh"

namespace moe {

namespace {

constexpr int kVec = 8;                     // elements of a vector

// With a rotation the rows of cos_sin say which positions there are.
__device__ __forceinline__ int last_of(const AppendArgs& a) { return a.rot ? a.max_pos - 1 : INT_MAX; }
// Items of a head of 16-byte vectors: the pairs that turn, and the others two by two.
__host__ __device__ inline int items_of(int D, int rot) { return rot / 2 / kVec + ((D - rot) / kVec + 1) / 2; }

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

// 16-byte vectors.  A unit is a token and a slice of its heads, nq of q's and nkv of k's and v's to a
// thread at most; a block takes units blockIdx.x, + gridDim.x, ..., with the next one's rows on
// their way into shared memory (every thread's own vectors into places of its own) while it
// turns and stores the current one's.
template <bool BF>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendArgs a, int slices, int nq, int nkv) {
    constexpr int WB = BF ? 16 : 32;                          // bytes of a vector
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, D = a.c.head_dim, kvh = a.c.heads, P = a.c.page_size, n = nq + nkv;
    const int items = items_of(D, a.rot), lanes = kAppendThreads / items, hl = tid / items;
    float* turns = reinterpret_cast<float*>(smem + 4 * n * kAppendThreads * WB);   // [2][rot], behind the rows
    float* inv = turns + 2 * a.rot;                           // [2 kvh] 1 / scale of E4M3 rows
    Item<kVec> it;
    it.place(tid - hl * items, D, a.rot / 2);
    pdl_allow_dependents();
    pdl_wait_primary();
    for (int i = tid; i < 2 * kvh; i += kAppendThreads) {
        const float* scale = i < kvh ? a.c.k_scale : a.c.v_scale;
        inv[i] = scale ? 1.0f / scale[i < kvh ? i : i - kvh] : 1.0f;
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
    auto fetch = [&](int buf, int t, int slice, int pos) {
        for (int s = 0, h = first_q(slice); s < nq && h < a.q_heads; ++s, h += lanes) {
            const long long o = t * a.q_ts + h * a.q_hs;
            copy(place(buf, s, 0), a.q, o + it.i0);
            if (it.two) copy(place(buf, s, 1), a.q, o + it.i1);
        }
        for (int s = nq, h = first_kv(slice); pos >= 0 && s < n && h < 2 * kvh; ++s, h += lanes) {
            const bool k = h < kvh;
            const void* p = k ? a.k : a.v;
            const long long o = k ? t * a.k_ts + h * a.k_hs : t * a.v_ts + (h - kvh) * a.v_hs;
            copy(place(buf, s, 0), p, o + it.i0);
            if (it.two) copy(place(buf, s, 1), p, o + it.i1);
        }
        if (pos >= 0 && pos < a.max_pos)
            for (int w = tid * 4; w < a.rot; w += kAppendThreads * 4)
                cp_async16(turns + buf * a.rot + w, a.cos_sin + (long long)pos * a.rot + w);
        cp_async_commit();
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
    int pos = position(t), pos1 = position(t1), req1 = request(t1), entry = page_of(a, request(t), pos, last);
    fetch(0, t, slice, pos);
    for (int buf = 0; t < a.T; buf ^= 1) {
        cp_async_wait<0>();
        __syncthreads();       // the turns are there, and nobody reads the other half's any more
        if (t1 < a.T) fetch(buf ^ 1, t1, slice1, pos1);
        advance(t2, slice2);
        const int entry1 = page_of(a, req1, pos1, last), pos2 = position(t2), req2 = request(t2);
        const int page = entry < a.c.num_pages ? entry : -1;
        // padding and tokens without a row in cos_sin keep their q as it is
        const bool turn = it.turn && pos >= 0 && pos < a.max_pos;
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
        for (int s = 0, h = first_q(slice); s < nq && h < a.q_heads; ++s, h += lanes) {
            get(s);
            if (turn) it.rotate(x, y);
            const long long d = t * a.o_ts + h * a.o_hs;
            store8(a.q_out, a.in_dt, d + it.i0, x);
            if (it.two) store8(a.q_out, a.in_dt, d + it.i1, y);
        }
        for (int s = nq, h = first_kv(slice); page >= 0 && s < n && h < 2 * kvh; ++s, h += lanes) {
            get(s);
            const bool k = h < kvh;
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

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s) {
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
        const int most = (heads * ((a.c.head_dim + 1) / 2) + kAppendThreads - 1) / kAppendThreads;
        const int slices = std::max(1, std::min(most, 8 * sms / a.T));
        return launch_pdl(bf ? kv_append_any_kernel<true> : kv_append_any_kernel<false>, dim3((unsigned)a.T, (unsigned)slices),
                          dim3(kAppendThreads), 0, s, a);
    }
    const int lanes = kAppendThreads / items_of(a.c.head_dim, a.rot);
    const int most_q = (a.q_heads + lanes - 1) / lanes, most_kv = (2 * a.c.heads + lanes - 1) / lanes;
    int slices = std::max(1, std::min(std::max(most_q, most_kv), 8 * sms / a.T)), nq, nkv;
    size_t smem;
    for (;; ++slices) {      // whole tokens where two units of them fit in shared memory
        nq = (most_q + slices - 1) / slices;
        nkv = (most_kv + slices - 1) / slices;
        smem = (size_t)4 * (nq + nkv) * kAppendThreads * (bf ? 16 : 32) + (2 * a.rot + 2 * a.c.heads) * 4;
        if (smem <= (size_t)kAppendSmem || nq + nkv <= 2) break;
    }
    auto kern = bf ? kv_append_kernel<true> : kv_append_kernel<false>;
    static std::atomic<uint64_t> done[2], blocks[2];
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kAppendSmem, done[bf]);
    int per_sm = 0;
    if (e == cudaSuccess) e = blocks_per_sm(reinterpret_cast<const void*>(kern), kAppendThreads, smem, blocks[bf], &per_sm);
    if (e != cudaSuccess) return e;
    const int grid = std::min(a.T * slices, per_sm * sms);
    return launch_pdl(kern, dim3((unsigned)grid), dim3(kAppendThreads), smem, s, a, slices, nq, nkv);
}

}  // namespace moe
