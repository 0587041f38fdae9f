// Rotary position encoding of q and k, and the new tokens' k, v rows into the
// paged cache.  Element i < rot / 2 of a head turns with element i + rot / 2:
//   a' = a cos - b sin,  b' = b cos + a sin.
//
// HBM bounds many tokens, latency a few.  An item of a head is two vectors of VEC elements,
// a rotated pair or two of the others; a thread has the same item of several heads, so that
// each element is read once and cos, sin once for all heads.  The loads of kBatch heads are
// issued together, and those of the first heads before the token's page is known.
//
// Measured, 12345 tokens of 56 + 8 + 8 heads of 128, bf16 into E4M3, half of each head rotated
// (431 MB): 86 us, 5.0 TB/s.  Batches of 2 heads at 80 registers (6 blocks of 128 per SM); at 64
// registers (8 blocks) 91 us, batches of 3 at the same registers 94 to 103 us; one head at a time
// with an item's vectors taken alone 126 us.
#include <algorithm>

#include "block.h"

namespace moe {

namespace {

constexpr int kAppendThreads = 128;
constexpr int kBatch = 2;

template <int VEC, bool BF>
struct RawVec {
    static constexpr int kWords = VEC * (BF ? 2 : 4) / 16;    // 16-byte words (VEC 8)
    uint4 w[kWords > 0 ? kWords : 1];
    float s;                                                   // VEC 1
    __device__ __forceinline__ void load(const void* p, long long i) {
        if constexpr (VEC == 8) {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (BF ? 2 : 4));
#pragma unroll
            for (int k = 0; k < kWords; ++k) w[k] = q[k];
        } else {
            s = BF ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
        }
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const {
        if constexpr (VEC == 1) {
            f[0] = s;
        } else if constexpr (BF) {
            unpack_bf16x8(w[0], f);
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                f[4 * k] = __uint_as_float(w[k].x);
                f[4 * k + 1] = __uint_as_float(w[k].y);
                f[4 * k + 2] = __uint_as_float(w[k].z);
                f[4 * k + 3] = __uint_as_float(w[k].w);
            }
        }
    }
};

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
    float cs[VEC], sn[VEC];
    __device__ __forceinline__ void rotate(float (&x)[VEC], float (&y)[VEC]) const {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float f = x[e], g = y[e];
            x[e] = f * cs[e] - g * sn[e];
            y[e] = g * cs[e] + f * sn[e];
        }
    }
};

// Heads first, first + step, ... < n of a row [heads, D]: kBatch heads' loads, then `place` (once),
// then their stores.
template <int VEC, bool BF, class Src, class Place, class Dst>
__device__ __forceinline__ void take_heads(const Item<VEC>& it, int first, int step, int n, Src src, Place place, Dst dst) {
    bool placed = false;
    for (int h0 = first; h0 < n; h0 += kBatch * step) {
        RawVec<VEC, BF> u[kBatch], v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int h = h0 + b * step;
            if (h < n) src(h, u[b], v[b]);
        }
        if (!placed) {
            placed = true;
            if (!place()) return;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int h = h0 + b * step;
            if (h < n) dst(h, u[b], v[b]);
        }
    }
}

// Grid: x = token, y = slice of the heads.
template <int VEC, bool BF>
__global__ void __launch_bounds__(kAppendThreads, 6) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    pdl_allow_dependents();
    pdl_wait_primary();
    const int t = blockIdx.x;
    const int pos = a.positions[t];
    // padding and tokens without a row in cos_sin keep their q as it is
    const int half = pos >= 0 && a.rot && pos < a.max_pos ? a.rot / 2 : 0;
    const int D = a.c.head_dim, kvh = a.c.heads;
    // items of a head: the pairs of vectors that turn, then the others two by two
    const int pairs = half / VEC, plain = (D - 2 * half) / VEC, items = pairs + (plain + 1) / 2;
    const int width = min(items, kAppendThreads), lanes = kAppendThreads / width;
    const int hl = threadIdx.x / width, step = lanes * gridDim.y, first = blockIdx.y * lanes + hl;
    if (hl >= lanes) return;
    for (int i = threadIdx.x - hl * width; i < items; i += width) {
        Item<VEC> it;
        it.turn = i < pairs;
        if (it.turn) {
            it.i0 = i * VEC;
            it.i1 = it.i0 + half;
            it.two = true;
            const float* row = a.cos_sin + (long long)pos * a.rot + it.i0;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                it.cs[e] = row[e];
                it.sn[e] = row[half + e];
            }
        } else {
            const int k = i - pairs, k1 = k + (plain + 1) / 2;
            it.i0 = 2 * half + k * VEC;
            it.i1 = 2 * half + k1 * VEC;
            it.two = k1 < plain;
        }
        using Raw = RawVec<VEC, BF>;
        // q
        take_heads<VEC, BF>(
            it, first, step, a.q_heads,
            [&](int h, Raw& u, Raw& v) {
                const long long s = t * a.q_ts + h * a.q_hs;
                u.load(a.q, s + it.i0);
                if (it.two) v.load(a.q, s + it.i1);
            },
            [] { return true; },
            [&](int h, const Raw& u, const Raw& v) {
                float x[VEC], y[VEC];
                u.get(x);
                v.get(y);
                if (it.turn) it.rotate(x, y);
                const long long d = t * a.o_ts + h * a.o_hs;
                store_vec<VEC>(a.q_out, a.in_dt, d + it.i0, x, 1.0f);
                if (it.two) store_vec<VEC>(a.q_out, a.in_dt, d + it.i1, y, 1.0f);
            });
        // k, then v: heads 0 .. 2 kvh - 1
        long long page = -1;
        int slot = 0;
        if (pos < 0) continue;
        take_heads<VEC, BF>(
            it, first, step, 2 * kvh,
            [&](int h, Raw& u, Raw& v) {
                const void* p = h < kvh ? a.k : a.v;
                const long long s = h < kvh ? t * a.k_ts + h * a.k_hs : t * a.v_ts + (h - kvh) * a.v_hs;
                u.load(p, s + it.i0);
                if (it.two) v.load(p, s + it.i1);
            },
            [&] {
                const int req = a.req ? a.req[t] : t, P = a.c.page_size, col = pos / P;
                bool dropped = req < 0 || req >= a.R || col >= a.max_pages || (a.rot && pos >= a.max_pos);
                if (!dropped) {
                    page = a.table[req * a.table_ld + col];
                    slot = pos - col * P;
                    dropped = page < 0 || page >= a.c.num_pages;
                }
                if (dropped && a.status) set_status(a.status, MOE_ERR_DEVICE);
                return !dropped;
            },
            [&](int h, const Raw& u, const Raw& v) {
                float x[VEC], y[VEC];
                u.get(x);
                v.get(y);
                const bool k = h < kvh;
                const int g = k ? h : h - kvh;
                if (it.turn && k) it.rotate(x, y);
                const float* scale = k ? a.c.k_scale : a.c.v_scale;
                const float inv = scale ? 1.0f / scale[g] : 1.0f;
                void* p = k ? a.c.k : a.c.v;
                const long long d = k ? page * a.c.k_page_stride + slot * a.c.k_slot_stride + g * a.c.k_head_stride
                                      : page * a.c.v_page_stride + slot * a.c.v_slot_stride + g * a.c.v_head_stride;
                store_vec<VEC>(p, a.c.dtype, d + it.i0, x, inv);
                if (it.two) store_vec<VEC>(p, a.c.dtype, d + it.i1, y, inv);
            });
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s) {
    // 16-byte vectors where every offset is a multiple of 8 elements
    auto m8 = [](long long v) { return v % 8 == 0; };
    const bool vec8 = a.rot % 16 == 0 && m8(a.k_ts) && m8(a.k_hs) && m8(a.v_ts) && m8(a.v_hs) && m8(a.q_ts) &&
                      m8(a.q_hs) && m8(a.o_ts) && m8(a.o_hs) &&
                      (((uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.q | (uintptr_t)a.q_out) & 15) == 0;
    const int vec = vec8 ? 8 : 1;
    // Few tokens: slices of the heads, until the blocks fill the GPU or a thread has one head.
    const int items = std::max(1, (a.c.head_dim / vec + 1) / 2), lanes = std::max(1, kAppendThreads / items);
    const int most = (std::max(a.q_heads, 2 * a.c.heads) + lanes - 1) / lanes;
    const int slices = std::max(1, std::min(most, 8 * device_sm_count() / a.T));
    const bool bf = a.in_dt == MOE_DTYPE_BF16;
    auto kern = vec8 ? (bf ? kv_append_kernel<8, true> : kv_append_kernel<8, false>)
                     : (bf ? kv_append_kernel<1, true> : kv_append_kernel<1, false>);
    return launch_pdl(kern, dim3((unsigned)a.T, (unsigned)slices), dim3(kAppendThreads), 0, s, a);
}

}  // namespace moe
