// Rotary position encoding of q and k, and the new tokens' k, v rows into the
// paged cache.  Element i < rot / 2 of a head turns with element i + rot / 2:
//   a' = a cos - b sin,  b' = b cos + a sin.
//
// One block per token (and per slice of its work): an item is one vector of
// VEC elements of a head, or both vectors of a rotated pair, which one thread
// takes so that each element is read once.
#include "block.h"

namespace moe {

namespace {

constexpr int kAppendThreads = 256;

template <int VEC>
__device__ __forceinline__ void load_vec(const void* p, int dt, long long i, float (&f)[VEC]) {
    if constexpr (VEC == 8) {
        load8_f32(p, dt, i, f);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            f[e] = dt == MOE_DTYPE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i + e])
                                        : static_cast<const float*>(p)[i + e];
    }
}

template <int VEC>
__device__ __forceinline__ void store_vec(void* p, int dt, long long i, const float (&f)[VEC], float scale) {
    if (dt == MOE_DTYPE_FP8_E4M3) {
        float g[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[e] = f[e] / scale;
        uint8_t* b = static_cast<uint8_t*>(p) + i;
        if constexpr (VEC == 8) {
            *reinterpret_cast<uint2*>(b) = make_uint2(pack_e4m3x4(g[0], g[1], g[2], g[3]),
                                                      pack_e4m3x4(g[4], g[5], g[6], g[7]));
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) b[e] = (uint8_t)__nv_cvt_float_to_fp8(g[e], __NV_SATFINITE, __NV_E4M3);
        }
    } else if constexpr (VEC == 8) {
        store8(p, dt, i, f);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (dt == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(p)[i + e] = __float2bfloat16_rn(f[e]);
            else static_cast<float*>(p)[i + e] = f[e];
        }
    }
}

template <int VEC>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    pdl_allow_dependents();
    pdl_wait_primary();
    const int t = blockIdx.x;
    const int pos = a.positions[t];
    const int req = a.req ? a.req[t] : t;
    const int P = a.c.page_size;
    // the token's slot, or no slot
    long long page = -1;
    int slot = 0;
    bool dropped = false;
    if (pos >= 0) {
        dropped = req < 0 || req >= a.R || pos / P >= a.max_pages || (a.rot && pos >= a.max_pos);
        if (!dropped) {
            page = a.table[req * a.table_ld + pos / P];
            slot = pos % P;
            if (page < 0 || page >= a.c.num_pages) {
                page = -1;
                dropped = true;
            }
        }
        if (dropped && a.status && threadIdx.x == 0 && blockIdx.y == 0) set_status(a.status, MOE_ERR_DEVICE);
    }
    // padding and tokens without a row in cos_sin keep their q as it is
    const int half = pos >= 0 && a.rot && pos < a.max_pos ? a.rot / 2 : 0;
    const int D = a.c.head_dim;
    const int pairs = half / VEC, items = pairs + (D - 2 * half) / VEC;
    const int heads = a.c.heads, total = (a.q_heads + 2 * heads) * items;
    for (int w = blockIdx.y * kAppendThreads + threadIdx.x; w < total; w += gridDim.y * kAppendThreads) {
        int h = w / items;
        const int it = w - h * items;
        const void* src;
        void* dst;
        long long si, di;
        int dt;
        float scale = 1.0f;
        bool is_v = false;
        if (h < a.q_heads) {
            src = a.q; si = t * a.q_ts + h * a.q_hs;
            dst = a.q_out; di = t * a.o_ts + h * a.o_hs;
            dt = a.in_dt;
        } else if (page < 0) {
            continue;
        } else if ((h -= a.q_heads) < heads) {
            src = a.k; si = t * a.k_ts + h * a.k_hs;
            dst = a.c.k; di = page * a.c.k_page_stride + slot * a.c.k_slot_stride + h * a.c.k_head_stride;
            dt = a.c.dtype;
            if (a.c.k_scale) scale = a.c.k_scale[h];
        } else {
            h -= heads;
            is_v = true;
            src = a.v; si = t * a.v_ts + h * a.v_hs;
            dst = a.c.v; di = page * a.c.v_page_stride + slot * a.c.v_slot_stride + h * a.c.v_head_stride;
            dt = a.c.dtype;
            if (a.c.v_scale) scale = a.c.v_scale[h];
        }
        if (it < pairs) {
            const int i = it * VEC;
            float u[VEC], w2[VEC];
            load_vec<VEC>(src, a.in_dt, si + i, u);
            load_vec<VEC>(src, a.in_dt, si + i + half, w2);
            if (!is_v) {
                const float* cs = a.cos_sin + (long long)pos * a.rot + i;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float c = cs[e], sn = cs[half + e], x0 = u[e], x1 = w2[e];
                    u[e] = x0 * c - x1 * sn;
                    w2[e] = x1 * c + x0 * sn;
                }
            }
            store_vec<VEC>(dst, dt, di + i, u, scale);
            store_vec<VEC>(dst, dt, di + i + half, w2, scale);
        } else {
            const int i = 2 * half + (it - pairs) * VEC;
            float u[VEC];
            load_vec<VEC>(src, a.in_dt, si + i, u);
            store_vec<VEC>(dst, dt, di + i, u, scale);
        }
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
    const int work = (a.q_heads + 2 * a.c.heads) * a.c.head_dim / vec;
    const int slices = (work + 4 * kAppendThreads - 1) / (4 * kAppendThreads);
    const dim3 grid((unsigned)a.T, (unsigned)slices);
    return launch_pdl(vec8 ? kv_append_kernel<8> : kv_append_kernel<1>, grid, dim3(kAppendThreads), 0, s, a);
}

}  // namespace moe
