// Attention of one new token per request over the paged cache: a block per
// (request, query head), its warps striding over the keys with a running
// maximum and sum each, joined in shared memory at the end.
#include <math_constants.h>

#include "block.h"

namespace moe {

namespace {

constexpr int kAttnWarps = 8;

__device__ __forceinline__ float cache_elem(const void* p, int dt, long long i) {
    if (dt == MOE_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return unpack_e4m3x2(static_cast<const uint8_t*>(p)[i]).x;
}

__global__ void __launch_bounds__(kAttnWarps * 32) attn_kernel(const __grid_constant__ AttnArgs a) {
    pdl_allow_dependents();
    pdl_wait_primary();
    const int b = blockIdx.x, h = blockIdx.y, g = h / a.group;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = a.c.head_dim, P = a.c.page_size;
    int n = max(a.seq_lens[b], 0);
    if ((long long)n > (long long)a.max_pages * P) {
        n = a.max_pages * P;
        if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE);
    }
    const int first = a.window > 0 ? max(0, n - a.window) : 0;
    float q[8], o[8];
    const float ks = a.c.k_scale ? a.c.k_scale[g] : 1.0f, vs = a.c.v_scale ? a.c.v_scale[g] : 1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = e * 32 + lane;
        q[e] = o[e] = 0.0f;
        if (c < D) {
            const long long i = b * a.q_bs + h * a.q_hs + c;
            q[e] = a.q_dt == MOE_DTYPE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[i])
                                            : static_cast<const float*>(a.q)[i];
        }
    }
    float m = -CUDART_INF_F, l = 0.0f;
    for (int j = first + warp; j < n; j += kAttnWarps) {
        const int page = a.table[b * a.table_ld + j / P];
        if (page < 0 || page >= a.c.num_pages) {
            set_status(a.status, MOE_ERR_DEVICE);
            continue;
        }
        const long long kb = page * a.c.k_page_stride + (j % P) * a.c.k_slot_stride + g * a.c.k_head_stride;
        const long long vb = page * a.c.v_page_stride + (j % P) * a.c.v_slot_stride + g * a.c.v_head_stride;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e * 32 + lane < D) s = fmaf(q[e], cache_elem(a.c.k, a.c.dtype, kb + e * 32 + lane), s);
        s = warp_sum(s) * ks * a.scale;
        if (a.softcap > 0.0f) s = a.softcap * tanhf(s / a.softcap);
        if (s == -CUDART_INF_F) continue;   // weighs nothing, also before the first finite score
        const float mn = fmaxf(m, s), corr = m == mn ? 1.0f : expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * corr + p;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e * 32 + lane < D)
                o[e] = o[e] * corr + p * cache_elem(a.c.v, a.c.dtype, vb + e * 32 + lane);
    }
    __shared__ float s_m[kAttnWarps], s_l[kAttnWarps], s_o[kAttnWarps][256];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s_o[warp][e * 32 + lane] = o[e];
    __syncthreads();
    float top = -CUDART_INF_F, sum = 0.0f, val = 0.0f;
    for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, s_m[w]);
    const int c = threadIdx.x;
    for (int w = 0; w < kAttnWarps; ++w) {
        if (s_l[w] == 0.0f) continue;
        const float f = expf(s_m[w] - top);
        sum += f * s_l[w];
        val += f * s_o[w][c];
    }
    if (c < D) {
        const float r = sum == 0.0f ? 0.0f : val / sum * vs;
        const long long i = b * a.o_bs + h * a.o_hs + c;
        if (a.o_dt == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(r);
        else static_cast<float*>(a.out)[i] = r;
    }
    if (a.lse && c == 0) a.lse[(long long)b * a.q_heads + h] = sum == 0.0f ? -CUDART_INF_F : top + logf(sum);
}

}  // namespace

size_t attn_workspace_bytes(int, int, int, int, size_t* done_off, size_t* parts_off) {
    *done_off = *parts_off = 512;
    return 512;
}

cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t s) {
    return launch_pdl(attn_kernel, dim3((unsigned)a.B, (unsigned)a.q_heads), dim3(kAttnWarps * 32), 0, s, a);
}

}  // namespace moe
