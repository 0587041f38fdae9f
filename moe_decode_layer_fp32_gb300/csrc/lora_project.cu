// Shared projection with low-rank adapters: y[t] = W x[t] + s_a B_a (A_a x[t]).
// Two kernels: v[t] = A_a x[t], then a warp per output row n that keeps the
// row of W and of each token's B_a against x[t] and v[t].
#include "block.h"

namespace moe {

namespace {

__device__ __forceinline__ void load8_any(const void* p, int dt, long long i, float (&f)[8]) {
    if (dt == MOE_DTYPE_FP8_E4M3) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + i);
        const uint32_t w[4] = {v.x, v.x >> 16, v.y, v.y >> 16};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 u = unpack_e4m3x2(w[e]);
            f[2 * e] = u.x;
            f[2 * e + 1] = u.y;
        }
    } else {
        load8_f32(p, dt, i, f);
    }
}

__device__ __forceinline__ int adapter_of(const LoraArgs& a, int t) {
    const int i = a.adapter[t];
    if (i >= a.na) set_status(a.status, MOE_ERR_DEVICE);
    return i >= 0 && i < a.na ? i : -1;
}

// A warp per (token, rank index).
__global__ void __launch_bounds__(256) lora_shrink_kernel(const __grid_constant__ LoraArgs a) {
    pdl_allow_dependents();
    pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    const int w = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= a.T * a.r) return;
    const int t = w / a.r, j = w - t * a.r;
    const int ad = adapter_of(a, t);
    float sum = 0.0f;
    if (ad >= 0) {
        const __nv_bfloat16* row = a.la + ((long long)ad * a.r + j) * a.d;
        for (int c = lane * 8; c < a.d; c += 256) {
            float u[8], x[8];
            load8_f32(row, MOE_DTYPE_BF16, c, u);
            load8_any(a.x, a.x_dt, t * a.x_ld + c, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(u[e], x[e], sum);
        }
    }
    sum = warp_sum(sum);
    if (lane == 0) a.v[t * a.r + j] = ad < 0 ? 0.0f : a.x_scale ? sum * a.x_scale[t] : sum;
}

// A warp per output row.
__global__ void __launch_bounds__(256) lora_project_kernel(const __grid_constant__ LoraArgs a) {
    pdl_allow_dependents();
    pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (n >= a.N) return;
    const int wdt = a.w_scale ? MOE_DTYPE_FP8_E4M3 : MOE_DTYPE_BF16;
    for (int t = 0; t < a.T; ++t) {
        float sum = 0.0f;
        for (int c = lane * 8; c < a.d; c += 256) {
            float u[8], x[8];
            load8_any(a.w, wdt, n * a.w_ld + c, u);
            load8_any(a.x, a.x_dt, t * a.x_ld + c, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(u[e], x[e], sum);
        }
        sum = warp_sum(sum);
        if (a.w_scale) sum *= a.w_scale[n] * a.x_scale[t];
        if (a.r > 0) {
            const int ad = adapter_of(a, t);
            if (ad >= 0) {
                float low = 0.0f;
                for (int j = lane; j < a.r; j += 32)
                    low = fmaf(__bfloat162float(a.lb[((long long)ad * a.N + n) * a.r + j]), a.v[t * a.r + j], low);
                sum += a.ls[ad] * warp_sum(low);
            }
        }
        if (lane == 0) {
            if (a.y_dt == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.y)[t * a.y_ld + n] = __float2bfloat16_rn(sum);
            else static_cast<float*>(a.y)[t * a.y_ld + n] = sum;
        }
    }
}

}  // namespace

size_t lora_workspace_bytes(int T, int d, int r, size_t* v_off, size_t* xs_off) {
    size_t off = 512;
    *v_off = off;
    off += ((size_t)T * r * 4 + 255) / 256 * 256;
    *xs_off = off;
    return off + (size_t)T * d * 6;
}

cudaError_t launch_lora_project(const LoraArgs& a, cudaStream_t s) {
    if (a.r > 0) {
        const cudaError_t e = launch_pdl(lora_shrink_kernel, dim3((unsigned)((a.T * a.r + 7) / 8)), dim3(256), 0, s, a);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(lora_project_kernel, dim3((unsigned)((a.N + 7) / 8)), dim3(256), 0, s, a);
}

}  // namespace moe
