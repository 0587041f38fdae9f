// Root-mean-square norm with the residual's addition and an optional E4M3
// output: z = x + residual, y = z / sqrt(mean(z^2) + eps) * weight.
//
// One block per row holds the row in registers between the sum of squares and
// the output, so that each input is read once.
#include "block.h"

namespace moe {

namespace {

template <int CH>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const __grid_constant__ NormArgs a) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    __shared__ float s_sum[32], s_max[32];
    const long long t = blockIdx.x;
    pdl_allow_dependents();
    pdl_wait_primary();
    float z[CH][8];
    float sum = 0.0f, mx = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (j * blockDim.x + tid) * 8;
        if (c < a.d) {
            load8_f32(a.x, a.x_dt, t * a.x_ld + c, z[j]);
            if (a.residual) {
                float r[8];
                load8_f32(a.residual, a.r_dt, t * a.r_ld + c, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) z[j][e] += r[e];
            }
            if (a.residual_out) store8(a.residual_out, a.r_dt, t * a.ro_ld + c, z[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(z[j][e], z[j][e], sum);
            if (a.weight) {
                float w[8];
                load8_f32(a.weight, a.w_dt, c, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) z[j][e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(z[j][e]));
        }
    }
    sum = warp_sum(sum);
    if (a.y_scale && a.group == 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if (lane == 0) {
        s_sum[warp] = sum;
        s_max[warp] = mx;
    }
    __syncthreads();
    sum = 0.0f;
    mx = 0.0f;
    for (int w = 0; w < nw; ++w) {
        sum += s_sum[w];
        mx = fmaxf(mx, s_max[w]);
    }
    const float rstd = 1.0f / sqrtf(sum / (float)a.d + a.eps);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (j * blockDim.x + tid) * 8;
        float amax = mx * rstd;
        if (a.group) {
            amax = 0.0f;
            if (c < a.d) {
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(z[j][e]));
            }
            __syncwarp();
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            amax *= rstd;
        }
        if (c >= a.d) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) z[j][e] *= rstd;
        if (a.y_scale) {
            const float scale = amax > 0.0f ? amax / 448.0f : 1.0f;
            if (a.group) {
                if (c % a.group == 0) a.y_scale[t * (a.d / a.group) + c / a.group] = scale;
            } else if (c == 0) {
                a.y_scale[t] = scale;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) z[j][e] /= scale;
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + t * a.y_ld + c) =
                make_uint2(pack_e4m3x4(z[j][0], z[j][1], z[j][2], z[j][3]),
                           pack_e4m3x4(z[j][4], z[j][5], z[j][6], z[j][7]));
        } else {
            store8(a.y, a.y_dt, t * a.y_ld + c, z[j]);
        }
    }
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t s) {
    const int chunks = a.d / 8;
    const int ch = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
    const int threads = ((chunks + ch - 1) / ch + 31) / 32 * 32;
    auto kern = ch == 1 ? rmsnorm_kernel<1> : ch == 2 ? rmsnorm_kernel<2> : rmsnorm_kernel<4>;
    return launch_pdl(kern, dim3((unsigned)a.T), dim3((unsigned)threads), 0, s, a);
}

}  // namespace moe
