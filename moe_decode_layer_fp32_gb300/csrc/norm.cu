// Root-mean-square norm with the residual's addition and an optional E4M3
// output: z = x + residual, y = z / sqrt(mean(z^2) + eps) * weight.
//
// HBM bounds many rows, latency a few.  A block holds a row in registers between
// the sum of squares and the output, so that each input is read once, and needs one
// barrier for it: the row's amax is max |z w| times the same factor, taken together with the sum.
// Many rows: as many blocks as the GPU holds walk over them, each with the next row's
// copy in flight while it finishes the current one; few rows: one block each, of as many
// threads as the row has 8-element chunks.
//
// Measured, 8191 x 7168 bf16 + residual -> E4M3 by 128 columns (413 MB): 78 us, 5.3 TB/s.  Blocks
// of 256 threads (4 chunks each) 110 us, of 896 (1 chunk) 86 us, a ring of 3 rows (2 blocks per
// SM instead of 3) 89 us; one row per block without a ring 125 us.
#include <algorithm>

#include "block.h"

namespace moe {

namespace {

constexpr int kWalkThreads = 512;    // most threads of a block that walks over rows
constexpr int kDepth = 2;            // rows of a thread's ring

template <bool BF>
__device__ __forceinline__ void raw8(const char* p, float (&f)[8]) {
    if constexpr (BF) {
        unpack_bf16x8(*reinterpret_cast<const uint4*>(p), f);
    } else {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}
template <bool BF>
__device__ __forceinline__ void copy8(char* dst, const void* src, long long i) {
    const char* s = static_cast<const char*>(src) + i * (BF ? 2 : 4);
    cp_async16(dst, s);
    if constexpr (!BF) cp_async16(dst + 16, s + 16);
}
__device__ __forceinline__ float warp_max(float v) {
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// CH: chunks of 8 elements a thread holds.  XBF, RBF: x, residual in bf16.  WALK: the block
// takes rows blockIdx.x, + gridDim.x, ..., and every thread copies its own chunks of the
// rows ahead into a ring of its own in shared memory (which needs no barrier).
template <int CH, bool XBF, bool RBF, bool WALK>
__global__ void __launch_bounds__(WALK ? kWalkThreads : 1024) rmsnorm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int XB = XBF ? 16 : 32, RB = RBF ? 16 : 32;
    extern __shared__ __align__(16) char ring[];
    __shared__ float s_sum[2][32], s_max[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5, nt = blockDim.x;
    pdl_allow_dependents();
    pdl_wait_primary();
    // chunk j of ring row s: 16-byte words of a warp's lanes next to one another
    auto at = [&](int s, int j) { return ring + ((s * CH + j) * nt + tid) * XB; };
    auto at_r = [&](int s, int j) { return ring + kDepth * CH * nt * XB + ((s * CH + j) * nt + tid) * RB; };
    auto fetch = [&](int s, long long t) {
        if (t < a.T) {
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int c = (j * nt + tid) * 8;
                if (c < a.d) {
                    copy8<XBF>(at(s, j), a.x, t * a.x_ld + c);
                    if (a.residual) copy8<RBF>(at_r(s, j), a.residual, t * a.r_ld + c);
                }
            }
        }
        cp_async_commit();
    };
    if constexpr (WALK) {
        for (int s = 0; s < kDepth - 1; ++s) fetch(s, blockIdx.x + (long long)s * gridDim.x);
    }
    int phase = 0, row = 0;
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
        float z[CH][8];
        float sum = 0.0f, mx = 0.0f;
        if constexpr (WALK) {
            cp_async_wait<kDepth - 2>();
        }
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (j * nt + tid) * 8;
            if (c < a.d) {
                if constexpr (WALK) raw8<XBF>(at(row, j), z[j]);
                else load8_f32(a.x, XBF ? MOE_DTYPE_BF16 : MOE_DTYPE_F32, t * a.x_ld + c, z[j]);
                if (a.residual) {
                    float u[8];
                    if constexpr (WALK) raw8<RBF>(at_r(row, j), u);
                    else load8_f32(a.residual, RBF ? MOE_DTYPE_BF16 : MOE_DTYPE_F32, t * a.r_ld + c, u);
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[j][e] += u[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) z[j][e] = 0.0f;
            }
        }
        if constexpr (WALK) {
            fetch(row == 0 ? kDepth - 1 : row - 1, t + (long long)(kDepth - 1) * gridDim.x);
            row = row + 1 == kDepth ? 0 : row + 1;
        }
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (j * nt + tid) * 8;
            if (a.residual_out && c < a.d) store8(a.residual_out, a.r_dt, t * a.ro_ld + c, z[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(z[j][e], z[j][e], sum);
            if (a.weight && c < a.d) {
                float w[8];
                load8_f32(a.weight, a.w_dt, c, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) z[j][e] *= w[e];
            }
        }
        const bool row_scale = a.y_scale && a.group == 0;
        if (row_scale) {
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(z[j][e]));
            mx = warp_max(mx);
        }
        sum = warp_sum(sum);
        // the two halves of the shared words take turns, so one barrier a row is enough
        if (lane == 0) {
            s_sum[phase][warp] = sum;
            s_max[phase][warp] = mx;
        }
        __syncthreads();
        sum = warp_sum(lane < nw ? s_sum[phase][lane] : 0.0f);
        const float rstd = 1.0f / sqrtf(sum / (float)a.d + a.eps);
        // E4M3: with m = max |z w|, the scale is m rstd / 448 and a code z w rstd / scale =
        // z w (448 / m): within 3 ulp of the division, which moves a code only next to a tie
        float up = 0.0f;
        auto scale_of = [&](float m, float* out, bool mine) {
            const float amax = m * rstd;
            up = amax > 0.0f ? __fdividef(448.0f, m) : rstd;
            if (mine) *out = amax > 0.0f ? amax / 448.0f : 1.0f;
        };
        if (row_scale) {
            mx = warp_max(lane < nw ? s_max[phase][lane] : 0.0f);
            scale_of(mx, a.y_scale + t, tid == 0);
        }
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (j * nt + tid) * 8;
            if (a.group) {
                // the 16 lanes of 128 columns (all of them inside the row or none)
                float m = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(z[j][e]));
                __syncwarp();
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                scale_of(m, a.y_scale + t * (a.d / 128) + c / 128, c < a.d && lane % 16 == 0);
            }
            if (c >= a.d) continue;
            const float f = a.y_scale ? up : rstd;
#pragma unroll
            for (int e = 0; e < 8; ++e) z[j][e] *= f;
            if (a.y_scale)
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + t * a.y_ld + c) =
                    make_uint2(pack_e4m3x4(z[j][0], z[j][1], z[j][2], z[j][3]),
                               pack_e4m3x4(z[j][4], z[j][5], z[j][6], z[j][7]));
            else
                store8(a.y, a.y_dt, t * a.y_ld + c, z[j]);
        }
        phase ^= 1;
    }
}

template <int CH, bool WALK>
cudaError_t launch(const NormArgs& a, int threads, cudaStream_t s) {
    const bool x = a.x_dt == MOE_DTYPE_BF16, r = a.r_dt == MOE_DTYPE_BF16;
    auto kern = x ? (r ? rmsnorm_kernel<CH, true, true, WALK> : rmsnorm_kernel<CH, true, false, WALK>)
                  : (r ? rmsnorm_kernel<CH, false, true, WALK> : rmsnorm_kernel<CH, false, false, WALK>);
    int grid = a.T;
    size_t smem = 0;
    if (WALK) {
        smem = (size_t)kDepth * CH * threads * ((x ? 16 : 32) + (a.residual ? r ? 16 : 32 : 0));
        static std::atomic<uint64_t> done[4];
        cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), 224 * 1024, done[2 * x + r]);
        int per_sm = 0;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
        if (e != cudaSuccess) return e;
        grid = std::min(grid, std::max(1, per_sm) * device_sm_count());
    }
    return launch_pdl(kern, dim3((unsigned)grid), dim3((unsigned)threads), smem, s, a);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t s) {
    const int chunks = a.d / 8;
    auto threads = [&](int ch) { return ((chunks + ch - 1) / ch + 31) / 32 * 32; };
    // More rows than SMs: blocks that walk over the rows.
    if (a.T > device_sm_count() && chunks <= 4 * kWalkThreads) {
        if (chunks <= kWalkThreads) return launch<1, true>(a, threads(1), s);
        if (chunks <= 2 * kWalkThreads) return launch<2, true>(a, threads(2), s);
        return launch<4, true>(a, threads(4), s);
    }
    if (chunks <= 1024) return launch<1, false>(a, threads(1), s);
    if (chunks <= 2048) return launch<2, false>(a, threads(2), s);
    return launch<4, false>(a, threads(4), s);
}

}  // namespace moe
