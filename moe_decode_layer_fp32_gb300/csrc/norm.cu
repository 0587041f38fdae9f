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
// Measured, 8191 x 7168 bf16 + residual -> E4M3 by 128 columns (413 MB): 65.6 us, 6.3 TB/s.  It stands
// close to the issue rate too: with fp32 in pairs (two elements an instruction) 70 us where one by
// one took 78.  Two rows of each thread in flight instead of one 67 us; blocks of 256 threads (4
// chunks each) 73 us, of 896 (1 chunk) 70 us; one row per block without the copy ahead 125 us.  Rows
// of more than 16384 elements are taken that way (2048 x 16384 bf16 22 us, 88 % of the copy rate; x 16512 36 us,
// 56 %): a block that walks over them would need more registers or shared memory than two blocks have.
#include <algorithm>

#include "block.h"

namespace moe {

namespace {

constexpr int kWalkThreads = 512;    // most threads of a block that walks over rows
constexpr float kFewest = 0x1p-50f;  // 448 is divided directly by maxima from here to its reciprocal

template <bool BF>
__device__ __forceinline__ void raw8(const char* p, float2 (&f)[4]) {
    if constexpr (BF) {
        unpack_bf16x8_f2(*reinterpret_cast<const uint4*>(p), f);
    } else {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        f[0] = make_float2(a.x, a.y);
        f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y);
        f[3] = make_float2(b.z, b.w);
    }
}
__device__ __forceinline__ void put8(char* p, bool bf, const float2 (&f)[4]) {
    if (bf) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                                                  pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
    } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
}
template <int BYTES>
__device__ __forceinline__ void copy8(char* dst, const char* src) {
    cp_async16(dst, src);
    if constexpr (BYTES == 32) cp_async16(dst + 16, src + 16);
}
__device__ __forceinline__ float warp_max(float v) {
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float max8(const float2 (&f)[4]) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, fmaxf(fabsf(f[e].x), fabsf(f[e].y)));
    return m;
}
// amax / 448, rounded: the product with 1/448 and one step with its residual.
__device__ __forceinline__ float over_448(float amax) {
    const float q = amax * (1.0f / 448.0f);
    const float s = fmaf(fmaf(-448.0f, q, amax), 1.0f / 448.0f, q);
    return q < INFINITY ? s : q;
}

// CH: chunks of 8 elements a thread holds.  XBF, RBF: x, residual in bf16.  WALK: the block
// takes rows blockIdx.x, + gridDim.x, ..., and every thread copies its own chunks of the
// next row into places of its own in shared memory (which needs no barrier).
template <int CH, bool XBF, bool RBF, bool WALK>
__global__ void __launch_bounds__(WALK ? kWalkThreads : 1024, !WALK ? 1 : CH <= 2 ? 3 : 2) rmsnorm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int XB = XBF ? 16 : 32, RB = RBF ? 16 : 32;     // bytes of a chunk
    extern __shared__ __align__(16) char next[];
    __shared__ float s_sum[2][32], s_max[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5, nt = blockDim.x;
    const int chunks = a.d / 8, groups = a.d / 128;
    const float inv_d = 1.0f / (float)a.d;
    const bool wbf = a.w_dt == MOE_DTYPE_BF16, ybf = a.y_dt == MOE_DTYPE_BF16;
    pdl_allow_dependents();
    pdl_wait_primary();
    // chunk j of the next row: 16-byte words of a warp's lanes next to one another
    auto at = [&](int j) { return next + (j * nt + tid) * XB; };
    auto at_r = [&](int j) { return next + CH * nt * XB + (j * nt + tid) * RB; };
    auto x_row = [&](long long t) { return static_cast<const char*>(a.x) + t * a.x_ld * (XB / 8); };
    auto r_row = [&](long long t) { return static_cast<const char*>(a.residual) + t * a.r_ld * (RB / 8); };
    auto fetch = [&](long long t) {
        if (t < a.T) {
            const char *xr = x_row(t), *rr = r_row(t);
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int c = j * nt + tid;
                if (c < chunks) {
                    copy8<XB>(at(j), xr + c * XB);
                    if (a.residual) copy8<RB>(at_r(j), rr + c * RB);
                }
            }
        }
        cp_async_commit();
    };
    if constexpr (WALK) fetch(blockIdx.x);
    int phase = 0;
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
        float2 z[CH][4];
        float2 sum2 = make_float2(0.0f, 0.0f);
        if constexpr (WALK) cp_async_wait<0>();
        const char *xr = x_row(t), *rr = r_row(t);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = j * nt + tid;
            if (c < chunks) {
                raw8<XBF>(WALK ? at(j) : xr + c * XB, z[j]);
                if (a.residual) {
                    float2 u[4];
                    raw8<RBF>(WALK ? at_r(j) : rr + c * RB, u);
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[j][e] = fadd2(z[j][e], u[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) z[j][e] = make_float2(0.0f, 0.0f);
            }
        }
        char* out = static_cast<char*>(a.residual_out) + t * a.ro_ld * (RB / 8);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = j * nt + tid;
            if (a.residual_out && c < chunks) put8(out + c * RB, RBF, z[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum2 = ffma2(z[j][e], z[j][e], sum2);
            if (a.weight && c < chunks) {
                float2 w[4];
                if (wbf) raw8<true>(static_cast<const char*>(a.weight) + c * 16, w);
                else raw8<false>(static_cast<const char*>(a.weight) + c * 32, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) z[j][e] = fmul2(z[j][e], w[e]);
            }
        }
        const bool row_scale = a.y_scale && a.group == 0;
        // the two halves of the shared words take turns, so one barrier a row is enough
        if (row_scale) {
            float mx = 0.0f;
#pragma unroll
            for (int j = 0; j < CH; ++j) mx = fmaxf(mx, max8(z[j]));
            mx = warp_max(mx);
            if (lane == 0) s_max[phase][warp] = mx;
        }
        float sum = warp_sum(sum2.x + sum2.y);
        if (lane == 0) s_sum[phase][warp] = sum;
        // the sum holds all that the thread read of this row: the next one may take its place
        if constexpr (WALK) fetch(t + gridDim.x);
        __syncthreads();
        sum = warp_sum(lane < nw ? s_sum[phase][lane] : 0.0f);
        // 1 / sqrt(v): the fast one and a Newton step
        const float v = fmaf(sum, inv_d, a.eps), r0 = rsqrtf(v);
        const float rstd = r0 > 0.0f ? r0 * fmaf(-0.5f * v * r0, r0, 1.5f) : r0;
        // E4M3: with m = max |z w|, the scale is m rstd / 448 and a code z w rstd / scale =
        // z w (448 / m): within 3 ulp of the division, which moves a code only next to a tie.  Where
        // m is so far from 1 that 448 / m, or the few bits of a subnormal scale, might not do, z w is brought
        // near 1 by a power of two and divided by the scale as stored.  A scale that is 0 in fp32 becomes 1.
        float up = rstd, near_one = 1.0f;
        // m in [kFewest, 1 / kFewest) as one unsigned comparison of its bits; none where rstd is 0 or NaN
        const uint32_t plain = rstd >= kFewest * kFewest ? __float_as_uint(1.0f / kFewest) - __float_as_uint(kFewest) : 0u;
        auto scale_of = [&](float m, float* out, bool mine) {
            float s = over_448(m * rstd);
            up = rstd;
            near_one = 1.0f;
            if (__float_as_uint(m) - __float_as_uint(kFewest) < plain) {
                up = __fdividef(448.0f, m);
            } else if (s > 0.0f) {
                near_one = m > 1.0f ? 0x1p-100f : 0x1p100f;
                up = rstd / (s * near_one);
            } else {
                s = 1.0f;        // also beside a NaN
            }
            if (mine) *out = s;
        };
        if (row_scale) {
            const float mx = warp_max(lane < nw ? s_max[phase][lane] : 0.0f);
            scale_of(mx, a.y_scale + t, tid == 0);
        }
        char* y = static_cast<char*>(a.y) + t * a.y_ld * (a.y_scale ? 1 : ybf ? 2 : 4);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = j * nt + tid;
            if (a.group) {
                // the 16 lanes of 128 columns (all of them inside the row or none)
                float m = max8(z[j]);
                __syncwarp();
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                scale_of(m, a.y_scale + t * groups + c / 16, c < chunks && lane % 16 == 0);
            }
            if (c >= chunks) continue;
            if (near_one != 1.0f) {
#pragma unroll
                for (int e = 0; e < 4; ++e) z[j][e] = fmul2(z[j][e], make_float2(near_one, near_one));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) z[j][e] = fmul2(z[j][e], make_float2(up, up));
            if (a.y_scale)
                *reinterpret_cast<uint2*>(y + c * 8) = make_uint2(pack_e4m3x4(z[j][0].x, z[j][0].y, z[j][1].x, z[j][1].y),
                                                                  pack_e4m3x4(z[j][2].x, z[j][2].y, z[j][3].x, z[j][3].y));
            else
                put8(y + c * (ybf ? 16 : 32), ybf, z[j]);
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
        smem = (size_t)CH * threads * ((x ? 16 : 32) + (a.residual ? r ? 16 : 32 : 0));
        static std::atomic<uint64_t> done[4], blocks[4];
        cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), 224 * 1024, done[2 * x + r]);
        int per_sm = 0;
        if (e == cudaSuccess) e = blocks_per_sm(reinterpret_cast<const void*>(kern), threads, smem, blocks[2 * x + r], &per_sm);
        if (e != cudaSuccess) return e;
        grid = std::min(grid, per_sm * device_sm_count());
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
