// Shared projection with low-rank adapters for one or two tokens, on the CUDA cores:
//   y[t] = W x[t] + s_a B_a (A_a x[t]).
//
// W is read once; with so few tokens the products are a few fp32 multiply-adds per
// weight, and HBM (or, for a small W, latency) bounds the call.  Every thread owns 8
// columns of d; the block takes 4 rows of W at a time with the next 4 in flight and sums
// them over its threads; a warp per token of its own joins the sums with the adapter's
// part and writes the 4 outputs (with its registers in the same threads the loop spilled:
// 31 instead of 22 us for one token of 7168 -> 9216).  The first rows of W are
// fetched before the kernel ahead has ended, and where A_a is small (below) every
// block forms v = A_a x itself, so that the call is one launch.
#include <algorithm>

#include "block.h"

namespace moe {

namespace {

constexpr int kGemvRows = 4;
constexpr int kGemvMaxHidden = 7168;        // 896 threads and the writers: 64 registers each

template <bool F8>
struct WRaw {
    uint4 w;
    __device__ __forceinline__ void load(const void* p, long long i) {
        if constexpr (F8) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + i));
            w.x = v.x;
            w.y = v.y;
        } else {
            w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i));
        }
    }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
        if constexpr (F8) {
            f[0] = unpack_e4m3x2<false>(w.x);
            f[1] = unpack_e4m3x2<true>(w.x);
            f[2] = unpack_e4m3x2<false>(w.y);
            f[3] = unpack_e4m3x2<true>(w.y);
        } else {
            unpack_bf16x8_f2(w, f);
        }
    }
};

// TT: tokens.  own_v: the block forms v itself; otherwise a.v has it.
template <int TT, bool F8>
__global__ void __launch_bounds__(kGemvMaxHidden / 8 + 32 * TT) lora_gemv_kernel(const __grid_constant__ LoraArgs a, int own_v) {
    constexpr int V = kGemvRows * TT;
    extern __shared__ __align__(16) float4 xs[];             // [TT][2][chunks]: first and last halves of the chunks of x
    __shared__ float s_part[2][32][V];
    __shared__ int s_ad[TT];
    __shared__ float s_scale[TT];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nw = (blockDim.x >> 5) - TT;                   // warps on W; TT writers after them
    const int chunks = a.d / 8, batches = a.N / kGemvRows;
    float* vs = reinterpret_cast<float*>(xs + TT * 2 * chunks);   // [TT][r]: v times the adapter's scale
    const bool active = tid < chunks;
    WRaw<F8> w[kGemvRows];
    auto fetch = [&](int b) {
        if (active) {
#pragma unroll
            for (int r = 0; r < kGemvRows; ++r) w[r].load(a.w, ((long long)b * kGemvRows + r) * a.w_ld + tid * 8);
        }
    };
    fetch(blockIdx.x);
    pdl_allow_dependents();
    pdl_wait_primary();

    for (int i = tid; i < TT * chunks; i += blockDim.x) {
        const int t = i / chunks, c = i - t * chunks;
        float f[8];
        load8_any(a.x, a.x_dt, t * a.x_ld + c * 8, f);
        xs[(t * 2) * chunks + c] = make_float4(f[0], f[1], f[2], f[3]);
        xs[(t * 2 + 1) * chunks + c] = make_float4(f[4], f[5], f[6], f[7]);
    }
    if (lane == 0 && warp >= nw) {
        const int t = warp - nw, ad = a.r > 0 ? adapter_of(a, t) : -1;
        s_ad[t] = ad;
        s_scale[t] = ad >= 0 ? a.ls[ad] * (F8 && own_v ? a.x_scale[t] : 1.0f) : 0.0f;
    }
    __syncthreads();
    if (own_v) {
        // a warp takes two rows of A_a (of one token: r is even)
        for (int i = warp * 2; i < TT * a.r; i += (nw + TT) * 2) {
            const int t = i / a.r, j = i - t * a.r, ad = s_ad[t];
            if (ad < 0) continue;
            const uint4* row = reinterpret_cast<const uint4*>(a.la + ((long long)ad * a.r + j) * a.d);
            float sum[2] = {};
#pragma unroll 4
            for (int c = lane; c < chunks; c += 32) {
                const uint4 r0 = __ldg(row + c), r1 = __ldg(row + chunks + c);
                const float4 x0 = xs[(t * 2) * chunks + c], x1 = xs[(t * 2 + 1) * chunks + c];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float u[8];
                    unpack_bf16x8(k ? r1 : r0, u);
                    sum[k] = fmaf(u[0], x0.x, fmaf(u[1], x0.y, fmaf(u[2], x0.z, fmaf(u[3], x0.w, sum[k]))));
                    sum[k] = fmaf(u[4], x1.x, fmaf(u[5], x1.y, fmaf(u[6], x1.z, fmaf(u[7], x1.w, sum[k]))));
                }
            }
            const float s0 = warp_sum(sum[0]), s1 = warp_sum(sum[1]);
            if (lane < 2) vs[i + lane] = (lane ? s1 : s0) * s_scale[t];
        }
    } else {
        for (int i = tid; i < TT * a.r; i += blockDim.x)
            if (s_ad[i / a.r] >= 0) vs[i] = a.v[i] * s_scale[i / a.r];
    }
    __syncthreads();

    // the halves of s_part take turns, so one barrier a batch is enough
    int phase = 0;
    if (warp < nw) {
        for (int b = blockIdx.x; b < batches; b += gridDim.x, phase ^= 1) {
            float2 sum[kGemvRows][TT];
#pragma unroll
            for (int r = 0; r < kGemvRows; ++r)
#pragma unroll
                for (int t = 0; t < TT; ++t) sum[r][t] = make_float2(0.0f, 0.0f);
            if (active) {
                float2 f[kGemvRows][4];
#pragma unroll
                for (int r = 0; r < kGemvRows; ++r) w[r].get(f[r]);
                if (b + (int)gridDim.x < batches) fetch(b + gridDim.x);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const float4 x0 = xs[(t * 2) * chunks + tid], x1 = xs[(t * 2 + 1) * chunks + tid];
#pragma unroll
                    for (int r = 0; r < kGemvRows; ++r) {
                        float2 s = ffma2(f[r][0], make_float2(x0.x, x0.y), sum[r][t]);
                        s = ffma2(f[r][1], make_float2(x0.z, x0.w), s);
                        s = ffma2(f[r][2], make_float2(x1.x, x1.y), s);
                        sum[r][t] = ffma2(f[r][3], make_float2(x1.z, x1.w), s);
                    }
                }
            }
            float acc[V];
#pragma unroll
            for (int r = 0; r < kGemvRows; ++r)
#pragma unroll
                for (int t = 0; t < TT; ++t) acc[t * kGemvRows + r] = sum[r][t].x + sum[r][t].y;
            int vi;
            const float part = warp_reduce_spread<V>(acc, lane, vi);
            if ((lane & (32 / V - 1)) == 0) s_part[phase][warp][vi] = part;
            __syncthreads();
        }
        return;
    }
    // writer of token t: 8 lanes per row of the batch; the row of B_a in 16-byte chunks l and
    // l + 8, a batch ahead like W
    const int t = warp - nw, l = lane % 8, orow = lane / 8, ad = s_ad[t];
    const float4* v = reinterpret_cast<const float4*>(vs + t * a.r);
    uint4 lb[2] = {};
    auto fetch_b = [&](int b) {
        if (ad >= 0) {
            const uint4* row = reinterpret_cast<const uint4*>(a.lb + ((long long)ad * a.N + b * kGemvRows + orow) * a.r);
            if (l < a.r / 8) lb[0] = __ldg(row + l);
            if (l + 8 < a.r / 8) lb[1] = __ldg(row + l + 8);
        }
    };
    fetch_b(blockIdx.x);
    for (int b = blockIdx.x; b < batches; b += gridDim.x, phase ^= 1) {
        const int n = b * kGemvRows + orow;
        float low = 0.0f;
        if (ad >= 0) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = l + 8 * k;
                if (c < a.r / 8) {
                    float u[8];
                    unpack_bf16x8(lb[k], u);
                    const float4 v0 = v[2 * c], v1 = v[2 * c + 1];
                    low = fmaf(u[0], v0.x, fmaf(u[1], v0.y, fmaf(u[2], v0.z, fmaf(u[3], v0.w, low))));
                    low = fmaf(u[4], v1.x, fmaf(u[5], v1.y, fmaf(u[6], v1.z, fmaf(u[7], v1.w, low))));
                }
            }
            if (b + (int)gridDim.x < batches) fetch_b(b + gridDim.x);
        }
        __syncthreads();
        float s = 0.0f;
        for (int k = l; k < nw; k += 8) s += s_part[phase][k][t * kGemvRows + orow];
        if (F8) s *= a.x_scale[t] * a.w_scale[n];
        s += low;
        __syncwarp();
#pragma unroll
        for (int m = 4; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
        if (l == 0) {
            const long long i = t * a.y_ld + n;
            if (a.y_dt == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.y)[i] = __float2bfloat16_rn(s);
            else static_cast<float*>(a.y)[i] = s;
        }
    }
}

template <int TT, bool F8>
cudaError_t launch(const LoraArgs& a, bool own_v, cudaStream_t s) {
    auto kern = lora_gemv_kernel<TT, F8>;
    static std::atomic<uint64_t> done;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), 200 * 1024, done);
    if (e != cudaSuccess) return e;
    const int threads = (a.d / 8 + 31) / 32 * 32 + 32 * TT;
    const size_t smem = (size_t)TT * (a.d + a.r) * sizeof(float);
    // blocks that run at once: 64 registers a thread, 228 KB of shared memory an SM
    const int per_sm = std::max(1, std::min(1024 / threads, (int)(220 * 1024 / (smem + 6 * 1024))));
    const int grid = std::min(a.N / kGemvRows, per_sm * device_sm_count());
    return launch_pdl(kern, dim3((unsigned)grid), dim3((unsigned)threads), smem, s, a, (int)own_v);
}

}  // namespace

// Against the tensor-core kernel (us, that one second; without adapters): one token of 2048 -> 2560
// bf16 3.1 / 5.6, of 7168 -> 9216 21.1 / 22.7; two tokens 4.1 / 5.6 and 28.9 / 22.7, of 4096 -> 4096
// (34 MB) 10.5 / 9.6: there the shared memory reads of x bound it, so two tokens only over up to 20 MB
// of W, or in fp32 (7168 -> 9216 29.0 / 31.1), whose three terms the other one multiplies.
bool lora_gemv_fits(const LoraArgs& a) {
    const long long bytes = (long long)a.N * a.d * (a.x_dt == MOE_DTYPE_FP8_E4M3 ? 1 : 2);
    return a.d <= kGemvMaxHidden && (a.T == 1 || (a.T == 2 && (a.x_dt == MOE_DTYPE_F32 || bytes <= 20ll << 20)));
}

// A_a x in every block: while a block reads no more than 128 KB for it (from L2, at about 64
// bytes a clock: 1 us), which is less than another launch takes.
bool lora_gemv_own_v(const LoraArgs& a) { return (long long)a.T * a.r * a.d * 2 <= 128 * 1024; }

cudaError_t launch_lora_gemv(const LoraArgs& a, cudaStream_t s) {
    const bool f8 = a.x_dt == MOE_DTYPE_FP8_E4M3, own = lora_gemv_own_v(a);
    if (a.T == 1) return f8 ? launch<1, true>(a, own, s) : launch<1, false>(a, own, s);
    return f8 ? launch<2, true>(a, own, s) : launch<2, false>(a, own, s);
}

}  // namespace moe
