// Shared projection with low-rank adapters: y[t] = W x[t] + s_a B_a (A_a x[t]).
//
// W is read once for all T <= 128 tokens (2 T flops per byte of bf16, far below what
// the tensor cores need to be busy), so the rows of W are the 128 rows of the MMA
// and the tokens its columns: the W tiles go from HBM through a TMA ring straight
// into tcgen05.mma as its A operand, whatever T is.
//
// Split.  A tile of 128 rows of W is one CTA, or a cluster of 2, 4 or 8 of them that
// divide d where the tiles are fewer than the SMs; the cluster adds its parts up over
// distributed shared memory in a fixed order, each CTA for its share of the tokens.
//
// Sums.  The tensor cores cut their running sums to 24 bits instead of rounding, so
// they run over at most 16 MMAs (512 bytes of a row); the epilogue warps add each such
// block to fp32 registers (rounded) while the next one runs in the other half of the
// accumulators.  fp32 activations are three bf16 terms (24 bits); the two small ones
// have accumulators of their own.
//
// Adapters.  v[t] = A_a x[t] is taken by a small kernel before this one (which
// overlaps it: W is fetched meanwhile).  The tokens are sorted by adapter; the 128
// rows of B_a, which lie next to one another, come as one bulk copy for all tokens of
// the adapter, and four warps multiply them with v in fp32 beside the MMAs.  A token
// meets no weights but its own adapter's, whatever the others hold.
#include <algorithm>

#include "block.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr int kRowsM = 128;                 // rows of W per tile
constexpr int kBlockBytes = 128;            // bytes of a row per stage (one swizzle row)
constexpr int kWBytes = kRowsM * kBlockBytes;
constexpr int kChunkBlocks = 4;             // stages per accumulator block
constexpr int kMaxStages = 12;
constexpr int kLoraStages = 8;              // at most
constexpr int kLoraTokens = 4;              // tokens of an adapter taken together
constexpr int kProjThreads = 384;           // 12 warps: TMA, MMA, adapter copies, idle, 4 adapter, 4 epilogue
constexpr int kProjSmem = 226 * 1024;

// ---- v = A_a x, and the bf16 terms of fp32 activations -----------------------

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

// -1 for a token without an adapter; an index beyond the adapters is reported and counts as none.
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int t) {
    const int i = a.adapter[t];
    if (i >= a.na) set_status(a.status, MOE_ERR_DEVICE);
    return i >= 0 && i < a.na ? i : -1;
}

constexpr int kShrinkThreads = 256;

// Blocks [0, T r / ROWS): ROWS rows of A_a against x[t], d shared out over the block's
// threads.  The blocks after them write the terms of x.
template <int ROWS>
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_kernel(const __grid_constant__ LoraArgs a) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_allow_dependents();
    pdl_wait_primary();
    const int groups = a.r / ROWS, shrink_blocks = a.T * groups;
    if ((int)blockIdx.x >= shrink_blocks) {
        const int chunks = a.d / 8;
        const long long plane = (long long)a.T * a.d;
        for (int i = (blockIdx.x - shrink_blocks) * kShrinkThreads + tid; i < a.T * chunks;
             i += (gridDim.x - shrink_blocks) * kShrinkThreads) {
            const int t = i / chunks, c = (i - t * chunks) * 8;
            float f[8];
            load8_f32(a.x, MOE_DTYPE_F32, t * a.x_ld + c, f);
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float b = __uint_as_float(h ? w[e] & 0xffff0000u : w[e] << 16);
                        // an infinite or NaN first term stands alone
                        f[2 * e + h] = fabsf(b) <= 3.4028234e38f ? f[2 * e + h] - b : 0.0f;
                    }
                }
                *reinterpret_cast<uint4*>(a.xs + p * plane + (long long)t * a.d + c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        return;
    }
    __shared__ float s_part[kShrinkThreads / 32][ROWS];
    const int t = blockIdx.x / groups, j0 = (blockIdx.x - t * groups) * ROWS;
    const int ad = adapter_of(a, t);
    float sum[ROWS] = {};
    if (ad >= 0) {
        const __nv_bfloat16* rows = a.la + ((long long)ad * a.r + j0) * a.d;
#pragma unroll (ROWS == 2 ? 4 : 2)
        for (int c = tid * 8; c < a.d; c += kShrinkThreads * 8) {
            float x[8];
            load8_any(a.x, a.x_dt, t * a.x_ld + c, x);
            uint4 w[ROWS];
#pragma unroll
            for (int j = 0; j < ROWS; ++j) w[j] = __ldg(reinterpret_cast<const uint4*>(rows + (long long)j * a.d + c));
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                float u[8];
                unpack_bf16x8(w[j], u);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[j] = fmaf(u[e], x[e], sum[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        const float s = warp_sum(sum[j]);
        if (lane == 0) s_part[warp][j] = s;
    }
    __syncthreads();
    if (tid < ROWS) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kShrinkThreads / 32; ++w) s += s_part[w][tid];
        a.v[t * a.r + j0 + tid] = a.x_scale ? s * a.x_scale[t] : s;
    }
}

// ---- projection --------------------------------------------------------------

struct ProjArgs {
    LoraArgs l;
    CUtensorMap wmap, xmap;     // W [N, d]; x [T, d], or its terms [3, T, d]
    int blocks;                 // 128-byte blocks of a row
    int split;                  // CTAs of a cluster
    int stages, lora_stages;
    int lacc_off, v_off, lring_off, wring_off;   // byte offsets in shared memory
};

// 3-D tile load without a cache hint: what many CTAs read.
__device__ __forceinline__ void tma_load_3d_plain(void* dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(dst)),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes of CTA `rank`'s shared memory at this CTA's address p.
__device__ __forceinline__ float4 ld_cluster4(const void* p, uint32_t rank) {
    uint32_t addr;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

struct ProjShared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t lfull[kLoraStages], lempty[kLoraStages];
    uint64_t mma_done;
    uint32_t tmem;
    int key[kLoraMaxT];        // adapter of each token
    int order[kLoraMaxT];      // tokens by adapter (those without first), then by index
};

// out[k][128] = the thread's row of B_a times v[k], for TOK tokens.  The lanes start at different
// 16-byte chunks of their rows (distinct banks); four pairs of sums per token keep the
// multiply-adds independent.
template <int TOK>
__device__ __forceinline__ void lora_rows(const uint4* row, const float* v, int r, int C, int m, float* out) {
    float2 acc[TOK][4];
#pragma unroll
    for (int k = 0; k < TOK; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[k][e] = make_float2(0.0f, 0.0f);
    int c = m % C;
#pragma unroll 4
    for (int j = 0; j < C; ++j) {
        float2 b[4];
        unpack_bf16x8_f2(row[c], b);
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            const float4* u = reinterpret_cast<const float4*>(v + k * r + c * 8);
            const float4 x = u[0], y = u[1];
            acc[k][0] = ffma2(b[0], make_float2(x.x, x.y), acc[k][0]);
            acc[k][1] = ffma2(b[1], make_float2(x.z, x.w), acc[k][1]);
            acc[k][2] = ffma2(b[2], make_float2(y.x, y.y), acc[k][2]);
            acc[k][3] = ffma2(b[3], make_float2(y.z, y.w), acc[k][3]);
        }
        c = c + 1 == C ? 0 : c + 1;
    }
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        const float2 s = make_float2((acc[k][0].x + acc[k][1].x) + (acc[k][2].x + acc[k][3].x),
                                     (acc[k][0].y + acc[k][1].y) + (acc[k][2].y + acc[k][3].y));
        out[k * kRowsM] = s.x + s.y;
    }
}

// TP: tokens rounded up to 16, 32, 64 or 128 (MMA columns).  F8: E4M3.  TERMS: bf16
// terms of x (1, or 3 for fp32).
template <int TP, bool F8, int TERMS>
__global__ void __launch_bounds__(kProjThreads, 1) lora_project_kernel(const __grid_constant__ ProjArgs p) {
    constexpr int kAccs = TERMS > 1 ? 2 : 1;                  // the first term's sum, and the others'
    constexpr uint32_t kBufCols = kAccs * TP;
    constexpr uint32_t kTmemCols = 2 * kBufCols;              // 32 to 512, a power of two
    constexpr int kXBytes = TP * kBlockBytes;                 // one term
    constexpr int kStageBytes = kWBytes + TERMS * kXBytes;
    const LoraArgs& a = p.l;
    extern __shared__ unsigned char smem_dyn[];
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    ProjShared& sm = *reinterpret_cast<ProjShared*>(base);
    float* lacc = reinterpret_cast<float*>(base + p.lacc_off);       // [own tokens][128] adapter part
    float* vs = reinterpret_cast<float*>(base + p.v_off);            // [own tokens][r] v, times the adapter's scale
    unsigned char* lring = base + p.lring_off;
    unsigned char* ring = base + p.wring_off;
    float* red = reinterpret_cast<float*>(ring);                     // after the stream: [T][128] this CTA's sums

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = p.split > 1 ? (int)cluster_rank() : 0;
    const int n0 = (int)(blockIdx.x / p.split) * kRowsM;
    const int kb0 = p.blocks * rank / p.split, kb1 = p.blocks * (rank + 1) / p.split;
    const int nkb = kb1 - kb0, chunks = (nkb + kChunkBlocks - 1) / kChunkBlocks;
    // positions of the sorted tokens that this CTA adds up and writes
    const int p0 = a.T * rank / p.split, p1 = a.T * (rank + 1) / p.split;

    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.acc_full[i], 1);
            mbar_init(&sm.acc_empty[i], 4);
        }
        for (int i = 0; i < kLoraStages; ++i) {
            mbar_init(&sm.lfull[i], 1);
            mbar_init(&sm.lempty[i], 4);
        }
        mbar_init(&sm.mma_done, 1);
        mbar_init_fence();
        tma_prefetch_map(&p.wmap);
        tma_prefetch_map(&p.xmap);
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sm.tmem;
    pdl_allow_dependents();

    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (ok && !mbar_wait_bounded(bar, parity)) {
            ok = false;
            set_status(a.status, kDevErrTimeout);
        }
        return ok;
    };

    // ---- TMA producer, first part: W of the first stages, before x is there
    const uint64_t pol = l2_policy_evict_first();
    constexpr int kColsPerBlock = F8 ? 128 : 64;
    auto load_w = [&](int i) {
        const int slot = i % p.stages;
        mbar_arrive_expect_tx(&sm.full[slot], kStageBytes);
        tma_load_2d(ring + slot * kStageBytes, &p.wmap, (kb0 + i) * kColsPerBlock, n0, &sm.full[slot], pol);
    };
    const int early = min(nkb, p.stages);
    if (warp == 0 && lane == 0)
        for (int i = 0; i < early; ++i) load_w(i);

    pdl_wait_primary();

    // ---- order of the tokens
    if (a.r > 0) {
        for (int t = tid; t < a.T; t += kProjThreads) sm.key[t] = adapter_of(a, t);
        __syncthreads();
        for (int t = tid; t < a.T; t += kProjThreads) {
            const int k = sm.key[t];
            int pos = 0;
            for (int u = 0; u < a.T; ++u) pos += sm.key[u] < k || (sm.key[u] == k && u < t);
            sm.order[pos] = t;
        }
        __syncthreads();
        for (int i = tid; i < (p1 - p0) * (a.r / 4); i += kProjThreads) {
            const int q = i / (a.r / 4), j = i - q * (a.r / 4), t = sm.order[p0 + q], ad = sm.key[t];
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (ad >= 0) {
                const float f = a.ls[ad];
                v = *reinterpret_cast<const float4*>(a.v + t * a.r + j * 4);
                v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
            }
            reinterpret_cast<float4*>(vs)[i] = v;
        }
    } else {
        for (int t = tid; t < a.T; t += kProjThreads) sm.order[t] = t;
    }
    __syncthreads();

    if (warp == 0) {
        // ===================== TMA producer =====================
        if (lane == 0) {
            auto load_x = [&](int i) {
                const int slot = i % p.stages;
                unsigned char* dst = ring + slot * kStageBytes + kWBytes;
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
                    tma_load_3d_plain(dst + t * kXBytes, &p.xmap, (kb0 + i) * kColsPerBlock, 0, t, &sm.full[slot]);
            };
            for (int i = 0; i < early; ++i) load_x(i);
            int i = early;
            for (; i < nkb; ++i) {
                if (!wait(&sm.empty[i % p.stages], ((i / p.stages) & 1u) ^ 1u)) break;
                load_w(i);
                load_x(i);
            }
            // every copy has landed before the CTA may exit
            for (int j = max(0, i - p.stages); j < i; ++j) mbar_wait_bounded(&sm.full[j % p.stages], (j / p.stages) & 1u);
        }
    } else if (warp == 1) {
        // ===================== MMA issuer =====================
        if (lane == 0) {
            const uint64_t a0 = smem_desc_sw128(smem_u32(ring), 16, 1024);
            const uint64_t b0 = smem_desc_sw128(smem_u32(ring + kWBytes), 16, 1024);
            const uint32_t idesc = F8 ? idesc_e4m3_f32(128, TP) : idesc_bf16_f32(128, TP, false, false);
            for (int c = 0; ok && c < chunks; ++c) {
                const uint32_t buf = c & 1;
                if (!wait(&sm.acc_empty[buf], ((c >> 1) & 1u) ^ 1u)) break;
                tc_fence_after_sync();
                const int end = min(nkb, (c + 1) * kChunkBlocks);
                for (int i = c * kChunkBlocks; i < end; ++i) {
                    const int slot = i % p.stages;
                    if (!wait(&sm.full[slot], (i / p.stages) & 1u)) break;
                    tc_fence_after_sync();
                    const uint64_t ad = a0 + ((slot * kStageBytes) >> 4), bd = b0 + ((slot * kStageBytes) >> 4);
                    const bool fresh = i == c * kChunkBlocks;
#pragma unroll
                    for (int t = 0; t < TERMS; ++t)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            const uint32_t col = tmem + buf * kBufCols + (t > 0 ? TP : 0);
                            const uint32_t acc = fresh && ks == 0 && t <= 1 ? 0u : 1u;
                            if constexpr (F8) umma_e4m3(col, ad + ks * 2, bd + ks * 2, idesc, acc);
                            else umma_bf16(col, ad + ks * 2, bd + ((t * kXBytes) >> 4) + ks * 2, idesc, acc);
                        }
                    umma_commit(&sm.empty[slot]);
                }
                if (!ok) break;
                umma_commit(&sm.acc_full[buf]);
            }
            umma_commit(&sm.mma_done);
            mbar_wait_bounded(&sm.mma_done, 0);   // all MMAs have ended before TMEM is freed
        }
    } else if (warp == 2) {
        // ===================== adapter copies =====================
        if (lane == 0 && a.r > 0) {
            const uint32_t bytes = (uint32_t)min(kRowsM, a.N - n0) * a.r * 2;
            const int lstage = kRowsM * a.r * 2;
            int it = 0, last = -1;
            for (int q = p0; q < p1; ++q) {
                const int ad = sm.key[sm.order[q]];
                if (ad < 0 || ad == last) continue;
                last = ad;
                const int slot = it % p.lora_stages;
                if (!wait(&sm.lempty[slot], ((it / p.lora_stages) & 1u) ^ 1u)) break;
                mbar_arrive_expect_tx(&sm.lfull[slot], bytes);
                bulk_load(lring + slot * lstage, a.lb + ((long long)ad * a.N + n0) * a.r, bytes, &sm.lfull[slot], pol);
                ++it;
            }
            for (int j = max(0, it - p.lora_stages); j < it; ++j)
                mbar_wait_bounded(&sm.lfull[j % p.lora_stages], (j / p.lora_stages) & 1u);
        }
    } else if (warp >= 4 && warp < 8) {
        // ===================== adapters: s B_a v on the CUDA cores =====================
        if (a.r > 0) {
            const int m = (warp - 4) * 32 + lane, C = a.r / 8;
            const int lstage = kRowsM * a.r * 2;
            int it = 0;
            for (int q = p0; q < p1;) {
                const int ad = sm.key[sm.order[q]];
                if (ad < 0) {
                    lacc[(q - p0) * kRowsM + m] = 0.0f;
                    ++q;
                    continue;
                }
                const int slot = it % p.lora_stages;
                wait(&sm.lfull[slot], (it / p.lora_stages) & 1u);
                const uint4* row = reinterpret_cast<const uint4*>(lring + slot * lstage) + m * C;
                while (q < p1 && sm.key[sm.order[q]] == ad) {
                    int count = 1;
                    while (count < kLoraTokens && q + count < p1 && sm.key[sm.order[q + count]] == ad) ++count;
                    const float* v0 = vs + (q - p0) * a.r;
                    if (count == 1) lora_rows<1>(row, v0, a.r, C, m, lacc + (q - p0) * kRowsM + m);
                    else if (count == 2) lora_rows<2>(row, v0, a.r, C, m, lacc + (q - p0) * kRowsM + m);
                    else if (count == 3) lora_rows<3>(row, v0, a.r, C, m, lacc + (q - p0) * kRowsM + m);
                    else lora_rows<4>(row, v0, a.r, C, m, lacc + (q - p0) * kRowsM + m);
                    q += count;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.lempty[slot]);
                ++it;
            }
        }
    } else if (warp >= 8) {
        // ===================== epilogue: blocks of sums into registers =====================
        float acc[TP];
#pragma unroll
        for (int t = 0; t < TP; ++t) acc[t] = 0.0f;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        for (int c = 0; c < chunks; ++c) {
            const uint32_t buf = c & 1;
            if (!__all_sync(0xffffffffu, wait(&sm.acc_full[buf], (c >> 1) & 1u))) break;
            tc_fence_after_sync();
#pragma unroll
            for (int g = 0; g < kAccs; ++g)
#pragma unroll
                for (int t = 0; t < TP; t += 16) {
                    float v[16];
                    tmem_ld16(tmem + buf * kBufCols + g * TP + t + lanes, v);
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[t + e] += v[e];
                }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.acc_empty[buf]);
        }
        // the last block's MMAs have ended: nothing reads or writes the ring any more
        const int m = (warp & 3) * 32 + lane;
#pragma unroll
        for (int t = 0; t < TP; ++t)
            if (t < a.T) red[t * kRowsM + m] = acc[t];
    }
    tc_fence_before_sync();
    if (p.split > 1) cluster_sync_all();
    else __syncthreads();
    tc_fence_after_sync();

    // ---- the cluster's sum of this CTA's tokens, scales, adapter part, output
    const int warps = kProjThreads / 32, n = n0 + lane * 4;
    for (int q = p0 + warp; q < p1; q += warps) {
        const int t = sm.order[q];
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float* at = red + t * kRowsM + lane * 4;
        if (p.split > 1) {
#pragma unroll 8
            for (int k = 0; k < p.split; ++k) {
                const float4 v = ld_cluster4(at, (uint32_t)k);
                s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
            }
        } else {
            s = *reinterpret_cast<const float4*>(at);
        }
        if (n < a.N) {
            if constexpr (F8) {
                const float xs = a.x_scale[t];
                s.x *= xs * a.w_scale[n];
                s.y *= xs * a.w_scale[n + 1];
                s.z *= xs * a.w_scale[n + 2];
                s.w *= xs * a.w_scale[n + 3];
            }
            if (a.r > 0) {
                const float4 l = *reinterpret_cast<const float4*>(lacc + (q - p0) * kRowsM + lane * 4);
                s.x += l.x; s.y += l.y; s.z += l.z; s.w += l.w;
            }
            const long long i = t * a.y_ld + n;
            if (a.y_dt == MOE_DTYPE_BF16)
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + i) =
                    make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
            else
                *reinterpret_cast<float4*>(static_cast<float*>(a.y) + i) = s;
        }
    }
    // peers may still read this CTA's sums
    if (p.split > 1) cluster_sync_all();
    else __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// ---- host ----------------------------------------------------------------------

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static const EncodeTiledFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiledFn>(f) : nullptr;
    }();
    return fn;
}

// [planes, rows, d] row-major with row stride ld: boxes of 128 bytes x box_rows, 128 B swizzle.
// What lies beyond d or the rows reads as zero.
bool encode_rows(CUtensorMap* m, const void* ptr, int planes, int rows, int d, long long ld, int box_rows, bool f8) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t es = f8 ? 1 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * es, (cuuint64_t)rows * ld * es};
    const cuuint32_t box[3] = {f8 ? 128u : 64u, (cuuint32_t)box_rows, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return fn(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, planes > 0 ? 3 : 2,
              const_cast<void*>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int round_up(int v, int to) { return (v + to - 1) / to * to; }

template <int TP, bool F8, int TERMS>
cudaError_t launch_project(ProjArgs& p, cudaStream_t s) {
    const LoraArgs& a = p.l;
    constexpr int kStageBytes = kWBytes + TERMS * TP * kBlockBytes;
    auto kern = lora_project_kernel<TP, F8, TERMS>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kProjSmem);
    if (e != cudaSuccess) return e;
    const int tiles = (a.N + kRowsM - 1) / kRowsM, sms = device_sm_count();
    p.blocks = (a.d * (F8 ? 1 : 2) + kBlockBytes - 1) / kBlockBytes;
    // Split d while the clusters still run at once (a cluster of 8 does not fill a
    // GPC: about 7/8 of the SMs) and a CTA keeps two blocks or more.
    p.split = 1;
    for (int k = 2; k <= 8; k *= 2)
        if (tiles * k <= (k == 8 ? sms * 13 / 16 : sms) && p.blocks / k >= 2) p.split = k;
    // Shared memory: control words, adapter part of the own tokens, B_a ring, W ring (whose
    // place the CTA's sums take at the end).
    auto plan = [&] {
        int off = round_up((int)sizeof(ProjShared), 1024);
        p.lacc_off = off;
        if (a.r > 0) off = round_up(off + (a.T + p.split - 1) / p.split * kRowsM * 4, 1024);
        p.v_off = off;
        off = round_up(off + (a.T + p.split - 1) / p.split * a.r * 4, 1024);
        p.lring_off = off;
        const int lstage = kRowsM * a.r * 2;
        // 64 KB of B_a in flight, one tile at least, and three stages of W beside them where they fit
        p.lora_stages = a.r > 0 ? std::min({kLoraStages, 65536 / lstage, (a.T + p.split - 1) / p.split}) : 1;
        while (p.lora_stages > 1 && kProjSmem - 1024 - off - p.lora_stages * lstage < 3 * kStageBytes) --p.lora_stages;
        off = round_up(off + p.lora_stages * lstage, 1024);
        p.wring_off = off;
        p.stages = std::min(kMaxStages, (kProjSmem - 1024 - off) / kStageBytes);
    };
    plan();
    if (p.stages < 2 && p.split == 1 && p.blocks >= 2) {
        p.split = 2;     // half the own tokens: room for the ring
        plan();
    }
    p.stages = std::min(p.stages, (p.blocks + p.split - 1) / p.split);
    // At least half an SM's shared memory: two CTAs that shared an SM's TMEM could wait for each
    // other's through their clusters.
    const size_t smem = std::max((size_t)(1024 + p.wring_off + std::max(p.stages * kStageBytes, a.T * kRowsM * 4)),
                                 (size_t)116 * 1024);
    if (p.stages < 1 || smem > (size_t)kProjSmem) return cudaErrorInvalidConfiguration;
    const bool three = TERMS == 3;
    if (!encode_rows(&p.wmap, a.w, 0, a.N, a.d, a.w_ld, kRowsM, F8) ||
        !encode_rows(&p.xmap, three ? (const void*)a.xs : a.x, three ? 3 : 1, a.T, a.d, three ? a.d : a.x_ld, TP, F8))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.split));
    cfg.blockDim = dim3(kProjThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool F8, int TERMS>
cudaError_t launch_tp(ProjArgs& p, cudaStream_t s) {
    const int T = p.l.T;
    if (T <= 16) return launch_project<16, F8, TERMS>(p, s);
    if (T <= 32) return launch_project<32, F8, TERMS>(p, s);
    if (T <= 64) return launch_project<64, F8, TERMS>(p, s);
    return launch_project<128, F8, TERMS>(p, s);
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
    const bool f32 = a.x_dt == MOE_DTYPE_F32;
    if (a.r > 0 || f32) {
        const int split_blocks = f32 ? std::min(4 * device_sm_count(), (a.T * a.d / 8 + kShrinkThreads - 1) / kShrinkThreads) : 0;
        // few products: 2 rows of A per block, so that more SMs share the reading
        const bool few = a.T * a.r / 8 < 4 * device_sm_count();
        const int rows = few ? 2 : 8;
        const cudaError_t e = launch_pdl(few ? lora_shrink_kernel<2> : lora_shrink_kernel<8>,
                                         dim3((unsigned)(a.T * (a.r / rows) + split_blocks)), dim3(kShrinkThreads), 0, s, a);
        if (e != cudaSuccess) return e;
    }
    ProjArgs p = {};
    p.l = a;
    if (a.x_dt == MOE_DTYPE_FP8_E4M3) return launch_tp<true, 1>(p, s);
    return f32 ? launch_tp<false, 3>(p, s) : launch_tp<false, 1>(p, s);
}

}  // namespace moe
