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
// Adapters.  v[t] = A_a x[t] is taken before, while W is fetched already: by a small kernel, or
// for many rows by this one with the rows of A in the place of W.  The tokens are sorted by
// adapter; the 128 rows of B_a come once for all tokens of the adapter, and a warp
// multiplies them with v (three bf16 terms) beside the MMAs.  A token meets no
// weights but its own adapter's, whatever the others hold.
//
// Measured (without adapters): 16 to 32 tokens of 7168 -> 9216, bf16 (132 MB) 26.7 us, 128
// tokens 29 us; 128 tokens of 7168 -> 7168 E4M3 (51 MB) 18 us.  The stream of W alone takes
// 22 us of the first (6.65 TB/s): the four MMAs of a block, about 0.09 us each however few
// the tokens are, take a little longer than the block's bytes.  With 64 adapters of
// rank 64 (58 MB each of A and B) the third takes 59 us, 25 of them A x.
#include <algorithm>
#include <climits>

#include "block.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr int kRowsM = 128;                 // rows of W per tile
constexpr int kBlockBytes = 128;            // bytes of a row per stage (one swizzle row)
constexpr int kWBytes = kRowsM * kBlockBytes;
constexpr int kChunkBlocks = 4;             // stages per accumulator block
constexpr int kMaxStages = 12;
constexpr int kLoraStages = 16;             // at most
constexpr int kLoraBox = kRowsM * 128;       // 128 rows x 64 columns of B_a
constexpr int kProjThreads = 384;           // 12 warps: TMA, MMA, adapter copies, idle, 4 adapter, 4 epilogue
constexpr int kProjSmem = 226 * 1024;

// ---- v = A_a x, and the bf16 terms of fp32 activations -----------------------

constexpr int kShrinkThreads = 256;
// Tokens times rank from which A x goes to the tensor cores: at 512 (32 tokens, d 7168) the small kernel
// takes 7.5 us, at 8192 26 us against 25, which it does for shared adapters too.
constexpr int kShrinkTc = 1024;

// Blocks [0, T r / ROWS): ROWS rows of A_a against x[t], d shared out over the block's
// threads.  The blocks after them write the terms of x: three bf16 of fp32, one of E4M3
// (which bf16 holds exactly).
template <int ROWS>
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_kernel(const __grid_constant__ LoraArgs a, int shrink_blocks) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_allow_dependents();
    pdl_wait_primary();
    const int groups = a.r / ROWS;
    if ((int)blockIdx.x >= shrink_blocks) {
        const int chunks = a.d / 8;
        const long long plane = (long long)a.T * a.d;
        for (int i = (blockIdx.x - shrink_blocks) * kShrinkThreads + tid; i < a.T * chunks;
             i += (gridDim.x - shrink_blocks) * kShrinkThreads) {
            const int t = i / chunks, c = (i - t * chunks) * 8;
            float f[8];
            load8_any(a.x, a.x_dt, t * a.x_ld + c, f);
            const int terms = a.x_dt == MOE_DTYPE_F32 ? 3 : 1;
            for (int p = 0; p < terms; ++p) {
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
    CUtensorMap wmap, xmap;     // W [N, d] (shrink: A [na r, d], boxes of r rows); x [T, d], or its terms [3, T, d]
    CUtensorMap bmap;           // B [na N, r]
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
    alignas(16) int key[kLoraMaxT];   // adapter of each token (beyond the tokens: INT_MAX)
    int order[kLoraMaxT];      // tokens by adapter (those without first), then by index
    int skey[kLoraMaxT];       // their adapters in that order
    int index[kLoraMaxT];      // ... and the adapters' places among those in use (-1: none)
    int used[kLoraMaxT];       // the adapters in use
    int seg[kLoraMaxT + 1];    // projection: first sorted token of each adapter among the own tokens
    int segs;
    int starts[kLoraMaxT / 32];
    float scale[kLoraMaxT];    // adapters' scales, by sorted token
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// f as three bf16 terms (an infinite or NaN first term stands alone).
__device__ __forceinline__ void split3(float f, __nv_bfloat16 (&t)[3]) {
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        t[p] = __float2bfloat16_rn(f);
        const float b = __bfloat162float(t[p]);
        f = fabsf(b) <= 3.4028234e38f ? f - b : 0.0f;
    }
}

// Tiles of B_a (128 rows): ranks of whole k16 steps up to 48 come as one bulk copy of rows as they
// lie; the others as boxes of 64 columns in 128-byte rows, zeros beyond the rank, whose
// permuted chunks spare ldmatrix the bank conflicts.
__host__ __device__ inline bool lora_bulk(int r) { return r <= 48 && r % 16 == 0; }
__host__ __device__ inline int lora_stage_bytes(int r) {
    return lora_bulk(r) ? kRowsM * r * 2 : (r + 63) / 64 * kLoraBox;
}
// Stride of a token's v terms in shared memory: whole k16 steps, and 16 bytes more so that
// tokens fall on different banks.
__host__ __device__ inline int v_stride(int r) { return (r + 15) / 16 * 16 + 8; }

// TP: tokens rounded up to 16, 32, 64 or 128 (MMA columns).  F8: E4M3.  TERMS: bf16
// terms of x (1, or 3 for fp32).  SHRINK: the same stream over the rows of A in the place
// of W, as many whole adapters in use per tile as 128 rows hold; each token keeps the
// rows of its own, v[t] = A_a x[t].
template <int TP, bool F8, int TERMS, bool SHRINK>
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
    // [3][own tokens][v_stride]: bf16 terms of v times the adapter's scale
    __nv_bfloat16* vs = reinterpret_cast<__nv_bfloat16*>(base + p.v_off);
    unsigned char* lring = base + p.lring_off;
    unsigned char* ring = base + p.wring_off;
    float* red = reinterpret_cast<float*>(ring);                     // after the stream: [T][128] this CTA's sums

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = p.split > 1 ? (int)cluster_rank() : 0;
    const int tile = (int)(blockIdx.x / p.split), n0 = SHRINK ? 0 : tile * kRowsM;
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
            mbar_init(&sm.lempty[i], 1);
        }
        mbar_init(&sm.mma_done, 1);
        mbar_init_fence();
        tma_prefetch_map(&p.wmap);
        tma_prefetch_map(&p.xmap);
        if (!SHRINK && a.r > 0) tma_prefetch_map(&p.bmap);
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
    const int early = min(nkb, p.stages);
    // shrink: the tile's adapters are used[first_ad .. + ads)
    const int per_tile = SHRINK ? kRowsM / a.r : 0, first_ad = tile * per_tile;
    int ads = 0;
    auto load_w = [&](int i) {
        const int slot = i % p.stages;
        unsigned char* dst = ring + slot * kStageBytes;
        if constexpr (SHRINK) {
            mbar_arrive_expect_tx(&sm.full[slot], kStageBytes - kWBytes + ads * a.r * kBlockBytes);
            for (int k = 0; k < ads; ++k)
                tma_load_2d(dst + k * a.r * kBlockBytes, &p.wmap, (kb0 + i) * kColsPerBlock, sm.used[first_ad + k] * a.r,
                            &sm.full[slot], pol);
        } else {
            mbar_arrive_expect_tx(&sm.full[slot], kStageBytes);
            tma_load_2d(dst, &p.wmap, (kb0 + i) * kColsPerBlock, n0, &sm.full[slot], pol);
        }
    };
    if (!SHRINK && warp == 0 && lane == 0)
        for (int i = 0; i < early; ++i) load_w(i);

    pdl_wait_primary();

    // ---- order of the tokens: by the warps that need it first (the adapters' copies and
    // products; in the shrink form the W copies too, so all of them), the others go ahead
    const bool sorter = SHRINK || warp == 2 || (warp >= 4 && warp < 8);
    constexpr int kSorters = SHRINK ? kProjThreads : 160;
    const int sid = SHRINK ? tid : warp == 2 ? 128 + lane : tid - 128;
    auto sort_sync = [&] { named_bar_sync(1, kSorters); };
    if (a.r > 0 && sorter) {
        float scale = 0.0f;
        if (sid < kLoraMaxT) {
            const int k = sid < a.T ? adapter_of(a, sid) : INT_MAX;
            sm.key[sid] = k;
            if (!SHRINK && sid < a.T && k >= 0) scale = a.ls[k];
        }
        sort_sync();
        if (sid < a.T) {
            const int k = sm.key[sid];
            int pos = 0;
#pragma unroll 8
            for (int u = 0; u < kLoraMaxT; u += 4) {
                const int4 w = *reinterpret_cast<const int4*>(sm.key + u);
                pos += (w.x < k || (w.x == k && u < sid)) + (w.y < k || (w.y == k && u + 1 < sid)) +
                       (w.z < k || (w.z == k && u + 2 < sid)) + (w.w < k || (w.w == k && u + 3 < sid));
            }
            sm.order[pos] = sid;
            sm.skey[pos] = k;
            sm.scale[pos] = scale;
        }
        sort_sync();
        // A sorted token whose adapter differs from the one before starts an adapter in use: of all
        // tokens (shrink) or of the own ones.
        {
            const int q0 = SHRINK ? 0 : p0, q1 = SHRINK ? a.T : p1;
            const bool start = sid < a.T && sid >= q0 && sid < q1 && sm.skey[sid] >= 0 &&
                               (sid == q0 || sm.skey[sid - 1] != sm.skey[sid]);
            const uint32_t bits = __ballot_sync(0xffffffffu, start);
            if (sid < kLoraMaxT && lane == 0) sm.starts[sid / 32] = __popc(bits);
            sort_sync();
            int before = 0, count = 0;
#pragma unroll
            for (int w = 0; w < kLoraMaxT / 32; ++w) {
                if (w < sid / 32) before += sm.starts[w];
                count += sm.starts[w];
            }
            if (sid < a.T) {
                const int index = before + __popc(bits & (0xffffffffu >> (31 - lane))) - 1;
                if (SHRINK) sm.index[sid] = sm.skey[sid] >= 0 ? index : -1;
                if (start && SHRINK) sm.used[index] = sm.skey[sid];
                if (start && !SHRINK) sm.seg[index] = sid;
            }
            if (!SHRINK && sid == 0) {
                sm.segs = count;
                sm.seg[count] = p1;
            }
            sort_sync();
            if (SHRINK) ads = max(0, min(per_tile, count - first_ad));
        }
        if (!SHRINK && warp != 2) {
            const int vstr = v_stride(a.r), own = p1 - p0;
            // two elements of a token's v at a time, the loads of kAhead of them together
            constexpr int kAhead = 6;
            const int pairs = vstr / 2, n = own * pairs;
            for (int i0 = sid; i0 < n; i0 += kAhead * 128) {
                float2 v[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int i = i0 + u * 128, q = i / pairs, j = (i - q * pairs) * 2;
                    v[u] = make_float2(0.0f, 0.0f);
                    if (i < n && j < a.r && sm.skey[p0 + q] >= 0)
                        v[u] = *reinterpret_cast<const float2*>(a.v + sm.order[p0 + q] * a.r + j);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int i = i0 + u * 128, q = i / pairs, j = (i - q * pairs) * 2;
                    if (i >= n) break;
                    const float f = sm.scale[p0 + q];
                    __nv_bfloat16 t0[3], t1[3];
                    split3(v[u].x * f, t0);
                    split3(v[u].y * f, t1);
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        *reinterpret_cast<__nv_bfloat162*>(vs + (k * own + q) * vstr + j) = __halves2bfloat162(t0[k], t1[k]);
                }
            }
            named_bar_sync(2, 128);
        }
    } else if (a.r == 0) {
        for (int t = tid; t < a.T; t += kProjThreads) sm.order[t] = t;
    }
    if (SHRINK) __syncthreads();
    const bool idle = SHRINK && ads == 0;          // a tile beyond the adapters in use

    if (warp == 0) {
        // ===================== TMA producer =====================
        if (lane == 0 && !idle) {
            auto load_x = [&](int i) {
                const int slot = i % p.stages;
                unsigned char* dst = ring + slot * kStageBytes + kWBytes;
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
                    tma_load_3d_plain(dst + t * kXBytes, &p.xmap, (kb0 + i) * kColsPerBlock, 0, t, &sm.full[slot]);
            };
            for (int i = 0; i < early; ++i) {
                if (SHRINK) load_w(i);
                load_x(i);
            }
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
            for (int c = 0; ok && !idle && c < chunks; ++c) {
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
        if (!SHRINK && lane == 0 && a.r > 0) {
            const int boxes = (a.r + 63) / 64, lstage = lora_stage_bytes(a.r);
            const uint32_t bulk = (uint32_t)min(kRowsM, a.N - n0) * a.r * 2;
            int it = 0;
            for (; it < sm.segs; ++it) {
                const int ad = sm.skey[sm.seg[it]];
                const int slot = it % p.lora_stages;
                if (!wait(&sm.lempty[slot], ((it / p.lora_stages) & 1u) ^ 1u)) break;
                if (lora_bulk(a.r)) {
                    mbar_arrive_expect_tx(&sm.lfull[slot], bulk);
                    bulk_load(lring + slot * lstage, a.lb + ((long long)ad * a.N + n0) * a.r, bulk, &sm.lfull[slot], pol);
                } else {
                    mbar_arrive_expect_tx(&sm.lfull[slot], boxes * kLoraBox);
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(lring + slot * lstage + b * kLoraBox, &p.bmap, b * 64, ad * a.N + n0, &sm.lfull[slot], pol);
                }
            }
            for (int j = max(0, it - p.lora_stages); j < it; ++j)
                mbar_wait_bounded(&sm.lfull[j % p.lora_stages], (j / p.lora_stages) & 1u);
        }
    } else if (warp >= 4 && warp < 8) {
        // ===================== adapters: B_a v, an adapter per warp, up to 8 of its tokens at once =====================
        if (!SHRINK && a.r > 0) {
            const int steps = (a.r + 15) / 16, lstage = lora_stage_bytes(a.r);
            // rows of 128 bytes with permuted chunks, or of 2 r bytes as they are
            const int pitch = lora_bulk(a.r) ? a.r * 2 : 128, swizzle = lora_bulk(a.r) ? 0 : 7;
            const int vstr = v_stride(a.r), own = p1 - p0, segs = sm.segs;
            // ldmatrix: lane's row and 16-byte chunk within a 16 x 16 block
            const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lch = lane >> 4;
            for (int i = (warp - 4) * 32 + lane; i < (sm.seg[0] - p0) * kRowsM; i += 128) lacc[i] = 0.0f;
            for (int it = 0; it < segs; ++it) {
                // a slot belongs to one warp: a wait by parity holds only for a waiter that has seen
                // the slot's phase before
                const int slot = it % p.lora_stages, end = sm.seg[it + 1];
                if (slot % 4 != warp - 4) continue;
                wait(&sm.lfull[slot], (it / p.lora_stages) & 1u);
                __syncwarp();
                const uint32_t tile_b = smem_u32(lring + slot * lstage) + lrow * pitch;
                for (int q = sm.seg[it]; q < end; q += 8) {
                    const int count = min(8, end - q);
                    const __nv_bfloat16* v = vs + (q - p0 + lane / 4) * vstr + (lane & 3) * 2;
                    float* out = lacc + (q - p0 + (lane & 3) * 2) * kRowsM + lane / 4;
                    const bool t0 = (lane & 3) * 2 < count, t1 = (lane & 3) * 2 + 1 < count;
                    // up to 64 columns of B_a at a time: v's fragments stay in registers over the 128 rows
                    for (int k0 = 0; k0 < steps; k0 += 4) {
                        uint32_t b[4][3][2] = {};
                        if (lane / 4 < count) {
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                if (k0 + ks < steps) {
#pragma unroll
                                    for (int k = 0; k < 3; ++k) {
                                        b[ks][k][0] = *reinterpret_cast<const uint32_t*>(v + k * own * vstr + (k0 + ks) * 16);
                                        b[ks][k][1] = *reinterpret_cast<const uint32_t*>(v + k * own * vstr + (k0 + ks) * 16 + 8);
                                    }
                                }
                        }
#pragma unroll 2
                        for (int m = 0; m < kRowsM; m += 16) {
                            float c[3][4] = {};             // a sum per term: short chains of MMAs
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                if (k0 + ks < steps) {
                                    uint32_t f[4];
                                    ldmatrix_x4(tile_b + (k0 >> 2) * kLoraBox + m * pitch + (((ks * 2 + lch) ^ (lrow & swizzle)) << 4), f);
#pragma unroll
                                    for (int k = 0; k < 3; ++k) mma_bf16(c[k], f[0], f[1], f[2], f[3], b[ks][k][0], b[ks][k][1]);
                                }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float* at = out + (e & 1) * kRowsM + m + (e >> 1) * 8;
                                const float s = c[0][e] + (c[1][e] + c[2][e]);
                                if ((e & 1) ? t1 : t0) *at = k0 == 0 ? s : *at + s;
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.lempty[slot]);
            }
        }
    } else if (warp >= 8) {
        // ===================== epilogue: blocks of sums into registers =====================
        float acc[TP];
#pragma unroll
        for (int t = 0; t < TP; ++t) acc[t] = 0.0f;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        for (int c = 0; c < chunks && !idle; ++c) {
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
    const int warps = kProjThreads / 32;
    for (int q = p0 + warp; q < p1; q += warps) {
        const int t = sm.order[q];
        int col = lane * 4;                      // of the tile's 128 rows
        if constexpr (SHRINK) {
            const int k = sm.index[q] - first_ad;
            if (sm.index[q] < 0 || k < 0 || k >= ads || col >= a.r) continue;
            col += k * a.r;
        }
        const int n = n0 + col;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float* at = red + t * kRowsM + col;
        if (p.split > 1) {
#pragma unroll 8
            for (int k = 0; k < p.split; ++k) {
                const float4 v = ld_cluster4(at, (uint32_t)k);
                s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
            }
        } else {
            s = *reinterpret_cast<const float4*>(at);
        }
        if constexpr (SHRINK) {
            const float f = a.x_scale ? a.x_scale[t] : 1.0f;
            *reinterpret_cast<float4*>(a.v + t * a.r + lane * 4) = make_float4(s.x * f, s.y * f, s.z * f, s.w * f);
        } else if (n < a.N) {
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
bool encode_rows(CUtensorMap* m, const void* ptr, int planes, long long rows, int d, long long ld, int box_rows, bool f8) {
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

template <int TP, bool F8, int TERMS, bool SHRINK>
cudaError_t launch_project(ProjArgs& p, cudaStream_t s) {
    const LoraArgs& a = p.l;
    constexpr int kStageBytes = kWBytes + TERMS * TP * kBlockBytes;
    auto kern = lora_project_kernel<TP, F8, TERMS, SHRINK>;
    static std::atomic<uint64_t> done;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kProjSmem, done);
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count();
    // shrink: at most min(T, na) adapters are in use
    const int per_tile = SHRINK ? kRowsM / a.r : 1;
    const int tiles = SHRINK ? (std::min(a.T, a.na) + per_tile - 1) / per_tile : (a.N + kRowsM - 1) / kRowsM;
    const bool low = !SHRINK && a.r > 0;
    p.blocks = (a.d * (F8 ? 1 : 2) + kBlockBytes - 1) / kBlockBytes;
    // Split d while the clusters still run at once (a cluster of 8 does not fill a
    // GPC: about 7/8 of the SMs) and a CTA keeps two blocks or more.
    p.split = 1;
    for (int k = 2; k <= 8; k *= 2)
        if (tiles * k <= (k == 8 ? sms * 13 / 16 : sms) && p.blocks / k >= 2) p.split = k;
    // Shared memory: control words, adapter part of the own tokens, their v, B_a ring, W ring
    // (whose place the CTA's sums take at the end).
    const int lstage = low ? lora_stage_bytes(a.r) : 0;
    auto plan = [&] {
        const int own = (a.T + p.split - 1) / p.split;
        int off = round_up((int)sizeof(ProjShared), 1024);
        p.lacc_off = off;
        if (low) off = round_up(off + own * kRowsM * 4, 1024);
        p.v_off = off;
        if (low) off = round_up(off + 3 * own * v_stride(a.r) * 2, 1024);
        p.lring_off = off;
        // 64 KB of B_a in flight, one tile at least, and three stages of W beside them where they fit
        p.lora_stages = low ? std::min({kLoraStages, 65536 / lstage, own}) : 1;
        while (p.lora_stages > 1 && kProjSmem - 1024 - off - p.lora_stages * lstage < 3 * kStageBytes) --p.lora_stages;
        off = round_up(off + p.lora_stages * lstage, 1024);
        p.wring_off = off;
        p.stages = std::min(kMaxStages, (kProjSmem - 1024 - off) / kStageBytes);
    };
    plan();
    while (p.stages < 2 && p.split < 8) {
        p.split *= 2;     // fewer own tokens: room for the ring
        plan();
    }
    p.stages = std::min(p.stages, (p.blocks + p.split - 1) / p.split);
    // At least half an SM's shared memory: two CTAs that shared an SM's TMEM could wait for each
    // other's through their clusters.
    const size_t smem = std::max((size_t)(1024 + p.wring_off + std::max(p.stages * kStageBytes, a.T * kRowsM * 4)),
                                 (size_t)116 * 1024);
    if (p.stages < 1 || smem > (size_t)kProjSmem) return cudaErrorInvalidConfiguration;
    // fp32 x comes as its terms, and so does E4M3 x for the bf16 rows of A
    const bool terms = TERMS == 3 || (SHRINK && a.x_dt == MOE_DTYPE_FP8_E4M3);
    const bool maps =
        (SHRINK ? encode_rows(&p.wmap, a.la, 0, (long long)a.na * a.r, a.d, a.d, a.r, false)
                : encode_rows(&p.wmap, a.w, 0, a.N, a.d, a.w_ld, kRowsM, F8)) &&
        encode_rows(&p.xmap, terms ? (const void*)a.xs : a.x, TERMS, a.T, a.d, terms ? a.d : a.x_ld, TP, F8) &&
        (!low || encode_rows(&p.bmap, a.lb, 0, (long long)a.na * a.N, a.r, a.r, kRowsM, false));
    if (!maps) return cudaErrorInvalidValue;
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

template <bool F8, int TERMS, bool SHRINK>
cudaError_t launch_tp(const LoraArgs& a, cudaStream_t s) {
    ProjArgs p = {};
    p.l = a;
    if (a.T <= 16) return launch_project<16, F8, TERMS, SHRINK>(p, s);
    if (a.T <= 32) return launch_project<32, F8, TERMS, SHRINK>(p, s);
    if (a.T <= 64) return launch_project<64, F8, TERMS, SHRINK>(p, s);
    return launch_project<128, F8, TERMS, SHRINK>(p, s);
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
    const bool f32 = a.x_dt == MOE_DTYPE_F32, f8 = a.x_dt == MOE_DTYPE_FP8_E4M3;
    // v = A_a x: many rows on the tensor cores, which read each adapter once for all its
    // tokens; a few are done sooner by one small kernel, together with the terms of x.
    const bool gemv = lora_gemv_fits(a);
    if (gemv && (a.r == 0 || lora_gemv_own_v(a))) return launch_lora_gemv(a, s);
    const bool tc = !gemv && a.T * a.r >= kShrinkTc;
    const int split_blocks = (f32 && !gemv) || (f8 && tc)
                                 ? std::min(4 * device_sm_count(), (a.T * (a.d / 8) + kShrinkThreads - 1) / kShrinkThreads) : 0;
    const bool few = a.T * a.r / 8 < 4 * device_sm_count();    // 2 rows of A per block: more SMs share the reading
    const int shrink_blocks = tc ? 0 : a.T * (a.r / (few ? 2 : 8));
    cudaError_t e = cudaSuccess;
    if (shrink_blocks + split_blocks > 0)
        e = launch_pdl(few ? lora_shrink_kernel<2> : lora_shrink_kernel<8>, dim3((unsigned)(shrink_blocks + split_blocks)),
                       dim3(kShrinkThreads), 0, s, a, shrink_blocks);
    if (e == cudaSuccess && tc) e = f32 ? launch_tp<false, 3, true>(a, s) : launch_tp<false, 1, true>(a, s);
    if (e != cudaSuccess) return e;
    if (gemv) return launch_lora_gemv(a, s);
    if (f8) return launch_tp<true, 1, false>(a, s);
    return f32 ? launch_tp<false, 3, false>(a, s) : launch_tp<false, 1, false>(a, s);
}

}  // namespace moe
