// Shared projection with low-rank adapters: y[t] = W x[t] + s_a B_a (A_a x[t]).
//
// W is read once for all T <= 128 tokens (2 T flops per byte of bf16, far below what
// the tensor cores need to be busy), so the rows of W are the 128 rows of the MMA
// and the tokens its columns: the W tiles go from HBM through a TMA ring straight
// into tcgen05.mma as its A operand, whatever T is.
//
// Split.  A tile of 128 rows of W is one CTA, or a cluster of 2 to 8 of them that
// divide d where the tiles are fewer than the SMs; the cluster adds its parts up over
// distributed shared memory in a fixed order, each CTA for its share of the tokens.
//
// Sums.  The tensor cores cut their running sums to 24 bits instead of rounding, so
// they run over at most 16 MMAs (512 bytes of a row); the epilogue warps add each such
// block to fp32 registers (rounded) while the next one runs in the other half of the
// accumulators.  fp32 activations are three bf16 terms (24 bits); the two small ones
// have accumulators of their own.
//
// Adapters.  v[t] = A_a x[t] is taken before, by a kernel of its own that streams the rows of A
// and writes v times the adapter's scale as three bf16 terms; meanwhile this one sorts the
// tokens by adapter and fetches W and B.  128 rows of B_a come once for all tokens of the
// adapter, and four warps multiply 32 of them each with v beside the MMAs of W: all
// four on one tile, so that its place in the ring is free again sooner (an adapter to
// a warp took 337 us where this takes 160: 128 tokens, 128 adapters of rank 128).  A
// token meets no weights but its own adapter's, whatever the others hold.
//
// Measured (without adapters): 16 to 32 tokens of 7168 -> 9216, bf16 (132 MB) 23.7 us, 5.6 TB/s,
// 128 tokens 26.6 us; 128 tokens of 7168 -> 7168 E4M3 (51 MB) 16 us.  The stream of W alone takes
// 22 us of the first; what the issuing warp does for a 128-byte block between two waits bounds the
// rest (with a division for the place in the ring, and one lane instead of a uniform warp, 26.7 us).
// With 64 adapters of rank 64 (58 MB each of A and B) the third takes 44 us, 14 of them A x.
#include <algorithm>
#include <cfloat>
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

constexpr int kShrinkThreads = 128;
// Tokens times rank from which a warp takes two rows by itself.  Whole projections, this way and
// the other: 2048 rows, d 7168, 8 adapters 28.7 and 32.9 us, 32 adapters 45.4 and 42.1; d 2048, fp32 13.4
// and 15.5; 512 rows 28.5 and 28.8; 128 rows, d 2048 7.2 and 6.4.
constexpr int kShrinkMany = 1024;

// f as three bf16 terms (an infinite or NaN first term stands alone).
__device__ __forceinline__ void split3(float f, __nv_bfloat16 (&t)[3]) {
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        t[p] = __float2bfloat16_rn(f);
        const float b = __bfloat162float(t[p]);
        f = fabsf(b) <= 3.4028234e38f ? f - b : 0.0f;
    }
}

// 8 elements of x as loaded.
template <int DT>
struct XRaw {
    uint4 w[DT == MOE_DTYPE_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, long long i) {
        if constexpr (DT == MOE_DTYPE_F32) {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
            w[0] = q[0];
            w[1] = q[1];
        } else if constexpr (DT == MOE_DTYPE_BF16) {
            w[0] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + i);
            w[0].x = v.x;
            w[0].y = v.y;
        }
    }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
        if constexpr (DT == MOE_DTYPE_F32) {
            f[0] = make_float2(__uint_as_float(w[0].x), __uint_as_float(w[0].y));
            f[1] = make_float2(__uint_as_float(w[0].z), __uint_as_float(w[0].w));
            f[2] = make_float2(__uint_as_float(w[1].x), __uint_as_float(w[1].y));
            f[3] = make_float2(__uint_as_float(w[1].z), __uint_as_float(w[1].w));
        } else if constexpr (DT == MOE_DTYPE_BF16) {
            unpack_bf16x8_f2(w[0], f);
        } else {
            f[0] = unpack_e4m3x2<false>(w[0].x);
            f[1] = unpack_e4m3x2<true>(w[0].x);
            f[2] = unpack_e4m3x2<false>(w[0].y);
            f[3] = unpack_e4m3x2<true>(w[0].y);
        }
    }
};

// Blocks [0, shrink_blocks): A_a x[t], two rows of A_a to a warp (MANY), or one to the
// block's four, with the loads of several steps along d together: HBM (L2 for adapters that
// several tokens share) bounds it.  The blocks after them write the three bf16 terms of
// fp32 x.  Blocks of 128 threads leave room for one of the projection kernel's beside them.
template <int DT, bool MANY>
__global__ void __launch_bounds__(kShrinkThreads, 4) lora_shrink_kernel(const __grid_constant__ LoraArgs a, int shrink_blocks) {
    constexpr int ROWS = MANY ? 2 : 1, kWarps = kShrinkThreads / 32, kSplit = MANY ? 1 : kWarps;
    constexpr int kSteps = DT == MOE_DTYPE_F32 ? 4 : 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, chunks = a.d / 8;
    // in this order: what the kernel before wrote is there when the projection kernel starts
    pdl_wait_primary();
    pdl_allow_dependents();
    if ((int)blockIdx.x >= shrink_blocks) {
        const long long plane = (long long)a.T * a.d;
        for (int i = (blockIdx.x - shrink_blocks) * kShrinkThreads + tid; i < a.T * chunks;
             i += (gridDim.x - shrink_blocks) * kShrinkThreads) {
            const int t = i / chunks, c = (i - t * chunks) * 8;
            float f[8];
            load8_f32(a.x, MOE_DTYPE_F32, t * a.x_ld + c, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += 0.0f;       // every NaN has its first fraction bit set
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // truncated, so that all terms have x's sign: 8 bits each
                    w[e] = __byte_perm(__float_as_uint(f[2 * e]), __float_as_uint(f[2 * e + 1]), 0x7632);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float b = __uint_as_float(h ? w[e] & 0xffff0000u : w[e] << 16);
                        // an infinite or NaN first term stands alone
                        f[2 * e + h] = fabsf(b) <= FLT_MAX ? f[2 * e + h] - b : 0.0f;
                    }
                }
                *reinterpret_cast<uint4*>(a.xs + p * plane + (long long)t * a.d + c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        return;
    }
    const int unit = MANY ? blockIdx.x * kWarps + warp : blockIdx.x;
    if (unit >= a.T * a.r / ROWS) return;
    const int t = unit / (a.r / ROWS), j0 = (unit - t * (a.r / ROWS)) * ROWS;
    const int ad = adapter_of(a, t);
    if (ad < 0) return;                  // nobody reads its v
    const uint4* rows = reinterpret_cast<const uint4*>(a.la + ((long long)ad * a.r + j0) * a.d);
    float2 sum[ROWS][4];
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[j][e] = make_float2(0.0f, 0.0f);
    for (int c0 = MANY ? lane : tid; c0 < chunks; c0 += 32 * kSplit * kSteps) {
        uint4 w[kSteps][ROWS];
        XRaw<DT> x[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int c = c0 + 32 * kSplit * k;
            if (c < chunks) {
#pragma unroll
                for (int j = 0; j < ROWS; ++j) w[k][j] = __ldg(rows + (long long)j * chunks + c);
                x[k].load(a.x, t * a.x_ld + c * 8);
            }
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            if (c0 + 32 * kSplit * k < chunks) {
                float2 v[4];
                x[k].get(v);
#pragma unroll
                for (int j = 0; j < ROWS; ++j) {
                    float2 u[4];
                    unpack_bf16x8_f2(w[k][j], u);
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[j][e] = ffma2(u[e], v[e], sum[j][e]);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        const float2 p = make_float2((sum[j][0].x + sum[j][1].x) + (sum[j][2].x + sum[j][3].x),
                                     (sum[j][0].y + sum[j][1].y) + (sum[j][2].y + sum[j][3].y));
        float f = warp_sum(p.x + p.y);
        if constexpr (!MANY) {
            __shared__ float s_part[kWarps];
            if (lane == 0) s_part[warp] = f;
            __syncthreads();
            f = (s_part[0] + s_part[1]) + (s_part[2] + s_part[3]);
        }
        if (MANY ? lane == 0 : tid == 0) {
            if (a.x_scale) f *= a.x_scale[t];
            const int i = t * a.r + j0 + j;
            if (a.vt) {
                __nv_bfloat16 v[3];
                split3(f * a.ls[ad], v);
#pragma unroll
                for (int k = 0; k < 3; ++k) a.vt[(long long)k * a.T * a.r + i] = v[k];
            } else {
                a.v[i] = f;
            }
        }
    }
}

// ---- projection --------------------------------------------------------------

struct ProjArgs {
    LoraArgs l;
    CUtensorMap wmap, xmap;     // W [N, d]; x [T, d], or its terms [3, T, d]
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

__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
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
    int seg[kLoraMaxT + 1];    // first sorted token of each adapter among the own tokens
    int segs;
    int starts[kLoraMaxT / 32];
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
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
    // [3][own tokens][v_stride]: bf16 terms of v times the adapter's scale
    __nv_bfloat16* vs = reinterpret_cast<__nv_bfloat16*>(base + p.v_off);
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
        if (a.r > 0) tma_prefetch_map(&p.bmap);
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
    auto load_w = [&](int i, int slot) {
        mbar_arrive_expect_tx(&sm.full[slot], kStageBytes);
        tma_load_2d(ring + slot * kStageBytes, &p.wmap, (kb0 + i) * kColsPerBlock, n0, &sm.full[slot], pol);
    };
    if (warp == 0 && lane == 0)
        for (int i = 0; i < early; ++i) load_w(i, i);

    // With adapters the kernel before is the one above, which had seen the end of its own predecessor
    // before this one started: only what it writes itself is waited for, where it is read (other inputs
    // that an earlier kernel may have written come from L2, past what L1 may still hold).
    if (a.r == 0) pdl_wait_primary();

    // ---- order of the tokens: by the warps that need it first (the adapters' copies and
    // products), the others go ahead
    const bool sorter = warp == 2 || (warp >= 4 && warp < 8);
    const int sid = warp == 2 ? 128 + lane : tid - 128;
    auto sort_sync = [&] { named_bar_sync(1, 160); };
    if (a.r > 0 && sorter) {
        if (sid < kLoraMaxT) {
            const int k = sid < a.T ? adapter_of(a, sid) : INT_MAX;
            sm.key[sid] = k;
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
        }
        sort_sync();
        // an own token whose adapter differs from the one before starts an adapter in use
        const bool start = sid >= p0 && sid < p1 && sm.skey[sid] >= 0 && (sid == p0 || sm.skey[sid - 1] != sm.skey[sid]);
        const uint32_t bits = __ballot_sync(0xffffffffu, start);
        if (sid < kLoraMaxT && lane == 0) sm.starts[sid / 32] = __popc(bits);
        sort_sync();
        int before = 0, count = 0;
#pragma unroll
        for (int w = 0; w < kLoraMaxT / 32; ++w) {
            if (w < sid / 32) before += sm.starts[w];
            count += sm.starts[w];
        }
        if (start) sm.seg[before + __popc(bits & (0xffffffffu >> (31 - lane))) - 1] = sid;
        if (sid == 0) {
            sm.segs = count;
            sm.seg[count] = p1;
        }
        sort_sync();
        if (warp != 2) {
            pdl_wait_primary();
            // the terms of the own tokens' v, in 16-byte pieces, zeros beyond the rank
            const int vstr = v_stride(a.r), own = p1 - p0, pieces = vstr / 8 - 1;
            for (int i = sid; i < 3 * own * pieces; i += 128) {
                const int row = i / pieces, c = (i - row * pieces) * 8, k = row / own, q = row - k * own;
                __nv_bfloat16* dst = vs + row * vstr + c;
                if (c >= a.r) *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
                else if (sm.skey[p0 + q] >= 0) cp_async16(dst, a.vt + ((long long)k * a.T + sm.order[p0 + q]) * a.r + c);
            }
            cp_async_commit();
            cp_async_wait<0>();
            named_bar_sync(2, 128);
        }
    } else if (a.r == 0) {
        for (int t = tid; t < a.T; t += kProjThreads) sm.order[t] = t;
    }

    if (warp == 0) {
        // ===================== TMA producer =====================
        if (lane == 0) {
            auto load_x = [&](int i, int slot) {
                unsigned char* dst = ring + slot * kStageBytes + kWBytes;
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
                    tma_load_3d_plain(dst + t * kXBytes, &p.xmap, (kb0 + i) * kColsPerBlock, 0, t, &sm.full[slot]);
            };
            if (TERMS > 1 && a.r > 0) pdl_wait_primary();     // the terms of x
            for (int i = 0; i < early; ++i) load_x(i, i);
            int i = early, slot = 0;        // the ring is full: from its first place on
            uint32_t phase = 0;
            for (; i < nkb; ++i) {
                if (!wait(&sm.empty[slot], phase)) break;
                load_w(i, slot);
                load_x(i, slot);
                if (++slot == p.stages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            // every copy has landed before the CTA may exit
            for (int j = max(0, i - p.stages); j < i; ++j) mbar_wait_bounded(&sm.full[j % p.stages], (j / p.stages) & 1u);
        }
    } else if (warp == 1) {
        // ===================== MMA issuer (the whole warp, so that what the MMAs take is uniform) =====================
        const uint64_t a0 = smem_desc_sw128(smem_u32(ring), 16, 1024);
        const uint64_t b0 = smem_desc_sw128(smem_u32(ring + kWBytes), 16, 1024);
        const uint32_t idesc = F8 ? idesc_e4m3_f32(128, TP) : idesc_bf16_f32(128, TP, false, false);
        auto all_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
        int slot = 0;
        uint32_t phase = 0;
        bool run = true;
        for (int c = 0; run && c < chunks; ++c) {
            const uint32_t buf = c & 1;
            if (!all_wait(&sm.acc_empty[buf], ((c >> 1) & 1u) ^ 1u)) break;
            tc_fence_after_sync();
            const int end = min(nkb, (c + 1) * kChunkBlocks);
            for (int i = c * kChunkBlocks; i < end; ++i) {
                if (!all_wait(&sm.full[slot], phase)) {
                    run = false;
                    break;
                }
                tc_fence_after_sync();
                const uint64_t ad = a0 + ((slot * kStageBytes) >> 4), bd = b0 + ((slot * kStageBytes) >> 4);
                const bool fresh = i == c * kChunkBlocks;
                if (elect_one()) {
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
                    if (i + 1 == end) umma_commit(&sm.acc_full[buf]);
                }
                __syncwarp();
                if (++slot == p.stages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        if (elect_one()) {
            umma_commit(&sm.mma_done);
            mbar_wait_bounded(&sm.mma_done, 0);   // all MMAs have ended before TMEM is freed
        }
    } else if (warp == 2) {
        // ===================== adapter copies =====================
        if (lane == 0 && a.r > 0) {
            const int boxes = (a.r + 63) / 64, lstage = lora_stage_bytes(a.r);
            const uint32_t bulk = (uint32_t)min(kRowsM, a.N - n0) * a.r * 2;
            int it = 0, slot = 0;
            uint32_t phase = 1;
            for (; it < sm.segs; ++it) {
                const int ad = sm.skey[sm.seg[it]];
                if (!wait(&sm.lempty[slot], phase)) break;
                if (lora_bulk(a.r)) {
                    mbar_arrive_expect_tx(&sm.lfull[slot], bulk);
                    bulk_load(lring + slot * lstage, a.lb + ((long long)ad * a.N + n0) * a.r, bulk, &sm.lfull[slot], pol);
                } else {
                    mbar_arrive_expect_tx(&sm.lfull[slot], boxes * kLoraBox);
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(lring + slot * lstage + b * kLoraBox, &p.bmap, b * 64, ad * a.N + n0, &sm.lfull[slot], pol);
                }
                if (++slot == p.lora_stages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            for (int j = max(0, it - p.lora_stages); j < it; ++j)
                mbar_wait_bounded(&sm.lfull[j % p.lora_stages], (j / p.lora_stages) & 1u);
        }
    } else if (warp >= 4 && warp < 8) {
        // ===================== adapters: B_a v, 32 of the tile's rows per warp, up to 8 tokens at once =====================
        if (a.r > 0) {
            const int steps = (a.r + 15) / 16, lstage = lora_stage_bytes(a.r);
            // rows of 128 bytes with permuted chunks, or of 2 r bytes as they are
            const int pitch = lora_bulk(a.r) ? a.r * 2 : 128, swizzle = lora_bulk(a.r) ? 0 : 7;
            const int vstr = v_stride(a.r), own = p1 - p0, segs = sm.segs;
            // ldmatrix: lane's row and 16-byte chunk within a 16 x 16 block
            const int row0 = (warp - 4) * 32, lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lch = lane >> 4;
            for (int i = (warp - 4) * 32 + lane; i < (sm.seg[0] - p0) * kRowsM; i += 128) lacc[i] = 0.0f;
            // one or two tokens of an adapter: the terms of v side by side in the MMA's 8 columns (token
            // 0's in 0 to 2, token 1's in 4 to 6), a third of the MMAs
            const int term = (lane / 4) & 3, second = lane / 16;
            const __nv_bfloat16* v2 = vs + ((term < 3 ? term : 0) * own - p0 + second) * vstr + (lane & 3) * 2;
            float* out2 = lacc + ((lane & 3) / 2 - p0) * kRowsM + row0 + lane / 4;
            const int steps4 = min(steps, 4);
            const uint32_t at0 = smem_u32(lring) + (row0 + lrow) * pitch;
            uint32_t flip[4];                // byte of the lane's chunk in each k16 step
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) flip[ks] = ((ks * 2 + lch) ^ (lrow & swizzle)) << 4;
            int slot = 0, first = sm.seg[0], next = sm.seg[segs > 0];
            uint32_t phase = 0;
            for (int it = 0; it < segs; ++it) {
                const int end = next;
                if (it + 2 <= segs) next = sm.seg[it + 2];
                const bool packed = end - first <= 2;
                uint32_t pb[4][2];
                auto load_packed = [&](int k0, int n) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        pb[ks][0] = pb[ks][1] = 0u;
                        if (ks < n && term < 3 && first + second < end) {
                            pb[ks][0] = *reinterpret_cast<const uint32_t*>(v2 + first * vstr + (k0 + ks) * 16);
                            pb[ks][1] = *reinterpret_cast<const uint32_t*>(v2 + first * vstr + (k0 + ks) * 16 + 8);
                        }
                    }
                };
                if (packed) load_packed(0, steps4);
                wait(&sm.lfull[slot], phase);
                __syncwarp();
                const uint32_t tile_b = at0 + slot * lstage;
                if (packed) {
                    const bool write = (lane & 1) == 0 && first + (lane & 3) / 2 < end;
                    float* out = out2 + first * kRowsM;
                    for (int k0 = 0; k0 < steps; k0 += 4) {
                        if (k0 > 0) load_packed(k0, steps - k0);
                        float c[2][4] = {};
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (k0 + ks < steps) {
#pragma unroll
                                for (int m = 0; m < 2; ++m) {
                                    uint32_t f[4];
                                    ldmatrix_x4(tile_b + (k0 >> 2) * kLoraBox + m * 16 * pitch + flip[ks], f);
                                    mma_bf16(c[m], f[0], f[1], f[2], f[3], pb[ks][0], pb[ks][1]);
                                }
                            }
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const float lo = c[h / 2][h % 2 * 2], hi = c[h / 2][h % 2 * 2 + 1];
                            // an infinite product of the first term (an infinity in B_a) stands: the others' may
                            // be NaN or of the other sign
                            const float third = __shfl_xor_sync(0xffffffffu, lo, 1);
                            const float s = fabsf(lo) <= FLT_MAX ? lo + (hi + third) : lo;
                            if (write) out[h * 8] = k0 == 0 ? s : out[h * 8] + s;
                        }
                    }
                } else
                for (int q = first; q < end; q += 8) {
                    const int count = min(8, end - q);
                    const __nv_bfloat16* v = vs + (q - p0 + lane / 4) * vstr + (lane & 3) * 2;
                    float* out = lacc + (q - p0 + (lane & 3) * 2) * kRowsM + row0 + lane / 4;
                    const bool t0 = (lane & 3) * 2 < count, t1 = (lane & 3) * 2 + 1 < count;
                    // up to 64 columns of B_a at a time: v's fragments stay in registers over the rows
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
#pragma unroll
                        for (int m = 0; m < 32; m += 16) {
                            float c[3][4] = {};             // a sum per term: short chains of MMAs
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                if (k0 + ks < steps) {
                                    uint32_t f[4];
                                    ldmatrix_x4(tile_b + (k0 >> 2) * kLoraBox + m * pitch + flip[ks], f);
#pragma unroll
                                    for (int k = 0; k < 3; ++k) mma_bf16(c[k], f[0], f[1], f[2], f[3], b[ks][k][0], b[ks][k][1]);
                                }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float* at = out + (e & 1) * kRowsM + m + (e >> 1) * 8;
                                const float s = fabsf(c[0][e]) <= FLT_MAX ? c[0][e] + (c[1][e] + c[2][e]) : c[0][e];
                                if ((e & 1) ? t1 : t0) *at = k0 == 0 ? s : *at + s;
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.lempty[slot]);
                first = end;
                if (++slot == p.lora_stages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp >= 8) {
        // ===================== epilogue: blocks of sums into registers =====================
        float2 acc[TP / 2];
#pragma unroll
        for (int t = 0; t < TP / 2; ++t) acc[t] = make_float2(0.0f, 0.0f);
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
                    for (int e = 0; e < 16; e += 2) {
                        float2 u = make_float2(v[e], v[e + 1]);
                        // beside an infinite first term (of an infinite weight) the others are infinite of
                        // its sign, or NaN where a term is 0: that one stands
                        if (g > 0) u = make_float2(fminf(u.x, FLT_MAX), fminf(u.y, FLT_MAX));
                        acc[(t + e) / 2] = fadd2(acc[(t + e) / 2], u);
                    }
                }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.acc_empty[buf]);
        }
        // the last block's MMAs have ended: nothing reads or writes the ring any more
        const int m = (warp & 3) * 32 + lane;
#pragma unroll
        for (int t = 0; t < TP; ++t)
            if (t < a.T) red[t * kRowsM + m] = t % 2 ? acc[t / 2].y : acc[t / 2].x;
    }
    tc_fence_before_sync();
    if (p.split > 1) cluster_sync_all();
    else __syncthreads();
    tc_fence_after_sync();

    // ---- the cluster's sum of this CTA's tokens, scales, adapter part, output
    const int warps = kProjThreads / 32, n = n0 + lane * 4;
    float4 wsc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if constexpr (F8) {
        if (n < a.N) wsc = make_float4(__ldcg(a.w_scale + n), __ldcg(a.w_scale + n + 1), __ldcg(a.w_scale + n + 2), __ldcg(a.w_scale + n + 3));
    }
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
                const float xs = __ldcg(a.x_scale + t);
                s.x *= xs * wsc.x;
                s.y *= xs * wsc.y;
                s.z *= xs * wsc.z;
                s.w *= xs * wsc.w;
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

template <int TP, bool F8, int TERMS>
cudaError_t launch_project(ProjArgs& p, cudaStream_t s) {
    const LoraArgs& a = p.l;
    constexpr int kStageBytes = kWBytes + TERMS * TP * kBlockBytes;
    auto kern = lora_project_kernel<TP, F8, TERMS>;
    static std::atomic<uint64_t> done;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kProjSmem, done);
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count();
    const int tiles = (a.N + kRowsM - 1) / kRowsM;
    const bool low = a.r > 0;
    p.blocks = (a.d * (F8 ? 1 : 2) + kBlockBytes - 1) / kBlockBytes;
    // Split d while the clusters still run at once (clusters of 3 or 8 do not fill a
    // GPC: 120 CTAs in threes do, 144 do not) and a CTA keeps two blocks or more.  Threes: 32 tokens of
    // 7168 -> 5120 16.0 us against 19.8 in pairs; sixes gain 6 % there and lose 13 % at d 2048.
    p.split = 1;
    for (int k : {2, 3, 4, 8})
        if (tiles * k <= (k == 3 || k == 8 ? sms * 13 / 16 : sms) && p.blocks / k >= 2) p.split = k;
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
    while (p.stages < 2 && p.split <= 4) {
        p.split *= 2;     // fewer own tokens: room for the ring
        plan();
    }
    p.stages = std::min(p.stages, (p.blocks + p.split - 1) / p.split);
    // At least half an SM's shared memory: two CTAs that shared an SM's TMEM could wait for each
    // other's through their clusters.
    const size_t smem = std::max((size_t)(1024 + p.wring_off + std::max(p.stages * kStageBytes, a.T * kRowsM * 4)),
                                 (size_t)116 * 1024);
    if (p.stages < 1 || smem > (size_t)kProjSmem) return cudaErrorInvalidConfiguration;
    const bool terms = TERMS == 3;       // fp32 x comes as its terms
    const bool maps = encode_rows(&p.wmap, a.w, 0, a.N, a.d, a.w_ld, kRowsM, F8) &&
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

template <bool F8, int TERMS>
cudaError_t launch_tp(const LoraArgs& a, cudaStream_t s) {
    ProjArgs p = {};
    p.l = a;
    if (a.T <= 16) return launch_project<16, F8, TERMS>(p, s);
    if (a.T <= 32) return launch_project<32, F8, TERMS>(p, s);
    if (a.T <= 64) return launch_project<64, F8, TERMS>(p, s);
    return launch_project<128, F8, TERMS>(p, s);
}

}  // namespace

size_t lora_workspace_bytes(int T, int d, int r, size_t* v_off, size_t* xs_off) {
    size_t off = 512;
    *v_off = off;
    off += ((size_t)T * r * 6 + 255) / 256 * 256;
    *xs_off = off;
    return off + (size_t)T * d * 6;
}

cudaError_t launch_lora_project(const LoraArgs& args, cudaStream_t s) {
    LoraArgs a = args;
    const bool f32 = a.x_dt == MOE_DTYPE_F32, f8 = a.x_dt == MOE_DTYPE_FP8_E4M3;
    const bool gemv = lora_gemv_fits(a);
    if (gemv && (a.r == 0 || lora_gemv_own_v(a))) return launch_lora_gemv(a, s);
    if (!gemv) a.vt = reinterpret_cast<__nv_bfloat16*>(a.v);
    // v = A_a x and the terms of fp32 x, in one small kernel ahead of the projection
    const bool many = a.T * a.r >= kShrinkMany;
    const int shrink_blocks = many ? (a.T * a.r + kShrinkThreads / 16 - 1) / (kShrinkThreads / 16) : a.T * a.r;
    const int split_blocks =
        f32 && !gemv ? std::min(4 * device_sm_count(), (a.T * (a.d / 8) + kShrinkThreads - 1) / kShrinkThreads) : 0;
    if (shrink_blocks + split_blocks > 0) {
        auto kern = f32  ? (many ? lora_shrink_kernel<MOE_DTYPE_F32, true> : lora_shrink_kernel<MOE_DTYPE_F32, false>)
                    : f8 ? (many ? lora_shrink_kernel<MOE_DTYPE_FP8_E4M3, true> : lora_shrink_kernel<MOE_DTYPE_FP8_E4M3, false>)
                         : (many ? lora_shrink_kernel<MOE_DTYPE_BF16, true> : lora_shrink_kernel<MOE_DTYPE_BF16, false>);
        const cudaError_t e = launch_pdl(kern, dim3((unsigned)(shrink_blocks + split_blocks)), dim3(kShrinkThreads), 0, s, a,
                                         shrink_blocks);
        if (e != cudaSuccess) return e;
    }
    if (gemv) return launch_lora_gemv(a, s);
    if (f8) return launch_tp<true, 1>(a, s);
    return f32 ? launch_tp<false, 3>(a, s) : launch_tp<false, 1>(a, s);
}

}  // namespace moe
