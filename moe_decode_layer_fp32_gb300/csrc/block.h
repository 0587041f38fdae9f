// Arguments and launchers of the decode-block operators (norm, cache append,
// paged attention, adapter projection); internal to the library.
#pragma once

#include <atomic>

#include "../../include/moe_block.h"
#include "kernels.h"

namespace moe {

// Records the message of a failed call (moe_last_error) and returns `code`.
int api_fail(int code, const char* fmt, ...);

struct NormArgs {
    const void* x;
    const void* residual;      // null: none
    void* residual_out;        // null: not written
    const void* weight;        // null: ones
    void* y;
    float* y_scale;            // E4M3 output
    long long x_ld, r_ld, ro_ld, y_ld;
    int x_dt, r_dt, w_dt, y_dt;
    int T, d, group;
    float eps;
};
cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t s);

struct AppendArgs {
    const void* k;
    const void* v;
    const void* q;             // null: none
    void* q_out;
    long long k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, o_ts, o_hs;
    int in_dt, T, q_heads;
    moe_kv_cache c;
    const int32_t* table;
    long long table_ld;
    int R, max_pages;
    const int32_t* positions;
    const int32_t* req;        // null: token t is request t
    const float* cos_sin;
    int rot, max_pos;
    int32_t* status;
};
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s);

struct QkAppendArgs : AppendArgs {
    const void* q_weight;      // null: ones
    const void* k_weight;
    int w_dt, axes;            // axes 0: the rotation is that of `positions`
    float eps;
    const int32_t* axis_positions;   // [axes, T]
    uint8_t axis[128];         // of each pair
};
cudaError_t launch_qk_norm_append(const QkAppendArgs& a, cudaStream_t s);

// What the calls on pages have in common: the requests' tokens and their table.
struct PageArgs {
    const int32_t* table;
    long long table_ld;
    int B, max_pages, page_size;
    const int32_t* seq_lens;
    int32_t* status;
};
struct BoundsArgs : PageArgs {
    moe_kv_cache c;
    void* bounds;
    const int32_t* first;      // null: from the first token on
};
struct ScoresArgs : PageArgs {
    moe_kv_cache c;
    const void* q;
    long long q_bs, q_hs;
    int q_dt, group;           // group = q_heads / c.heads
    const void* bounds;
    float* scores;
};
struct SelectArgs : PageArgs {
    const float* scores;
    int heads, keep, sinks, recent;
    int32_t* tables;
    int32_t* lens;
};
cudaError_t launch_page_bounds(const BoundsArgs& a, cudaStream_t s);
cudaError_t launch_page_scores(const ScoresArgs& a, cudaStream_t s);
cudaError_t launch_page_select(const SelectArgs& a, cudaStream_t s);

struct AttnArgs {
    const void* q;
    void* out;
    float* lse;
    long long q_bs, q_hs, o_bs, o_hs;
    int q_dt, o_dt, B, q_heads, group;   // group = q_heads / c.heads
    moe_kv_cache c;
    const int32_t* table;
    long long table_ld;
    int max_pages;
    const int32_t* seq_lens;
    float scale, softcap;
    int window;
    int page_shift;            // log2 of the page size, or -1 (set by the launcher)
    int far;                   // cache offsets pass 2^32 steps of 16 bytes (set by the launcher)
    int32_t* status;
    uint32_t* done;            // counters, one per unit (zero between calls)
    uint32_t* group_done;      // and one per part
    float* parts;              // partial results
};
size_t attn_workspace_bytes(int B, int q_heads, int heads, int head_dim, size_t* done_off, size_t* group_off,
                            size_t* parts_off);
cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t s);
// B requests and heads, each with a table and a length of its own.
cudaError_t launch_attn_pages(const AttnArgs& a, cudaStream_t s);

struct LoraArgs {
    const void* x;
    const float* x_scale;
    const void* w;
    const float* w_scale;
    const __nv_bfloat16* la;   // null: no adapters
    const __nv_bfloat16* lb;
    const float* ls;
    const int32_t* adapter;
    void* y;
    long long x_ld, w_ld, y_ld;
    int x_dt, y_dt, T, d, N, na, r;
    int32_t* status;
    float* v;                  // [T, r]: A_a x[t], unscaled ...
    __nv_bfloat16* vt;         // ... or [3, T, r]: the bf16 terms of A_a x[t] times the adapter's scale
    __nv_bfloat16* xs;         // [3, T, d]: bf16 terms of fp32 x
};
constexpr int kLoraMaxT = 128;
constexpr int kLoraMaxRank = 128;
size_t lora_workspace_bytes(int T, int d, int r, size_t* v_off, size_t* xs_off);
cudaError_t launch_lora_project(const LoraArgs& a, cudaStream_t s);
// One or two tokens on the CUDA cores; unless lora_gemv_own_v, a.v has been formed before.
bool lora_gemv_fits(const LoraArgs& a);
bool lora_gemv_own_v(const LoraArgs& a);
cudaError_t launch_lora_gemv(const LoraArgs& a, cudaStream_t s);

// Allows a kernel `bytes` of dynamic shared memory, once per device: `done` is the kernel's own.
inline cudaError_t allow_smem(const void* kern, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Blocks of a kernel that an SM holds.  The runtime is asked once per device, threads and shared memory:
// `last` is the kernel's own, 0 or the last question (24 bits of shared memory, 12 of threads, 12 of
// device + 1) and its answer.
inline cudaError_t blocks_per_sm(const void* kern, int threads, size_t smem, std::atomic<uint64_t>& last, int* blocks) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t asked = (uint64_t)smem << 40 | (uint64_t)threads << 28 | (uint64_t)(dev + 1) << 16;
    const uint64_t have = last.load(std::memory_order_relaxed);
    if ((have & ~(uint64_t)0xffff) == asked) {
        *blocks = (int)(have & 0xffff);
        return cudaSuccess;
    }
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, kern, threads, smem);
    if (e == cudaSuccess) {
        *blocks = *blocks > 0 ? *blocks : 1;
        last.store(asked | (uint64_t)*blocks, std::memory_order_relaxed);
    }
    return e;
}

// Launch configuration of a programmatic dependent: the kernel may start
// before the one ahead of it on the stream has ended, and waits for it
// (griddepcontrol.wait) before it reads anything that one may have written.
template <typename... P, typename... A>
inline cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// ---- pairs of fp32 ------------------------------------------------------------

__device__ __forceinline__ float2 pair_op(unsigned long long d) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    unsigned long long d;
    asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%1, %2};\n\tmov.b64 rb, {%3, %4};\n\tadd.rn.f32x2 %0, ra, rb;\n\t}"
        : "=l"(d)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return pair_op(d);
}
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    unsigned long long d;
    asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%1, %2};\n\tmov.b64 rb, {%3, %4};\n\tmul.rn.f32x2 %0, ra, rb;\n\t}"
        : "=l"(d)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return pair_op(d);
}

// ---- element loads and stores of a run-time type (uniform branches) ----------

// 8 consecutive elements as fp32; p + i is aligned to 8 elements (at most 16 bytes).
__device__ __forceinline__ void load8_f32(const void* p, int dt, long long i, float (&f)[8]) {
    if (dt == MOE_DTYPE_BF16) {
        unpack_bf16x8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i), f);
    } else {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = q[0], b = q[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(void* p, int dt, long long i, const float (&f)[8]) {
    if (dt == MOE_DTYPE_BF16) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
    } else {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}
// Values outside E4M3's range go to +-448.  (The halves of a word by name rather than by shifts and
// masks: the conversions take either half of a register.)
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
// The two E4M3 of v's lower (HI: upper) half in f16, and in fp32.
template <bool HI>
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t r;
    if constexpr (HI) asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(v));
    else asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(v));
    return r;
}
template <bool HI>
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t v) {
    const uint32_t h = e4m3x2_to_f16x2<HI>(v);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 8 elements of any of the three types.
__device__ __forceinline__ void load8_any(const void* p, int dt, long long i, float (&f)[8]) {
    if (dt == MOE_DTYPE_FP8_E4M3) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t w = e < 2 ? v.x : v.y;
            const float2 u = e % 2 ? unpack_e4m3x2<true>(w) : unpack_e4m3x2<false>(w);
            f[2 * e] = u.x;
            f[2 * e + 1] = u.y;
        }
    } else {
        load8_f32(p, dt, i, f);
    }
}

__device__ __forceinline__ void cp_async16_to(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros where size is 0 (src is then not read).
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, uint32_t size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}

// -1 for a token without an adapter; an index beyond the adapters is reported and counts as none.
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int t) {
    const int i = __ldcg(a.adapter + t);     // from L2: the projection reads it without a wait of its own
    if (i >= a.na) set_status(a.status, MOE_ERR_DEVICE);
    return i >= 0 && i < a.na ? i : -1;
}

// C += A B: 16 x 16 by 16 x 8, bf16 into fp32.
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same in f16.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
// bf16 parts by truncation: p = hi + rest exactly, rest of p's sign.
__device__ __forceinline__ float bf16_trunc(float p) { return __uint_as_float(__float_as_uint(p) & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_hi(float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632); }

}  // namespace moe
