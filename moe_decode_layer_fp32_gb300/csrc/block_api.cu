// C ABI of the decode-block operators: host-side argument checks and launches.
// See include/moe_block.h for the contract of each call.
#include <algorithm>
#include <climits>
#include <cmath>

#include "block.h"

namespace {

using moe::api_fail;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool is_act(int dt) { return dt == MOE_DTYPE_F32 || dt == MOE_DTYPE_BF16; }

int launched(cudaError_t e, const char* who) {
    return e == cudaSuccess ? MOE_OK : api_fail(MOE_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

// A matrix of rows of d elements: present, aligned, its rows `step` elements apart or more.
int check_rows(const void* p, long long ld, int d, int step, const char* what, const char* who) {
    if (!p || !aligned16(p)) return api_fail(MOE_ERR_INVALID_ARG, "%s: %s null or unaligned", who, what);
    if (ld < d || ld % step != 0)
        return api_fail(MOE_ERR_INVALID_ARG, "%s: row stride %lld of %s must be a multiple of %d, at least %d", who,
                        ld, what, step, d);
    return MOE_OK;
}

int check_cache(const moe_kv_cache* c, const char* who) {
    if (!c) return api_fail(MOE_ERR_INVALID_ARG, "%s: cache is null", who);
    const bool f8 = c->dtype == MOE_DTYPE_FP8_E4M3;
    if (c->dtype != MOE_DTYPE_BF16 && !f8) return api_fail(MOE_ERR_UNSUPPORTED, "%s: cache dtype %d", who, c->dtype);
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v))
        return api_fail(MOE_ERR_INVALID_ARG, "%s: cache null or unaligned", who);
    if (f8 != (c->k_scale != nullptr) || f8 != (c->v_scale != nullptr))
        return api_fail(MOE_ERR_INVALID_ARG, "%s: k_scale and v_scale go with an E4M3 cache", who);
    const int step = f8 ? 16 : 8;
    if (c->head_dim < step || c->head_dim % step != 0)
        return api_fail(MOE_ERR_INVALID_ARG, "%s: head_dim=%d must be a positive multiple of %d", who, c->head_dim, step);
    if (c->head_dim > 256) return api_fail(MOE_ERR_UNSUPPORTED, "%s: head_dim=%d exceeds 256", who, c->head_dim);
    if (c->num_pages < 1 || c->page_size < 1 || c->heads < 1)
        return api_fail(MOE_ERR_INVALID_ARG, "%s: need num_pages, page_size, heads >= 1 (%d, %d, %d)", who,
                        c->num_pages, c->page_size, c->heads);
    const int64_t st[6] = {c->k_page_stride, c->k_slot_stride, c->k_head_stride,
                           c->v_page_stride, c->v_slot_stride, c->v_head_stride};
    for (int64_t v : st)
        if (v < 0 || v % step != 0)
            return api_fail(MOE_ERR_INVALID_ARG, "%s: cache strides must be multiples of 16 bytes", who);
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_rmsnorm(const void* x, int x_dtype, int64_t x_ld, const void* residual, int residual_dtype,
                int64_t residual_ld, void* residual_out, int64_t residual_out_ld, const void* weight,
                int weight_dtype, float eps, int T, int d, void* y, int y_dtype, int64_t y_ld,
                float* y_scale, int group, void* stream) {
    const char* who = "moe_rmsnorm";
    if (T < 0 || d < 8 || d % 8 != 0)
        return api_fail(MOE_ERR_INVALID_ARG, "%s: need T >= 0 and d a positive multiple of 8 (T=%d d=%d)", who, T, d);
    if (d > 32768) return api_fail(MOE_ERR_UNSUPPORTED, "%s: d=%d exceeds 32768", who, d);
    if (!(eps >= 0.0f) || std::isinf(eps)) return api_fail(MOE_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
    const bool f8 = y_dtype == MOE_DTYPE_FP8_E4M3;
    if (!is_act(x_dtype) || !(is_act(y_dtype) || f8) || ((residual || residual_out) && !is_act(residual_dtype)) ||
        (weight && !is_act(weight_dtype)))
        return api_fail(MOE_ERR_UNSUPPORTED, "%s: dtypes x %d, residual %d, weight %d, y %d", who, x_dtype,
                        residual_dtype, weight_dtype, y_dtype);
    if (group != 0 && (group != 128 || !f8 || d % 128 != 0))
        return api_fail(MOE_ERR_INVALID_ARG, "%s: group is 0, or 128 for E4M3 output with d %% 128 == 0 (group=%d d=%d)",
                        who, group, d);
    if (f8 != (y_scale != nullptr)) return api_fail(MOE_ERR_INVALID_ARG, "%s: y_scale goes with E4M3 output", who);
    if (T == 0) return MOE_OK;
    int rc;
    if ((rc = check_rows(x, x_ld, d, 8, "x", who)) || (rc = check_rows(y, y_ld, d, 8, "y", who)) ||
        (residual && (rc = check_rows(residual, residual_ld, d, 8, "residual", who))) ||
        (residual_out && (rc = check_rows(residual_out, residual_out_ld, d, 8, "residual_out", who))))
        return rc;
    if (weight && !aligned16(weight)) return api_fail(MOE_ERR_INVALID_ARG, "%s: weight unaligned", who);
    moe::NormArgs a = {};
    a.x = x; a.residual = residual; a.residual_out = residual_out; a.weight = weight; a.y = y; a.y_scale = y_scale;
    a.x_ld = x_ld; a.r_ld = residual_ld; a.ro_ld = residual_out_ld; a.y_ld = y_ld;
    a.x_dt = x_dtype; a.r_dt = residual_dtype; a.w_dt = weight_dtype; a.y_dt = y_dtype;
    a.T = T; a.d = d; a.group = group; a.eps = eps;
    return launched(moe::launch_rmsnorm(a, as_stream(stream)), who);
}

int moe_kv_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                  int64_t v_token_stride, int64_t v_head_stride, int in_dtype, int T,
                  const moe_kv_cache* cache, const int32_t* block_table, int64_t table_ld, int R,
                  int max_pages, const int32_t* positions, const int32_t* req, const float* cos_sin,
                  int rot, int max_pos, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                  void* q_out, int64_t qo_token_stride, int64_t qo_head_stride, int q_heads,
                  int32_t* status, void* stream) {
    const char* who = "moe_kv_append";
    int rc = check_cache(cache, who);
    if (rc) return rc;
    if (!is_act(in_dtype)) return api_fail(MOE_ERR_UNSUPPORTED, "%s: dtype %d of k, v", who, in_dtype);
    if (T < 0 || R < 0 || max_pages < 0 || table_ld < max_pages)
        return api_fail(MOE_ERR_INVALID_ARG, "%s: need T, R, max_pages >= 0 and table_ld >= max_pages (%d, %d, %d, %lld)",
                        who, T, R, max_pages, (long long)table_ld);
    if (rot < 0 || rot % 2 != 0 || rot > cache->head_dim || (rot > 0) != (cos_sin != nullptr) || (rot > 0 && max_pos < 1))
        return api_fail(MOE_ERR_INVALID_ARG, "%s: rot=%d must be even, at most head_dim=%d, and go with cos_sin of max_pos >= 1 rows",
                        who, rot, cache->head_dim);
    if ((q != nullptr) != (q_out != nullptr) || (q && q_heads < 1))
        return api_fail(MOE_ERR_INVALID_ARG, "%s: q and q_out go together, with q_heads >= 1", who);
    if (T == 0) return MOE_OK;
    if (!k || !v || !positions || !block_table) return api_fail(MOE_ERR_INVALID_ARG, "%s: null pointer", who);
    const uintptr_t size = in_dtype == MOE_DTYPE_BF16 ? 2 : 4;
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)q | (uintptr_t)q_out) % size != 0)
        return api_fail(MOE_ERR_INVALID_ARG, "%s: k, v or q not aligned to its elements", who);
    moe::AppendArgs a = {};
    a.k = k; a.v = v; a.q = q; a.q_out = q_out;
    a.k_ts = k_token_stride; a.k_hs = k_head_stride; a.v_ts = v_token_stride; a.v_hs = v_head_stride;
    a.q_ts = q_token_stride; a.q_hs = q_head_stride; a.o_ts = qo_token_stride; a.o_hs = qo_head_stride;
    a.in_dt = in_dtype; a.T = T; a.q_heads = q ? q_heads : 0;
    a.c = *cache;
    a.table = block_table; a.table_ld = table_ld; a.R = R; a.max_pages = max_pages;
    a.positions = positions; a.req = req; a.cos_sin = cos_sin; a.rot = rot; a.max_pos = max_pos;
    a.status = status;
    return launched(moe::launch_kv_append(a, as_stream(stream)), who);
}

size_t moe_attn_workspace_bytes(int B, int q_heads, int heads, int head_dim) {
    if (B < 0 || q_heads < 1 || heads < 1 || q_heads % heads != 0 || head_dim < 8 || head_dim % 8 != 0 || head_dim > 256)
        return 0;
    size_t d, g, p;
    return moe::attn_workspace_bytes(B, q_heads, heads, head_dim, &d, &g, &p);
}

int moe_attn_decode(const void* q, int q_dtype, int64_t q_batch_stride, int64_t q_head_stride, int B,
                    int q_heads, const moe_kv_cache* cache, const int32_t* block_table,
                    int64_t table_ld, int max_pages, const int32_t* seq_lens, float scale, int window,
                    float softcap, void* out, int out_dtype, int64_t out_batch_stride,
                    int64_t out_head_stride, float* lse, void* ws, size_t ws_bytes, void* stream) {
    const char* who = "moe_attn_decode";
    int rc = check_cache(cache, who);
    if (rc) return rc;
    if (!is_act(q_dtype) || !is_act(out_dtype))
        return api_fail(MOE_ERR_UNSUPPORTED, "%s: dtypes q %d, out %d", who, q_dtype, out_dtype);
    if (B < 0 || q_heads < 1 || q_heads % cache->heads != 0)
        return api_fail(MOE_ERR_INVALID_ARG, "%s: need B >= 0 and q_heads a multiple of the cache's %d heads (B=%d q_heads=%d)",
                        who, cache->heads, B, q_heads);
    if (max_pages < 0 || table_ld < max_pages || window < 0 || !(softcap >= 0.0f) || std::isinf(softcap) || !std::isfinite(scale))
        return api_fail(MOE_ERR_INVALID_ARG, "%s: need max_pages >= 0, table_ld >= max_pages, window >= 0, a finite softcap >= 0 and scale",
                        who);
    if (B == 0) return MOE_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out) || (q_batch_stride | q_head_stride | out_batch_stride | out_head_stride) % 8 != 0)
        return api_fail(MOE_ERR_INVALID_ARG, "%s: q or out null or unaligned, or a stride no multiple of 8", who);
    if (!block_table || !seq_lens) return api_fail(MOE_ERR_INVALID_ARG, "%s: null pointer", who);
    size_t done_off, group_off, parts_off;
    const size_t need = moe::attn_workspace_bytes(B, q_heads, cache->heads, cache->head_dim, &done_off, &group_off, &parts_off);
    if (!ws || !aligned16(ws)) return api_fail(MOE_ERR_INVALID_ARG, "%s: workspace null or unaligned", who);
    if (ws_bytes < need) return api_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu required", who, ws_bytes, need);
    moe::AttnArgs a = {};
    a.q = q; a.out = out; a.lse = lse;
    a.q_bs = q_batch_stride; a.q_hs = q_head_stride; a.o_bs = out_batch_stride; a.o_hs = out_head_stride;
    a.q_dt = q_dtype; a.o_dt = out_dtype; a.B = B; a.q_heads = q_heads; a.group = q_heads / cache->heads;
    a.c = *cache;
    a.table = block_table; a.table_ld = table_ld; a.max_pages = max_pages; a.seq_lens = seq_lens;
    a.scale = scale; a.softcap = softcap; a.window = window;
    a.status = static_cast<int32_t*>(ws);
    a.done = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + done_off);
    a.group_done = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + group_off);
    a.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + parts_off);
    return launched(moe::launch_attn_decode(a, as_stream(stream)), who);
}

size_t moe_lora_workspace_bytes(int T, int d, int r) {
    if (T < 0 || T > moe::kLoraMaxT || d < 8 || d % 8 != 0 || d > 32768 || r < 0 || r % 8 != 0 || r > moe::kLoraMaxRank) return 0;
    size_t v, x;
    return moe::lora_workspace_bytes(T, d, r, &v, &x);
}

int moe_lora_project(const void* x, int x_dtype, int64_t x_ld, const float* x_scale, int T, int d,
                     const void* w, int w_dtype, int64_t w_ld, const float* w_scale, int N,
                     const void* lora_a, const void* lora_b, const float* lora_scale, int n_adapters,
                     int r, const int32_t* adapter, void* y, int y_dtype, int64_t y_ld, void* ws,
                     size_t ws_bytes, void* stream) {
    const char* who = "moe_lora_project";
    const bool f8 = x_dtype == MOE_DTYPE_FP8_E4M3;
    if (!(f8 ? w_dtype == MOE_DTYPE_FP8_E4M3 : is_act(x_dtype) && w_dtype == MOE_DTYPE_BF16) || !is_act(y_dtype))
        return api_fail(MOE_ERR_UNSUPPORTED, "%s: dtypes x %d, w %d, y %d", who, x_dtype, w_dtype, y_dtype);
    if (f8 != (x_scale != nullptr) || f8 != (w_scale != nullptr))
        return api_fail(MOE_ERR_INVALID_ARG, "%s: x_scale and w_scale go with E4M3 x and w", who);
    const int step = f8 ? 16 : 8;
    if (T < 0 || d < step || d % step != 0 || N < 8 || N % 8 != 0)
        return api_fail(MOE_ERR_INVALID_ARG, "%s: need T >= 0, d a positive multiple of %d, N of 8 (T=%d d=%d N=%d)", who,
                        step, T, d, N);
    if (T > moe::kLoraMaxT || d > 32768)
        return api_fail(MOE_ERR_UNSUPPORTED, "%s: T=%d exceeds %d or d=%d exceeds 32768", who, T, moe::kLoraMaxT, d);
    const bool has = lora_a || lora_b || lora_scale || adapter;
    if (has != (r > 0) || (has && (!lora_a || !lora_b || !lora_scale || !adapter || n_adapters < 1)))
        return api_fail(MOE_ERR_INVALID_ARG, "%s: adapters need lora_a, lora_b, lora_scale, adapter, n_adapters >= 1 and r > 0; without them r = 0",
                        who);
    if (r % 8 != 0 || r > moe::kLoraMaxRank || r < 0)
        return api_fail(r < 0 || r % 8 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED, "%s: r=%d must be a multiple of 8 up to %d",
                        who, r, moe::kLoraMaxRank);
    if (has && (long long)n_adapters * std::max(N, r) > INT_MAX)
        return api_fail(MOE_ERR_UNSUPPORTED, "%s: %d adapters of N=%d rows exceed 2^31 rows", who, n_adapters, N);
    if (T == 0) return MOE_OK;
    int rc;
    const int xstep = x_dtype == MOE_DTYPE_F32 ? 4 : step;
    if ((rc = check_rows(x, x_ld, d, xstep, "x", who)) || (rc = check_rows(w, w_ld, d, step, "w", who)) ||
        (rc = check_rows(y, y_ld, N, 8, "y", who)))
        return rc;
    if (!aligned16(lora_a) || !aligned16(lora_b)) return api_fail(MOE_ERR_INVALID_ARG, "%s: lora_a or lora_b unaligned", who);
    size_t v_off, xs_off;
    const size_t need = moe::lora_workspace_bytes(T, d, r, &v_off, &xs_off);
    if (!ws || !aligned16(ws)) return api_fail(MOE_ERR_INVALID_ARG, "%s: workspace null or unaligned", who);
    if (ws_bytes < need) return api_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu required", who, ws_bytes, need);
    moe::LoraArgs a = {};
    a.x = x; a.x_scale = x_scale; a.w = w; a.w_scale = w_scale;
    a.la = static_cast<const __nv_bfloat16*>(lora_a); a.lb = static_cast<const __nv_bfloat16*>(lora_b);
    a.ls = lora_scale; a.adapter = adapter; a.y = y;
    a.x_ld = x_ld; a.w_ld = w_ld; a.y_ld = y_ld;
    a.x_dt = x_dtype; a.y_dt = y_dtype; a.T = T; a.d = d; a.N = N; a.na = n_adapters; a.r = r;
    a.status = static_cast<int32_t*>(ws);
    a.v = reinterpret_cast<float*>(static_cast<char*>(ws) + v_off);
    a.vt = nullptr;
    a.xs = reinterpret_cast<__nv_bfloat16*>(static_cast<char*>(ws) + xs_off);
    return launched(moe::launch_lora_project(a, as_stream(stream)), who);
}

}  // extern "C"
