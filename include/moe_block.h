/*
 * moe_block.h -- C ABI of the operators around the MoE layer in a decode block
 * (GB300, sm_103a): the norm before a layer, the paged key-value cache and the
 * attention that reads it, and projections with low-rank adapters.
 *
 *   h   = moe_rmsnorm(x)
 *   qkv = moe_lora_project(h)
 *   moe_kv_append(q, k, v)              rotate, write the new tokens' cache rows
 *   a   = moe_attn_decode(q, cache)     one new token per request
 *   o   = moe_lora_project(a)
 *   h   = moe_rmsnorm(o, residual x)    x += o
 *   y   = moe_layer_forward(h) ...      (moe_decode.h)
 *
 * Conventions are those of moe_decode.h: device pointers owned by the caller,
 * asynchronous on the given stream, no allocation, capturable in a CUDA graph,
 * MOE_OK or a negative MOE_ERR_* code with a message in moe_last_error(), and
 * nothing launched when a host-side check fails.  Beyond them:
 *   - Types are MOE_DTYPE_F32, MOE_DTYPE_BF16 and, where a call says so,
 *     MOE_DTYPE_FP8_E4M3.  All arithmetic is fp32; a result is rounded once.
 *   - Strides are in elements and may be any that keep each row's elements
 *     next to one another; `ld` is the stride between rows.
 *   - The kernels launch as programmatic dependents of the kernel before them
 *     on the stream.  Before that kernel has completed they read the
 *     projection's w and nothing else.  The rule of moe_decode.h on router
 *     weights holds for it too.
 *   - Sizes count from 0 where a call says so: an empty batch is MOE_OK and
 *     launches nothing.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------- */
/* Root-mean-square norm with the residual's addition                        */
/* ------------------------------------------------------------------------- */

/*
 * For each row t of T >= 0:
 *   z = x[t] + residual[t]              (z = x[t] without a residual)
 *   residual_out[t] = z                 (where given; may be residual or x)
 *   y[t] = z / sqrt(mean(z^2) + eps) * weight
 * The norm is that of z in fp32, not of the rounded residual_out.
 *   x             [T, d] F32 or BF16, row stride x_ld
 *   residual      [T, d] or NULL; residual_out [T, d] or NULL, both of
 *                 residual_dtype (F32 or BF16)
 *   weight        [d] F32 or BF16, or NULL for ones
 *   y             [T, d]: F32 or BF16 (y_scale is then NULL), or E4M3 codes
 *   y_scale       float[T] (group 0) or float[T, d / group] (group 128), rows
 *                 packed: amax / 448 of the row (of each 128 columns), 1 where
 *                 that is 0 in fp32; a code is y / scale rounded to E4M3
 * Limits: d a multiple of 8 in [8, 32768]; group 0 or 128 (d % 128 == 0);
 * pointers 16-byte aligned and row strides multiples of 8.
 * y may not overlap the inputs unless it is x (or residual) itself, of the
 * same type and stride.
 */
int moe_rmsnorm(const void* x, int x_dtype, int64_t x_ld, const void* residual, int residual_dtype,
                int64_t residual_ld, void* residual_out, int64_t residual_out_ld, const void* weight,
                int weight_dtype, float eps, int T, int d, void* y, int y_dtype, int64_t y_ld,
                float* y_scale, int group, void* stream);

/* ------------------------------------------------------------------------- */
/* Paged key-value cache                                                     */
/* ------------------------------------------------------------------------- */

/*
 * One layer's cache (host struct).  Slot `i` of page `p` holds, for each
 * key-value head h, D = head_dim key values at
 *   k + p * k_page_stride + i * k_slot_stride + h * k_head_stride
 * and the same for v.  BF16, or E4M3 with one fp32 scale per head (a value is
 * scale[h] * e4m3(code)); k_scale and v_scale are NULL for BF16.
 * Limits: head_dim a multiple of 8 (16 for E4M3) up to 256; pages of any size
 * >= 1; k and v 16-byte aligned, strides multiples of 16 bytes; scales positive,
 * from 2^-126 to 2^126.
 */
typedef struct moe_kv_cache {
    void* k;
    void* v;
    const float* k_scale; /* float[heads] */
    const float* v_scale;
    int64_t k_page_stride, k_slot_stride, k_head_stride;
    int64_t v_page_stride, v_slot_stride, v_head_stride;
    int dtype; /* MOE_DTYPE_BF16 or MOE_DTYPE_FP8_E4M3 */
    int num_pages, page_size, heads, head_dim;
} moe_kv_cache;

/*
 * Write T >= 0 new tokens into the cache, rotating q and k by position.
 * Token t has position p = positions[t] in request req[t] (request t where req
 * is NULL) and goes to slot p % page_size of page block_table[req][p / page_size].
 *   k, v        [T, heads, D] F32 or BF16 (in_dtype), strides between tokens
 *               and heads
 *   q           [T, q_heads, D] of in_dtype or NULL; q_out gets the rotated q
 *               (may be q itself)
 *   cos_sin     float[max_pos, rot]: row p holds cos(p f_i) for i < rot / 2,
 *               then sin(p f_i); element i < rot / 2 of a head is paired with
 *               element i + rot / 2, elements from rot on are copied.  NULL
 *               (with rot = 0): no rotation.
 *   block_table int32[R, max_pages], row stride table_ld
 *   status      int32[1] or NULL: receives MOE_ERR_DEVICE if a token was
 *               dropped, and is left alone otherwise
 * A token of negative position is padding: nothing is written for it but a
 * copy of its q.  A token whose request is outside [0, R), whose position has no
 * page in the table or no row in cos_sin, or whose page is outside the cache
 * is dropped (status).  Two tokens of one slot: its row may mix theirs.
 * Limits: rot even, 0 <= rot <= D.
 */
int moe_kv_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                  int64_t v_token_stride, int64_t v_head_stride, int in_dtype, int T,
                  const moe_kv_cache* cache, const int32_t* block_table, int64_t table_ld, int R,
                  int max_pages, const int32_t* positions, const int32_t* req, const float* cos_sin,
                  int rot, int max_pos, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                  void* q_out, int64_t qo_token_stride, int64_t qo_head_stride, int q_heads,
                  int32_t* status, void* stream);

/* Workspace bytes of moe_attn_decode for up to B requests (0: bad sizes).  Zero
 * it once with moe_workspace_init; one workspace serves any number of calls, one
 * after another, of the same q_heads, heads and head_dim.  Its status word is
 * read with moe_read_status (MOE_ERR_DEVICE: a length beyond the block table, or
 * a page outside the cache; such keys are left out), and stays until the workspace
 * is zeroed again. */
size_t moe_attn_workspace_bytes(int B, int q_heads, int heads, int head_dim);

/*
 * Attention of one new token per request over its cached keys and values:
 *   o[b, h] = sum_j softmax_j(f(scale q[b, h] . k[j, g])) v[j, g],
 * g = h / (q_heads / heads), over the slots j of request b with
 * max(0, n - window) <= j < n, n = seq_lens[b] (the new token included; append
 * it first); window 0 means all.  f(s) = softcap * tanh(s / softcap), or s for
 * softcap 0.  A request with n <= 0 gets zeros, and a score of -inf weighs
 * nothing (a head whose scores all are -inf gets zeros too).  Slots outside that range and
 * table entries of pages wholly outside it are not read.
 * Over an E4M3 cache a head with an infinity in a BF16 q gets NaN (a BF16 out and softcap <= 256).
 *   q           [B, q_heads, D] F32 or BF16; out the same shape, F32 or BF16
 *   block_table int32[B, max_pages], row stride table_ld
 *   lse         float[B, q_heads] or NULL: log of the sum of exp of the scores
 *               (-inf for an empty request)
 * The keys of all requests are shared out evenly over the GPU whatever their
 * lengths; the parts of a request are joined in a fixed order, so that equal
 * calls give equal bits.
 * Limits: heads divides q_heads; q, out 16-byte aligned, strides multiples of 8;
 * B >= 0.
 */
int moe_attn_decode(const void* q, int q_dtype, int64_t q_batch_stride, int64_t q_head_stride, int B,
                    int q_heads, const moe_kv_cache* cache, const int32_t* block_table,
                    int64_t table_ld, int max_pages, const int32_t* seq_lens, float scale, int window,
                    float softcap, void* out, int out_dtype, int64_t out_batch_stride,
                    int64_t out_head_stride, float* lse, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------- */
/* Shared projection with low-rank adapters                                  */
/* ------------------------------------------------------------------------- */

/* Workspace bytes of moe_lora_project for up to T tokens (0: bad sizes).  Zero it
 * once with moe_workspace_init.  Status (moe_read_status): MOE_ERR_DEVICE for an
 * adapter index >= n_adapters (its token gets the shared projection alone),
 * MOE_ERR_TIMEOUT for a wait that ran out. */
size_t moe_lora_workspace_bytes(int T, int d, int r);

/*
 *   y[t] = W x[t] + lora_scale[a] B_a (A_a x[t]),   a = adapter[t]
 * (the second term only where a >= 0), for 0 <= T <= 128 tokens.
 *   x          [T, d] row stride x_ld: F32 or BF16 with BF16 w, or E4M3 codes
 *              with x_scale float[T], E4M3 w and w_scale float[N]
 *   w          [N, d] row stride w_ld
 *   lora_a     BF16 [n_adapters, r, d] or NULL (no adapters: r = 0)
 *   lora_b     BF16 [n_adapters, N, r]
 *   lora_scale float[n_adapters]
 *   adapter    int32[T]
 *   y          [T, N] F32 or BF16, row stride y_ld
 * F32 activations enter the tensor cores as three bf16 terms (exact to 2^-24);
 * so does v = lora_scale A_a x[t] in the second product.
 * Limits: d a multiple of 8 (16 for E4M3) up to 32768, N of 8, r of 8 up to 128,
 * n_adapters * N < 2^31;
 * pointers 16-byte aligned, row strides of x and w multiples of 16 bytes.
 */
int moe_lora_project(const void* x, int x_dtype, int64_t x_ld, const float* x_scale, int T, int d,
                     const void* w, int w_dtype, int64_t w_ld, const float* w_scale, int N,
                     const void* lora_a, const void* lora_b, const float* lora_scale, int n_adapters,
                     int r, const int32_t* adapter, void* y, int y_dtype, int64_t y_ld, void* ws,
                     size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif
