// What the two appends to the paged cache share.
#pragma once

#include <climits>

#include "block.h"

namespace moe {

namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendSmem = 112 * 1024;     // two blocks per SM

// inv: 1 / scale of E4M3 rows (a code is the value times it, within 1 ulp of value / scale).
template <int VEC>
__device__ __forceinline__ void store_vec(void* p, int dt, long long i, const float (&f)[VEC], float inv) {
    if (dt == MOE_DTYPE_FP8_E4M3) {
        uint8_t* b = static_cast<uint8_t*>(p) + i;
        if constexpr (VEC == 8) {
            *reinterpret_cast<uint2*>(b) = make_uint2(pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                                                      pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
        } else if constexpr (VEC == 4) {
            *reinterpret_cast<uint32_t*>(b) = pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
        } else {
            b[0] = (uint8_t)__nv_cvt_float_to_fp8(f[0] * inv, __NV_SATFINITE, __NV_E4M3);
        }
    } else if constexpr (VEC == 8) {
        store8(p, dt, i, f);
    } else if constexpr (VEC == 4) {
        if (dt == MOE_DTYPE_BF16)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        if (dt == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f[0]);
        else static_cast<float*>(p)[i] = f[0];
    }
}

// What a thread has of every head it takes: elements [i0, + VEC) and (two) [i1, + VEC), turned
// into one another (turn) or left alone.
template <int VEC>
struct Item {
    int i0, i1;
    bool two, turn;
    alignas(16) float cs[VEC], sn[VEC];
    // item i of a head of D elements, whose first 2 half turn
    __device__ __forceinline__ void place(int i, int D, int half) {
        const int pairs = half / VEC, plain = (D - 2 * half) / VEC;
        turn = i < pairs;
        if (turn) {
            i0 = i * VEC;
            i1 = i0 + half;
            two = true;
        } else {
            const int k = i - pairs, k1 = k + (plain + 1) / 2;
            i0 = 2 * half + k * VEC;
            i1 = 2 * half + k1 * VEC;
            two = k1 < plain;
        }
    }
    __device__ __forceinline__ void rotate(float (&x)[VEC], float (&y)[VEC]) const {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float f = x[e], g = y[e];
            x[e] = f * cs[e] - g * sn[e];
            y[e] = g * cs[e] + f * sn[e];
        }
    }
};

// The request's page of a position as the table has it, which may not be one of the pool; -1: none.
// last: the last position that has one.
__device__ __forceinline__ int page_of(const AppendArgs& a, int req, int pos, int last) {
    const int col = pos / a.c.page_size;
    return pos < 0 || req < 0 || req >= a.R || col >= a.max_pages || pos > last ? -1 : a.table[req * a.table_ld + col];
}

}  // namespace

}  // namespace moe
