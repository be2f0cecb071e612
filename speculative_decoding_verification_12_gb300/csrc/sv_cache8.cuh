// sv_cache8.cuh -- the cache in 8 bits: its addressing, its scales and the checks of its arguments.
#pragma once

#include <cuda_fp8.h>
#include <math.h>

#include "sv_cache.cuh"

namespace svc {

struct Cache8 {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride, token_stride, head_stride;         // bytes
    int64_t s_page, s_block, s_head;                        // floats
    const int32_t *table;
    int num_pages, page_shift, block_shift, heads, D, max_pages;
};

constexpr float TOP8 = 448.f;                               // the largest e4m3 number
constexpr float LEAST_SCALE = 0x1p-40f, MOST_SCALE = 0x1p40f;

// A stored scale as it counts (not a number: the least one).
__device__ __forceinline__ float clean_scale(float s) { return fminf(fmaxf(s, LEAST_SCALE), MOST_SCALE); }

// The least power of two s in [LEAST_SCALE, MOST_SCALE] with amax <= 448 s, for a finite amax >= 0:
// 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int k = (int)(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x600000u ? 8 : 7);
    return __uint_as_float((uint32_t)(min(max(k, -40), 40) + 127) << 23);
}

// x / s and x f, cut off, and with the last bit set where anything was: what is rounded from there to a few bits is
// rounded once, from the exact value (the nearest fp32 number may be a tie of e4m3's that x / s is not).
__device__ __forceinline__ float over_odd(float x, float s) {
    const float q = __fdiv_rz(x, s);
    return fmaf(-q, s, x) != 0.f ? __uint_as_float(__float_as_uint(q) | 1u) : q;   // (the rest is exact)
}
__device__ __forceinline__ float times_odd(float x, float f) {
    const float p = __fmul_rz(x, f);
    return fmaf(x, f, -p) != 0.f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
}

// Two numbers as e4m3, nearest (ties to even), magnitudes above 448 as 448, not a number as NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 unpack_e4m3(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return __half22float2(__half2(h));
}

// --- host side ---

// check_batch for a cache in 8 bits: queries of `dtype`.
inline sv_status check_batch8(const int32_t *num_drafts, const int32_t *row_offsets, const int32_t *kv_seq_len,
                              int32_t B, int32_t k_max, int32_t total_rows, int32_t num_q_heads, sv_dtype dtype,
                              const sv_kv_cache8 &c, Batch &batch, Cache8 &cache) {
    sv_kv_cache as16{c.k, c.v, c.page_stride, c.token_stride, c.head_stride, c.num_pages, c.page_size, c.num_heads,
                     c.head_dim, dtype, c.max_pages, c.block_table};
    Cache ignored;
    const sv_status bad = check_batch(num_drafts, row_offsets, kv_seq_len, B, k_max, total_rows, num_q_heads, as16, 128,
                                      batch, ignored);
    if (bad != SV_OK) return bad;
    if (!c.k_scale || !c.v_scale || c.scale_page_stride <= 0 || c.scale_block_stride <= 0 || c.scale_head_stride <= 0)
        return SV_ERR_INVALID_ARG;
    if (c.head_dim % 16 || c.page_stride % 16 || c.token_stride % 16 || c.head_stride % 16) return SV_ERR_UNSUPPORTED;
    if (c.scale_tokens < 8 || c.scale_tokens > c.page_size || (c.scale_tokens & (c.scale_tokens - 1)))
        return SV_ERR_UNSUPPORTED;
    if (((uintptr_t)c.k_scale & 3) || ((uintptr_t)c.v_scale & 3)) return SV_ERR_UNSUPPORTED;
    if ((c.scale_page_stride | c.scale_block_stride | c.scale_head_stride) >> 38) return SV_ERR_UNSUPPORTED;
    cache = Cache8{static_cast<uint8_t *>(c.k), static_cast<uint8_t *>(c.v), c.k_scale, c.v_scale,
                   c.page_stride, c.token_stride, c.head_stride, c.scale_page_stride, c.scale_block_stride,
                   c.scale_head_stride, c.block_table, c.num_pages, ignored.page_shift,
                   __builtin_ctz((unsigned)c.scale_tokens), c.num_heads, c.head_dim, c.max_pages};
    return SV_OK;
}

}  // namespace svc
