// cache_append.cu -- spec_append: per-head norm and rotation of the new tokens' queries and keys
// and the append of keys and values to the paged cache.
//
// Mathematics: y = x * rsqrt(mean(x^2) + eps) * w; each pair (a, z) of y turns by the angle
// t * inv_freq[j].  The angle in turns is the exact product of the position t and inv_freq / 2 pi
// modulo 1, kept as a 64-bit binary fraction: inv_freq = m 2^e, so m * round(2^64 / 2 pi) shifted
// by e is inv_freq / 2 pi within 2^-64 (plus the shift's own truncation), and its product with t,
// wrapping at 2^64, is the fraction of a turn within t * 2^-63.  Only then does it become a float
// (24 bits of a half turn), so the rotation is as exact at position 10^6 as at 0.
#include <math.h>

#include "sv_cache.cuh"
#include "sv_rotate.cuh"
#include "sv_tc.cuh"

namespace svc {

struct AppendArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, out_stride;
    const void *qw, *kw;
    const float *inv_freq;
    void *out;
    int32_t *hdr;
    float eps, rope_scale;
    int Hq, half, interleaved;
};

constexpr int AT = 256;   // threads per CTA
constexpr int AU = 3;     // heads per thread and pass, all loaded before the first is used (4: 9.4 us, 2: 9.9)
constexpr int OCC = 3;    // CTAs per SM (2: 10.4 us; 4 spill: 12.5)
constexpr int ROWS = 16;  // rows per CTA at most: 16 KB of rotations

// Each CTA takes a few rows in a row.  LPH lanes hold one head, 8 elements each (a power of two >=
// head_dim / 8), so a thread's elements are the same in every head it meets, and its weights and
// rotations serve all of them.
//
// What bounds it: latency, in a call that is one wave of CTAs.  A row of 48 heads of 128 is 24 KB in and
// out, 4 ns at the memory's rate, and neither the memory nor the schedulers are full: an instruction is
// issued in 56 % of the cycles in which a CTA is resident and in 39 % of the kernel's, 5.3 warps per
// scheduler of which 1.3 could go on, and the others wait for arithmetic results (1.9 of 9.5 cycles per
// instruction), global and shared memory (1.4 and 1.0) and barriers (0.9).  The few rows of a CTA wait once
// for the chain offsets -> length -> page: one warp walks it, a lane per row, while the first row's data,
// the weights and the turns of the frequencies are under way, and all the rows' pairs are then turned at
// once: two barriers in all, and a warp asks for its next row's data before it works on this one's.  1280
// rows of 48 heads take 9.2 us (3.4 TB/s read and written; with the rotations per row behind a barrier
// each 10.4, and with one fp32 operation per instruction 10.9); one row takes 3.5 us, the launch.
// Background copies of the next rows to shared memory: 12.0 before those two steps, no gain; a row's
// addresses kept per thread and stepped instead of made anew: 9.5.
template <typename E, int LPH, int PAIR>
__global__ void __launch_bounds__(AT, OCC) append_kernel(const Batch A, const Cache C, const AppendArgs P, int per_cta) {
    __shared__ float2 turn[ROWS][128];   // (cos, sin) * rope_scale of each row's pairs
    __shared__ float ex[PAIR == PAIR_ANY ? AT * 8 : 1];
    __shared__ int64_t slot[ROWS];    // the tokens' offsets in the cache
    __shared__ int state[ROWS], pos[ROWS];   // state: 0: unused row, 1: used, 2: in error
    const int tid = threadIdx.x, lane = tid & 31;
    const int first = blockIdx.x * per_cta, rows = min(per_cta, A.R - first);
    const int D = C.D, Hq = P.Hq, Hk = C.heads, heads = Hq + 2 * Hk, max_tokens = C.max_pages << C.page_shift;
    constexpr int HPC = AT / LPH;     // heads per CTA and step
    const int sub = tid % LPH, h_first = tid / LPH;
    const int rot = 2 * P.half;
    const float inv_d = 1.f / (float)D;
    // one weight alone: a warp then holds heads with and without a norm
    const bool q_alone = P.kw == nullptr, one_alone = q_alone != (P.qw == nullptr);
    // this thread's elements: [d0, d0 + 4) and [d1, d1 + 4)
    const bool turns = PAIR == PAIR_HALVES ? sub * 4 < P.half : sub * 8 < rot;
    const int d0 = PAIR != PAIR_HALVES ? sub * 8 : turns ? sub * 4 : rot + (sub - P.half / 4) * 8;
    const int d1 = (PAIR == PAIR_HALVES && turns ? P.half + sub * 4 : d0 + 4) - d0;   // (from d0)
    const bool in = sub * 8 < D;
    auto take = [&](const E *at) {
        if (PAIR != PAIR_HALVES) return *reinterpret_cast<const uint4 *>(at);
        const uint2 a = *reinterpret_cast<const uint2 *>(at), b = *reinterpret_cast<const uint2 *>(at + d1);
        return make_uint4(a.x, a.y, b.x, b.y);
    };
    auto put = [&](E *at, uint4 w) {
        if (PAIR != PAIR_HALVES) {
            *reinterpret_cast<uint4 *>(at) = w;
        } else {
            *reinterpret_cast<uint2 *>(at) = make_uint2(w.x, w.y);
            *reinterpret_cast<uint2 *>(at + d1) = make_uint2(w.z, w.w);
        }
    };

    grid_wait();
    grid_launch_dependents();
    constexpr uint32_t ONE2 = Num<E>::ONE2;
    uint4 raw[AU], qw = make_uint4(ONE2, ONE2, ONE2, ONE2), kw = qw;   // (no weight: ones)
    // Row i's elements of head h.
    auto source = [&](int h, int i) {
        const int64_t r = first + i;
        if (h >= Hq + Hk) return static_cast<const E *>(P.v) + r * P.v_stride + ((h - Hq - Hk) * D + d0);
        if (h >= Hq) return static_cast<const E *>(P.k) + r * P.k_stride + ((h - Hq) * D + d0);
        return static_cast<const E *>(P.q) + r * P.q_stride + (h * D + d0);
    };
    auto begin = [&](int h0) {
#pragma unroll
        for (int u = 0; u < AU; u++) {
            const int h = h0 + u * HPC + h_first;
            raw[u] = make_uint4(0u, 0u, 0u, 0u);
            if (in && h < heads) raw[u] = take(source(h, 0));
        }
    };
    begin(0);
    const int hp = P.half > 64 ? 128 : P.half > 32 ? 64 : 32;   // threads per row for the turns
    const int pair = tid & (hp - 1);
    const float f = pair < P.half ? P.inv_freq[pair] : 0.f;
    if (in && P.qw) qw = take(static_cast<const E *>(P.qw) + d0);
    if (in && P.kw) kw = take(static_cast<const E *>(P.kw) + d0);
    if (tid >= AT - 32) {
        const int r = first + lane;
        const int b = request_of_rows(A, first, rows);   // (each lane its row's)
        int st = 0, p = 0, page = -1;
        if (lane < rows && b >= 0) {
            const Span s = span_of(A, max_tokens, b);
            if (s.err) st = 2;
            else if (r >= s.row0 && r - s.row0 < s.n) {
                st = 1;
                p = s.len - s.n + (r - s.row0);
                page = C.table[(int64_t)b * C.max_pages + (p >> C.page_shift)];
                if (page < 0 || page >= C.num_pages) {
                    record_error(P.hdr, SV_DEV_BAD_PAGE, b);
                    st = 2;
                }
            }
        }
        if (lane < rows) {
            state[lane] = st;
            pos[lane] = p;
            slot[lane] = page * C.page_stride + (p & ((1 << C.page_shift) - 1)) * C.token_stride;
        }
    } else if (tid >= AT - 64) {
        check_requests(A, max_tokens, P.hdr, blockIdx.x * 32 + lane, gridDim.x * 32);
    }
    const uint64_t t = turns_of(f);
    __syncthreads();
    if (pair < P.half)
        for (int i = tid / hp; i < rows; i += AT / hp) {
            float sn, cs;
            sincospif((float)(int32_t)(uint32_t)(t * (uint64_t)(uint32_t)pos[i] >> 32) * 0x1p-31f, &sn, &cs);
            if (!(fabsf(f) < INFINITY)) sn = cs = NAN;
            turn[i][pair] = make_float2(cs * P.rope_scale, sn * P.rope_scale);
        }
    __syncthreads();

#pragma unroll 1
    for (int h0 = 0; h0 < heads; h0 += AU * HPC) {
        if (h0) begin(h0);
#pragma unroll 1
        for (int i = 0; i < rows; i++) {
            const int st = state[i];
            const int64_t at_q = (first + i) * P.out_stride, at_kv = slot[i];
            // this thread's rotations: of its four pairs, or (any distance) of its eight elements
            constexpr int NR = PAIR == PAIR_ANY ? 8 : 4;
            float2 cs[NR];
#pragma unroll
            for (int e = 0; e < NR; e++) {
                const int j = PAIR != PAIR_ANY ? sub * 4 + e : d0 + e < P.half ? d0 + e : d0 + e - P.half;
                const bool on = PAIR == PAIR_ANY ? d0 + e < rot : j < P.half;
                cs[e] = on ? turn[i][j] : make_float2(1.f, 0.f);
            }
#pragma unroll
            for (int u = 0; u < AU; u++) {
                const int h = h0 + u * HPC + h_first;
                if (h0 + u * HPC >= heads) break;   // (the whole CTA)
                const bool is_v = h >= Hq + Hk, is_k = h >= Hq, on = in && h < heads;
                const uint4 mine = raw[u];
                if (on && i + 1 < rows) raw[u] = take(source(h, i + 1));
                E *to = is_v   ? static_cast<E *>(C.v) + at_kv + (h - Hq - Hk) * C.head_stride + d0
                        : is_k ? static_cast<E *>(C.k) + at_kv + (h - Hq) * C.head_stride + d0
                               : static_cast<E *>(P.out) + at_q + (h * D + d0);
                if (st != 1) {
                    const uint32_t w = st == 2 ? Num<E>::NAN2 : 0u;
                    if (on && !is_k) put(to, make_uint4(w, w, w, w));
                    continue;
                }
                if (h0 + u * HPC + (tid & ~31) / LPH >= Hq + Hk) {   // (the whole warp)
                    if (on) put(to, mine);
                    continue;
                }
                float2 x[4];
                unpack8<E>(mine, reinterpret_cast<float *>(x));
                if (P.qw || P.kw) {   // (the whole grid, so that a warp's shuffles are together)
                    float2 s2 = make_float2(0.f, 0.f), g[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) s2 = fma2(x[e], x[e], s2);
                    float ss = s2.x + s2.y;
#pragma unroll
                    for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    unpack8<E>(is_k ? kw : qw, reinterpret_cast<float *>(g));
                    float inv = rsqrtf(fmaf(ss, inv_d, P.eps));
                    if (one_alone && is_k == q_alone) inv = 1.f;   // (and its weights are ones)
#pragma unroll
                    for (int e = 0; e < 4; e++) x[e] = mul2(mul2(x[e], make_float2(inv, inv)), g[e]);
                }
                if (PAIR == PAIR_ANY) {
                    float2 *own = reinterpret_cast<float2 *>(ex + (tid - sub) * 8);
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 4; e++) own[sub * 4 + e] = x[e];
                    __syncwarp();
                    const float *all = ex + (tid - sub) * 8;
                    float *y = reinterpret_cast<float *>(x);
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int d = d0 + e;
                        if (d < P.half) y[e] = y[e] * cs[e % NR].x - all[d + P.half] * cs[e % NR].y;
                        else if (d < rot) y[e] = y[e] * cs[e % NR].x + all[d - P.half] * cs[e % NR].y;
                    }
                } else if (PAIR == PAIR_NEXT) {
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float2 c = cs[e % NR];
                        x[e] = fma2(x[e], make_float2(c.x, c.x), mul2(make_float2(x[e].y, x[e].x), make_float2(-c.y, c.y)));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const float2 a = x[e], z = x[e + 2], c = make_float2(cs[2 * e].x, cs[2 * e + 1].x),
                                     n = make_float2(cs[2 * e].y, cs[2 * e + 1].y);
                        x[e] = fma2(a, c, mul2(z, make_float2(-n.x, -n.y)));
                        x[e + 2] = fma2(z, c, mul2(a, n));
                    }
                }
                if (on) put(to, is_v ? mine : pack8<E>(reinterpret_cast<const float *>(x)));
            }
        }
    }
}

template <typename E, int LPH>
static cudaError_t launch_heads(const Batch &A, const Cache &C, const AppendArgs &P, cudaStream_t st) {
    int dev = 0, nsm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // one wave of resident CTAs where the rows allow
    int per = (A.R + OCC * nsm - 1) / (OCC * nsm);
    if (per > ROWS) per = ROWS;
    const int grid = (A.R + per - 1) / per;
    auto *const kernel = P.interleaved || P.half == 0 ? append_kernel<E, LPH, PAIR_NEXT>
                         : P.half % 4 == 0            ? append_kernel<E, LPH, PAIR_HALVES>
                                                      : append_kernel<E, LPH, PAIR_ANY>;
    return launch_dependent(kernel, dim3(grid), dim3(AT), 1, st, A, C, P, per);
}
template <typename E>
static cudaError_t launch_append(const Batch &A, const Cache &C, const AppendArgs &P, cudaStream_t st) {
    const int lanes = C.D / 8;
    return lanes <= 8 ? launch_heads<E, 8>(A, C, P, st) : lanes <= 16 ? launch_heads<E, 16>(A, C, P, st)
                                                                      : launch_heads<E, 32>(A, C, P, st);
}

}  // namespace svc

using namespace svc;

extern "C" sv_status spec_append(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                                 int64_t v_stride, int32_t num_q_heads, const void *q_weight, const void *k_weight,
                                 float eps, const float *inv_freq, int32_t rotary_dim, int32_t interleaved,
                                 float rope_scale, const int32_t *num_drafts, const int32_t *row_offsets,
                                 const int32_t *kv_seq_len, int32_t B, int32_t k_max, int32_t total_rows,
                                 sv_kv_cache cache, void *out_q, int64_t out_q_stride, void *workspace,
                                 void *stream) {
    Batch A;
    Cache C;
    const sv_status bad = check_batch(num_drafts, row_offsets, kv_seq_len, B, k_max, total_rows, num_q_heads, cache,
                                      256, A, C);
    if (bad != SV_OK) return bad;
    if (!q || !k || !v || !out_q || !workspace) return SV_ERR_INVALID_ARG;
    if (rotary_dim < 0 || rotary_dim % 2 || rotary_dim > cache.head_dim || (rotary_dim && !inv_freq))
        return SV_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !(eps < INFINITY) || !(fabsf(rope_scale) < INFINITY)) return SV_ERR_INVALID_ARG;
    const int64_t qw = (int64_t)num_q_heads * cache.head_dim, kw = (int64_t)cache.num_heads * cache.head_dim;
    if (q_stride < qw || out_q_stride < qw || k_stride < kw || v_stride < kw) return SV_ERR_INVALID_ARG;
    if ((q_stride | k_stride | v_stride | out_q_stride) % 8 || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
        !aligned16(out_q) || !aligned16(q_weight) || !aligned16(k_weight))
        return SV_ERR_UNSUPPORTED;
    if ((uintptr_t)workspace & 255) return SV_ERR_WORKSPACE;
    const AppendArgs P{q, k, v, q_stride, k_stride, v_stride, out_q_stride, q_weight, k_weight, inv_freq, out_q,
                       static_cast<int32_t *>(workspace), eps, rope_scale, num_q_heads, rotary_dim / 2, interleaved};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cache.dtype == SV_BF16 ? launch_append<__nv_bfloat16>(A, C, P, st)
                                                 : launch_append<__half>(A, C, P, st);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
