// cache_append8.cu -- spec_append8: per-head norm and rotation of the new tokens' queries and keys, and
// the append of keys and values to a paged cache of e4m3 numbers with a scale per block of tokens and head.
//
// Mathematics: norm and rotation as in cache_append.cu.  A block's scale s is the least power of two that
// holds its new elements, or the one it has where it holds older tokens and has a larger one; stored is
// RN(x / s).  With powers of two, x / s only shifts the exponent, so rewriting older tokens in a grown
// scale rounds nothing but what falls into e4m3's subnormal numbers: a block that grows with every
// token is as exact as one that was written at once.  (A kept scale that is no power of two divides, and is
// rewritten by a product, both rounded to odd first: see over_odd.)  The largest magnitude has to be known before the first
// element is rounded, so the new tokens of a block and head belong to one warp.
//
// Work.  One or more CTAs per request.  A warp takes a task at a time: the new tokens of one block of one key
// or value head (LPH lanes a token, so 2 or 4 tokens side by side, up to 4 such steps kept in registers
// between the maximum and the rounding, more are computed twice), or 2 or 4 query heads of a row.
//
// What bounds it: loads that a task begins with and waits for, with 16 warps a multiprocessor to cover them.  256 x 5 rows of
// 32 + 2 x 8 heads of 128 take 15.9 us in a graph (19.0 with inputs that are not in L2; 28 MB, 4.2 us at the memory's
// rate), where a request is 30 200 warp instructions and a CTA's chain is offsets -> length -> page -> rotations -> tasks;
// the schedulers issue in 36 % of the cycles.  append_kernel, whose threads keep their elements' weights and rotations
// over all heads, does the same rows in 16 bits in 9.3 us: queries need not be tasks of these warps, and 4096 x 1 rows (89.8 us
// for 26.4) show it most.  One row takes 4.3 us, the launch.  Integer divisions between
// tasks, and one per pair of the rotations, were a tenth of the instructions (17.7 us).  Asking for the next task's elements
// before this one's are worked on: 19.7, the registers then leave fewer CTAs; 8 warps a CTA: 16.9.
#include "sv_cache8.cuh"
#include "sv_rotate.cuh"
#include "sv_tc.cuh"

namespace svc {

struct Append8Args {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, out_stride;
    const void *qw, *kw;
    const float *inv_freq;
    void *out;
    int32_t *hdr;
    float eps, rope_scale;
    int Hq, half, interleaved;
    int split;   // CTAs per request
};

constexpr int AT8 = 128;         // threads per CTA (256 x 5 rows of 48 heads: 15.6 us, 16.9 with 256)
constexpr int STEPS = 4;         // steps of a task whose elements stay in registers

template <typename E, int LPH, int PAIR>
__global__ void __launch_bounds__(AT8) append8_kernel(const Batch A, const Cache8 C, const Append8Args P) {
    __shared__ float2 turn[MAXK + 1][64];   // (cos, sin) * rope_scale of each row's pairs
    __shared__ float ex[PAIR == PAIR_ANY ? AT8 * 8 : 1];
    __shared__ int page_of[MAXK + 1];       // each row's page, or -1
    constexpr int HPW = 32 / LPH;           // heads, or tokens, of a warp side by side
    const int tid = threadIdx.x, lane = tid & 31, sub = lane % LPH, team = lane / LPH;
    const int b = blockIdx.x / P.split, part = blockIdx.x - b * P.split;
    const int D = C.D, Hq = P.Hq, Hk = C.heads, max_tokens = C.max_pages << C.page_shift;
    const int rot = 2 * P.half;
    const float inv_d = 1.f / (float)D;
    // this thread's elements of a head: [d0, d0 + 4) and [d1, d1 + 4), as in append_kernel
    const bool turns = PAIR == PAIR_HALVES ? sub * 4 < P.half : sub * 8 < rot;
    const int d0 = PAIR != PAIR_HALVES ? sub * 8 : turns ? sub * 4 : rot + (sub - P.half / 4) * 8;
    const int d1 = PAIR == PAIR_HALVES && turns ? P.half + sub * 4 : d0 + 4;
    const bool in = sub * 8 < D;
    auto take = [&](const E *head) {
        if (PAIR != PAIR_HALVES) return *reinterpret_cast<const uint4 *>(head + d0);
        const uint2 a = *reinterpret_cast<const uint2 *>(head + d0), z = *reinterpret_cast<const uint2 *>(head + d1);
        return make_uint4(a.x, a.y, z.x, z.y);
    };

    grid_wait();
    grid_launch_dependents();
    const Span s = span_of(A, max_tokens, b);
    const int n = s.n, pos0 = s.len - n;

    // rows of this request that it does not use, and, at both ends, those of no request
    {
        int from = s.row0 + n, to = A.row_off ? A.row_off[b + 1] : s.row0 + A.k_max + 1;
        if (from < 0 || to > A.R || to < from) from = to = 0;
        const int head = A.row_off && b == 0 ? min(max(s.row0, 0), A.R) : 0;
        const int tail = A.row_off && b == A.B - 1 ? min(max(A.row_off[b + 1], 0), A.R) : A.R;
        const int per = Hq * D / 8;
        auto fill = [&](int r0, int r1, uint32_t w) {
            for (int64_t i = part * AT8 + tid; i < (int64_t)(r1 - r0) * per; i += P.split * AT8) {
                const int64_t r = i / per;
                *reinterpret_cast<uint4 *>(static_cast<E *>(P.out) + (r0 + r) * P.out_stride + (i - r * per) * 8) =
                    make_uint4(w, w, w, w);
            }
        };
        fill(from, to, s.err ? Num<E>::NAN2 : 0u);
        fill(0, head, 0u);
        fill(tail, A.R, 0u);
    }
    if (s.err && part == 0 && tid == 0) record_error(P.hdr, s.err, b);
    if (n == 0) return;

    const int32_t *table = C.table + (int64_t)b * C.max_pages;
    for (int i = tid; i < n; i += AT8) {
        int page = table[(pos0 + i) >> C.page_shift];
        if (page < 0 || page >= C.num_pages) {
            if (part == 0) record_error(P.hdr, SV_DEV_BAD_PAGE, b);
            page = -1;
        }
        page_of[i] = page;
    }
    {
        const int hp = P.half > 32 ? 64 : 32, pair = tid & (hp - 1);   // threads per row
        const float f = pair < P.half ? P.inv_freq[pair] : 0.f;
        const uint64_t turns = turns_of(f);
        if (pair < P.half)
            for (int row = tid / hp; row < n; row += AT8 / hp) {
                float sn, cs;
                sincospif((float)(int32_t)(uint32_t)(turns * (uint64_t)(uint32_t)(pos0 + row) >> 32) * 0x1p-31f, &sn, &cs);
                if (!(fabsf(f) < INFINITY)) sn = cs = NAN;
                turn[row][pair] = make_float2(cs * P.rope_scale, sn * P.rope_scale);
            }
    }
    constexpr uint32_t ONE2 = Num<E>::ONE2;
    uint4 qw = make_uint4(ONE2, ONE2, ONE2, ONE2), kw = qw;   // (no weight: ones)
    if (in && P.qw) qw = take(static_cast<const E *>(P.qw));
    if (in && P.kw) kw = take(static_cast<const E *>(P.kw));
    __syncthreads();

    // A head's 8 elements of this thread, normalised and turned to the position of `row`.  The whole warp.
    auto turned = [&](uint4 raw, uint4 weight, bool norm, int row, float2 x[4]) {
        unpack8<E>(raw, reinterpret_cast<float *>(x));
        if (norm) {
            float2 s2 = make_float2(0.f, 0.f), g[4];
#pragma unroll
            for (int e = 0; e < 4; e++) s2 = fma2(x[e], x[e], s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            unpack8<E>(weight, reinterpret_cast<float *>(g));
            const float inv = rsqrtf(fmaf(ss, inv_d, P.eps));
#pragma unroll
            for (int e = 0; e < 4; e++) x[e] = mul2(mul2(x[e], make_float2(inv, inv)), g[e]);
        }
        if (rot == 0) return;
        const float2 *c = turn[row];
        float *y = reinterpret_cast<float *>(x);
        if (PAIR == PAIR_ANY) {
            float *own = ex + (tid - sub) * 8;
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; e++) own[sub * 8 + e] = y[e];
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const int d = d0 + e;
                if (d < P.half) y[e] = y[e] * c[d].x - own[d + P.half] * c[d].y;
                else if (d < rot) y[e] = y[e] * c[d - P.half].x + own[d - P.half] * c[d - P.half].y;
            }
        } else if (PAIR == PAIR_NEXT) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if (sub * 4 + e >= P.half) break;
                const float2 r = c[sub * 4 + e];
                x[e] = fma2(x[e], make_float2(r.x, r.x), mul2(make_float2(x[e].y, x[e].x), make_float2(-r.y, r.y)));
            }
        } else if (turns) {
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float2 a = x[e], z = x[e + 2], r0 = c[sub * 4 + 2 * e], r1 = c[sub * 4 + 2 * e + 1],
                             cs = make_float2(r0.x, r1.x), sn = make_float2(r0.y, r1.y);
                x[e] = fma2(a, cs, mul2(z, make_float2(-sn.x, -sn.y)));
                x[e + 2] = fma2(z, cs, mul2(a, sn));
            }
        }
    };

    const int warps = P.split * (AT8 / 32), w = part * (AT8 / 32) + (tid >> 5);
    const int block0 = pos0 >> C.block_shift;
    const int blocks = ((s.len - 1) >> C.block_shift) - block0 + 1, stores = 2 * Hk * blocks;
    const int side_step = warps / blocks, block_step = warps - side_step * blocks;   // from a warp's task to its next
    for (int side = w / blocks, block = block0 + w - side * blocks; side < 2 * Hk; side += side_step, block += block_step) {
        if (block >= block0 + blocks) {
            block -= blocks;
            if (++side >= 2 * Hk) break;
        }
        const bool is_v = side >= Hk;
        const int h = is_v ? side - Hk : side;
        const int lo = max(pos0, block << C.block_shift), hi = min(s.len, (block + 1) << C.block_shift), count = hi - lo;
        const int page = page_of[lo - pos0];
        if (page < 0) continue;
        const E *from = static_cast<const E *>(is_v ? P.v : P.k) + (int64_t)h * D;
        const int64_t stride = is_v ? P.v_stride : P.k_stride;
        const int slot0 = (block << C.block_shift) & ((1 << C.page_shift) - 1), older = lo - (block << C.block_shift);
        uint8_t *to = (is_v ? C.v : C.k) + page * C.page_stride + slot0 * C.token_stride + h * C.head_stride;
        float *at = (is_v ? C.v_scale : C.k_scale) + page * C.s_page + (slot0 >> C.block_shift) * C.s_block + h * C.s_head;
        const float had = older ? clean_scale(*at) : 0.f;
        const int batches = (count + STEPS * HPW - 1) / (STEPS * HPW);
        float amax = 0.f, scale = 1.f, inv = 0.f;
        // the elements' maximum, then (again, unless they are all still here) their numbers
        for (int it = 0; it < (batches == 1 ? 1 : 2 * batches); it++) {
            const int i0 = (it < batches ? it : it - batches) * STEPS * HPW + team;
            uint4 raw[STEPS];
            float2 x[STEPS][4];
#pragma unroll
            for (int e = 0; e < STEPS; e++) {
                const int i = i0 + e * HPW;
                raw[e] = make_uint4(0u, 0u, 0u, 0u);
                if (in && i < count) raw[e] = take(from + (int64_t)(s.row0 + lo - pos0 + i) * stride);
            }
#pragma unroll
            for (int e = 0; e < STEPS; e++) {
                if (i0 - team + e * HPW >= count) break;   // (the whole warp)
                if (is_v) unpack8<E>(raw[e], reinterpret_cast<float *>(x[e]));
                else turned(raw[e], kw, P.kw != nullptr, min(lo - pos0 + i0 + e * HPW, n - 1), x[e]);
                const float *y = reinterpret_cast<const float *>(x[e]);
                if (it < batches)
#pragma unroll
                    for (int d = 0; d < 8; d++) amax = fmaxf(amax, in && fabsf(y[d]) < INFINITY ? fabsf(y[d]) : 0.f);
            }
            if (it == batches - 1) {
#pragma unroll
                for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                scale = fmaxf(scale_for(amax), had);
                inv = 1.f / scale;
                if (lane == 0) *at = scale;
                if (scale > had && older) {   // older tokens in the grown scale
                    const float f = had * inv;
                    const int words = D / 4;
                    for (int i = lane; i < older * words; i += 32) {
                        const int t = i / words;
                        uint32_t *p = reinterpret_cast<uint32_t *>(to + t * C.token_stride) + (i - t * words);
                        const uint32_t v = *p;
                        const float2 a = unpack_e4m3(v & 0xffffu), z = unpack_e4m3(v >> 16);
                        *p = pack_e4m3(times_odd(a.x, f), times_odd(a.y, f)) | pack_e4m3(times_odd(z.x, f), times_odd(z.y, f)) << 16;
                    }
                }
            }
            if (it < batches && batches > 1) continue;
            // a power of two shifts; a kept scale that is none (from elsewhere) divides
            const bool shifts = !(__float_as_uint(scale) & 0x7fffffu);
            const float by = shifts ? inv : 1.f;
#pragma unroll
            for (int e = 0; e < STEPS; e++) {
                const int i = i0 + e * HPW;
                if (!in || i >= count) break;
                float *y = reinterpret_cast<float *>(x[e]);
                if (!shifts)
#pragma unroll
                    for (int d = 0; d < 8; d++) y[d] = over_odd(y[d], scale);
                uint32_t two[4];
#pragma unroll
                for (int d = 0; d < 4; d++) {
                    const float a = y[2 * d], z = y[2 * d + 1];
                    two[d] = pack_e4m3(fabsf(a) < INFINITY ? a * by : NAN, fabsf(z) < INFINITY ? z * by : NAN);
                }
                uint8_t *head = to + (older + i) * C.token_stride;
                if (PAIR != PAIR_HALVES) {
                    *reinterpret_cast<uint2 *>(head + d0) = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
                } else {
                    *reinterpret_cast<uint32_t *>(head + d0) = two[0] | two[1] << 16;
                    *reinterpret_cast<uint32_t *>(head + d1) = two[2] | two[3] << 16;
                }
            }
        }
    }

    // queries: after the stores, so that every warp has as many tasks
    const int steps = (Hq + HPW - 1) / HPW, row_step = warps / steps, col_step = warps - row_step * steps;
    const int first = (w + warps - stores % warps) % warps;
    int row = first / steps, col = first - row * steps;   // of this warp's next task
    while (row < n) {
        uint4 raw[STEPS];
        int rows[STEPS], heads[STEPS];
#pragma unroll
        for (int e = 0; e < STEPS; e++) {
            rows[e] = row;
            heads[e] = col * HPW + team;
            raw[e] = make_uint4(0u, 0u, 0u, 0u);
            if (row < n && in && heads[e] < Hq)
                raw[e] = take(static_cast<const E *>(P.q) + (int64_t)(s.row0 + row) * P.q_stride + (int64_t)heads[e] * D);
            row += row_step;
            col += col_step;
            if (col >= steps) col -= steps, row++;
        }
#pragma unroll
        for (int e = 0; e < STEPS; e++) {
            const int row = rows[e], h = heads[e];
            if (row >= n) break;   // (the whole warp)
            float2 x[4];
            turned(raw[e], qw, P.qw != nullptr, row, x);
            uint4 y = pack8<E>(reinterpret_cast<const float *>(x));
            if (page_of[row] < 0) y = make_uint4(Num<E>::NAN2, Num<E>::NAN2, Num<E>::NAN2, Num<E>::NAN2);
            if (!in || h >= Hq) continue;
            E *to = static_cast<E *>(P.out) + (int64_t)(s.row0 + row) * P.out_stride + (int64_t)h * D;
            if (PAIR != PAIR_HALVES) {
                *reinterpret_cast<uint4 *>(to + d0) = y;
            } else {
                *reinterpret_cast<uint2 *>(to + d0) = make_uint2(y.x, y.y);
                *reinterpret_cast<uint2 *>(to + d1) = make_uint2(y.z, y.w);
            }
        }
    }
}

template <typename E, int LPH>
static cudaError_t launch_append8(const Batch &A, const Cache8 &C, Append8Args P, cudaStream_t st) {
    int dev = 0, nsm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // one wave of up to 4 CTAs per SM, and no more warps than tasks
    const int tasks = ((A.k_max + 1) * P.Hq + 2 * C.heads) / 2;
    P.split = 4 * nsm / A.B;
    P.split = P.split < (tasks + 3) / 4 ? P.split : (tasks + 3) / 4;
    P.split = P.split > 1 ? P.split : 1;
    auto *const kernel = P.interleaved || P.half == 0 ? append8_kernel<E, LPH, PAIR_NEXT>
                         : P.half % 4 == 0            ? append8_kernel<E, LPH, PAIR_HALVES>
                                                      : append8_kernel<E, LPH, PAIR_ANY>;
    return launch_dependent(kernel, dim3(A.B * P.split), dim3(AT8), 1, st, A, C, P);
}

}  // namespace svc

using namespace svc;

extern "C" sv_status spec_append8(const void *q, const void *k, const void *v, sv_dtype dtype, int64_t q_stride,
                                  int64_t k_stride, int64_t v_stride, int32_t num_q_heads, const void *q_weight,
                                  const void *k_weight, float eps, const float *inv_freq, int32_t rotary_dim,
                                  int32_t interleaved, float rope_scale, const int32_t *num_drafts,
                                  const int32_t *row_offsets, const int32_t *kv_seq_len, int32_t B, int32_t k_max,
                                  int32_t total_rows, sv_kv_cache8 cache, void *out_q, int64_t out_q_stride,
                                  void *workspace, void *stream) {
    Batch A;
    Cache8 C;
    const sv_status bad = check_batch8(num_drafts, row_offsets, kv_seq_len, B, k_max, total_rows, num_q_heads, dtype,
                                       cache, A, C);
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
    const Append8Args P{q, k, v, q_stride, k_stride, v_stride, out_q_stride, q_weight, k_weight, inv_freq, out_q,
                        static_cast<int32_t *>(workspace), eps, rope_scale, num_q_heads, rotary_dim / 2, interleaved, 1};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = cache.head_dim > 64;
    cudaError_t e;
    if (dtype == SV_BF16)
        e = wide ? launch_append8<__nv_bfloat16, 16>(A, C, P, st) : launch_append8<__nv_bfloat16, 8>(A, C, P, st);
    else
        e = wide ? launch_append8<__half, 16>(A, C, P, st) : launch_append8<__half, 8>(A, C, P, st);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
