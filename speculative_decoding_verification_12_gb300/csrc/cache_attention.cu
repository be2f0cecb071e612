// cache_attention.cu -- spec_attention: the new tokens' rows attend over the paged cache under a
// causal mask with an optional sliding window and first tokens that stay visible.
//
// One warp per (row, query head): one pass over the visible keys with the running maximum and sum
// of the softmax, the output in registers.
#include <math.h>

#include "sv_cache.cuh"

namespace svc {

struct AttnArgs {
    const void *q;
    int64_t q_stride;
    void *out;
    float *lse;
    int32_t *hdr;
    float scale;
    int Hq, window, sinks;
};

constexpr int NT = 128;

template <typename E>
__global__ void __launch_bounds__(NT) attention_kernel(const Batch A, const Cache C, const AttnArgs P) {
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y * (NT / 32) + (threadIdx.x >> 5), r = blockIdx.x;
    if (h >= P.Hq) return;
    const int D = C.D, d0 = lane * 4;
    const bool in = d0 < D;
    E *out = static_cast<E *>(P.out) + ((int64_t)r * P.Hq + h) * D + d0;
    const int b = request_of(A, r);
    Span s = {0, 0, 0, 0};
    if (b >= 0) s = span_of(A, C.max_pages << C.page_shift, b);
    if (h == 0 && lane == 0) check_requests(A, C.max_pages << C.page_shift, P.hdr, r, A.R);
    if (r - s.row0 >= s.n) {
        const uint32_t w = s.err ? Num<E>::NAN2 : 0u;
        if (in) *reinterpret_cast<uint2 *>(out) = make_uint2(w, w);
        if (P.lse && lane == 0) P.lse[(int64_t)r * P.Hq + h] = s.err ? NAN : 0.f;
        return;
    }
    float q[4] = {0, 0, 0, 0}, o[4] = {0, 0, 0, 0};
    if (in) {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const E *>(P.q) + r * P.q_stride + (int64_t)h * D + d0);
        const float2 x = Num<E>::up(w.x), y = Num<E>::up(w.y);
        q[0] = x.x, q[1] = x.y, q[2] = y.x, q[3] = y.y;
    }
    const int pos = s.len - s.n + (r - s.row0), kvh = h / (P.Hq / C.heads);
    const int first = P.window && pos >= P.window ? pos - P.window + 1 : 0;
    const int32_t *row = C.table + (int64_t)b * C.max_pages;
    float m = -INFINITY, l = 0.f;
    bool bad = false;
    for (int j = 0; j <= pos; j++) {
        if (j < first && j >= P.sinks) j = first;
        const int page = __ldg(row + (j >> C.page_shift));
        if (page < 0 || page >= C.num_pages) {
            bad = true;
            break;
        }
        const int64_t at = page * C.page_stride + (j & ((1 << C.page_shift) - 1)) * C.token_stride +
                           kvh * C.head_stride + d0;
        float k[4] = {0, 0, 0, 0}, v[4] = {0, 0, 0, 0};
        if (in) {
            const uint2 a = *reinterpret_cast<const uint2 *>(static_cast<const E *>(C.k) + at);
            const uint2 z = *reinterpret_cast<const uint2 *>(static_cast<const E *>(C.v) + at);
            float2 t = Num<E>::up(a.x);
            k[0] = t.x, k[1] = t.y;
            t = Num<E>::up(a.y);
            k[2] = t.x, k[3] = t.y;
            t = Num<E>::up(z.x);
            v[0] = t.x, v[1] = t.y;
            t = Num<E>::up(z.y);
            v[2] = t.x, v[3] = t.y;
        }
        float x = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
        for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
        x *= P.scale;
        const float top = fmaxf(m, x);
        const float w = top == -INFINITY ? 0.f : expf(m - top), e = top == -INFINITY ? 0.f : expf(x - top);
        l = l * w + e;
#pragma unroll
        for (int i = 0; i < 4; i++) o[i] = o[i] * w + e * v[i];
        m = top;
    }
    if (bad) {
        if (lane == 0) record_error(P.hdr, SV_DEV_BAD_PAGE, b);
        l = NAN;
    }
    if (in) *reinterpret_cast<uint2 *>(out) = make_uint2(Num<E>::down(o[0] / l, o[1] / l), Num<E>::down(o[2] / l, o[3] / l));
    if (P.lse && lane == 0) P.lse[(int64_t)r * P.Hq + h] = m + logf(l);
}

}  // namespace svc

using namespace svc;

extern "C" size_t sv_attention_workspace_bytes(int32_t head_dim) {
    if (head_dim < 8 || head_dim > 128 || head_dim % 8) return 0;
    return HEADER;
}

extern "C" sv_status spec_attention(const void *q, int64_t q_stride, int32_t num_q_heads, const int32_t *num_drafts,
                                    const int32_t *row_offsets, const int32_t *kv_seq_len, int32_t B, int32_t k_max,
                                    int32_t total_rows, sv_kv_cache cache, float scale, int32_t window, int32_t sinks,
                                    void *out, float *out_lse, void *workspace, size_t workspace_bytes,
                                    void *stream) {
    Batch A;
    Cache C;
    const sv_status bad = check_batch(num_drafts, row_offsets, kv_seq_len, B, k_max, total_rows, num_q_heads, cache,
                                      128, A, C);
    if (bad != SV_OK) return bad;
    if (!q || !out || !workspace || window < 0 || sinks < 0 || !(fabsf(scale) < INFINITY)) return SV_ERR_INVALID_ARG;
    if (q_stride < (int64_t)num_q_heads * cache.head_dim) return SV_ERR_INVALID_ARG;
    if (q_stride % 8 || !aligned16(q) || !aligned16(out)) return SV_ERR_UNSUPPORTED;
    if (((uintptr_t)workspace & 255) || workspace_bytes < sv_attention_workspace_bytes(cache.head_dim))
        return SV_ERR_WORKSPACE;
    const AttnArgs P{q, q_stride, out, out_lse, static_cast<int32_t *>(workspace), scale, num_q_heads, window, sinks};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(total_rows, (num_q_heads + NT / 32 - 1) / (NT / 32));
    if (cache.dtype == SV_BF16) attention_kernel<__nv_bfloat16><<<grid, NT, 0, st>>>(A, C, P);
    else attention_kernel<__half><<<grid, NT, 0, st>>>(A, C, P);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
