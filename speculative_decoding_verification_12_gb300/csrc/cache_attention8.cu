// cache_attention8.cu -- spec_attention8: the new tokens' rows attend over a paged cache of e4m3 numbers with
// a scale per block of tokens and head.
//
// A CTA per row and query head walks the keys 128 at a time with the running maximum and sum of the softmax:
// a thread a key for the scores, a thread an element for the values.
#include "sv_cache8.cuh"
#include "sv_tc.cuh"

namespace svc {

struct Attn8Args {
    const void *q;
    int64_t q_stride;
    void *out;
    float *lse;
    int32_t *hdr;
    float scale;
    int Hq, G, window, sinks;
};

template <typename E>
__global__ void __launch_bounds__(128) attention8_kernel(const Batch A, const Cache8 C, const Attn8Args P) {
    __shared__ float q[128], p[128], red[4];
    __shared__ int64_t at[128];
    const int tid = threadIdx.x, row = blockIdx.x, head = blockIdx.y, D = C.D, kvh = head / P.G;
    grid_wait();
    grid_launch_dependents();
    const int b = __shfl_sync(0xffffffffu, request_of_rows(A, row, 1), 0);
    Span s = {};
    if (b >= 0) s = span_of(A, C.max_pages << C.page_shift, b);
    if (head == 0) check_requests(A, C.max_pages << C.page_shift, P.hdr, row * 128 + tid, A.R * 128);
    E *out = static_cast<E *>(P.out) + ((int64_t)row * P.Hq + head) * D;
    const int i = row - s.row0;
    if (b < 0 || i >= s.n) {
        if (tid < D) out[tid] = (E)(s.err ? NAN : 0.f);
        if (tid == 0 && P.lse) P.lse[(int64_t)row * P.Hq + head] = s.err ? NAN : 0.f;
        return;
    }
    const int pos = s.len - s.n + i;
    if (tid < D) q[tid] = (float)static_cast<const E *>(P.q)[(int64_t)row * P.q_stride + head * D + tid];
    const int lo = P.window ? max(0, pos - P.window + 1) : 0;
    float m = -INFINITY, l = 0.f, o = 0.f;
    bool broken = false;
    for (int base = 0; base <= pos; base += 128) {
        if (base + 127 < lo && base >= P.sinks) continue;
        const int j = base + tid;
        float z = -INFINITY;
        __syncthreads();
        at[tid] = -1;
        if (j <= pos && (j >= lo || j < P.sinks)) {
            const int page = C.table[(int64_t)b * C.max_pages + (j >> C.page_shift)], slot = j & ((1 << C.page_shift) - 1);
            if (page < 0 || page >= C.num_pages) {
                record_error(P.hdr, SV_DEV_BAD_PAGE, b);
                broken = true;
            } else {
                at[tid] = (int64_t)page << 8 | slot;
                const uint8_t *k = C.k + page * C.page_stride + slot * C.token_stride + kvh * C.head_stride;
                float sum = 0.f;
                for (int d = 0; d < D; d += 2) {
                    const float2 x = unpack_e4m3(*reinterpret_cast<const uint16_t *>(k + d));
                    sum += x.x * q[d] + x.y * q[d + 1];
                }
                z = sum * P.scale * clean_scale(C.k_scale[page * C.s_page + (slot >> C.block_shift) * C.s_block + kvh * C.s_head]);
            }
        }
        float top = z;
        for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        if (tid % 32 == 0) red[tid / 32] = top;
        __syncthreads();
        top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float new_m = fmaxf(m, top), f = new_m == -INFINITY ? 1.f : expf(m - new_m);
        const float w = z == -INFINITY ? 0.f : expf(z - new_m);
        m = new_m;
        l *= f;
        o *= f;
        p[tid] = w;
        __syncthreads();
        for (int k = 0; k < 128; k++) {
            if (at[k] < 0) continue;
            l += p[k];
            if (tid >= D) continue;
            const int64_t page = at[k] >> 8;
            const int slot = (int)(at[k] & 255);
            const uint8_t *v = C.v + page * C.page_stride + slot * C.token_stride + kvh * C.head_stride;
            o += p[k] * clean_scale(C.v_scale[page * C.s_page + (slot >> C.block_shift) * C.s_block + kvh * C.s_head]) *
                 unpack_e4m3(v[tid]).x;
        }
    }
    if (__syncthreads_or(broken)) o = l = NAN;
    if (tid < D) out[tid] = (E)(o / l);
    if (tid == 0 && P.lse) P.lse[(int64_t)row * P.Hq + head] = m + logf(l);
}

}  // namespace svc

using namespace svc;

extern "C" sv_status spec_attention8(const void *q, sv_dtype dtype, int64_t q_stride, int32_t num_q_heads,
                                     const int32_t *num_drafts, const int32_t *row_offsets, const int32_t *kv_seq_len,
                                     int32_t B, int32_t k_max, int32_t total_rows, sv_kv_cache8 cache, float scale,
                                     int32_t window, int32_t sinks, void *out, float *out_lse, void *workspace,
                                     size_t workspace_bytes, void *stream) {
    Batch A;
    Cache8 C;
    const sv_status bad = check_batch8(num_drafts, row_offsets, kv_seq_len, B, k_max, total_rows, num_q_heads, dtype,
                                       cache, A, C);
    if (bad != SV_OK) return bad;
    if (!q || !out || !workspace || window < 0 || sinks < 0 || !(fabsf(scale) < INFINITY)) return SV_ERR_INVALID_ARG;
    if (q_stride < (int64_t)num_q_heads * cache.head_dim) return SV_ERR_INVALID_ARG;
    if (q_stride % 8 || !aligned16(q) || !aligned16(out)) return SV_ERR_UNSUPPORTED;
    if (((uintptr_t)workspace & 255) || workspace_bytes < sv_attention_workspace_bytes(cache.head_dim)) return SV_ERR_WORKSPACE;
    const Attn8Args P{q, q_stride, out, out_lse, static_cast<int32_t *>(workspace), scale, num_q_heads,
                      num_q_heads / cache.num_heads, window < (cache.max_pages << C.page_shift) ? window : 0, sinks};
    const dim3 grid(total_rows, num_q_heads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SV_BF16 ? launch_dependent(attention8_kernel<__nv_bfloat16>, grid, dim3(128), 1, st, A, C, P)
                                           : launch_dependent(attention8_kernel<__half>, grid, dim3(128), 1, st, A, C, P);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
