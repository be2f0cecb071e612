// sv_cache.cuh -- what the cache-side kernels (append, attention, page bookkeeping) share: the
// batch's rows and lengths, the paged cache's addressing, error records and small helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spec_cache.h"

namespace svc {

constexpr int MAXK = 64;            // largest k_max, as in spec_verify
constexpr int MAXB = 1 << 25;       // requests (exclusive), as in spec_verify
constexpr int MAXHEADS = 1024;
constexpr int HEADER = 256;         // bytes of the workspace's header (error word, request)

// Records a device-data error: the first code wins; the lowest request index is kept.
__device__ __forceinline__ void record_error(int32_t *hdr, int code, int b) {
    atomicCAS(hdr, 0, code);
    atomicMax(hdr + 1, 0x7fffffff - b);
}

// Everything here is read with plain loads: under a programmatic launch the work before may still be
// writing it while this grid is already resident, which the read-only path does not allow for.
struct Batch {
    const int32_t *nd;        // num_drafts
    const int32_t *row_off;   // NULL: uniform layout
    const int32_t *len;       // kv_seq_len
    int B, k_max, R;
};

struct Cache {
    void *k, *v;
    int64_t page_stride, token_stride, head_stride;
    const int32_t *table;
    int num_pages, page_shift, heads, D, max_pages;
};

// A request's rows: the first one, how many it uses (0: idle or in error) and its length.
struct Span {
    int row0, n, len, err;   // err: SV_DEV_* (0: none)
};

__device__ __forceinline__ Span span_of(const Batch &A, int max_tokens, int b) {
    Span s;
    int owned;
    if (A.row_off) {
        s.row0 = A.row_off[b];
        const int end = A.row_off[b + 1];
        owned = (s.row0 >= 0 && end >= s.row0 && end <= A.R) ? end - s.row0 : -1;
    } else {
        s.row0 = b * (A.k_max + 1);
        owned = A.k_max + 1;
    }
    const int k = A.nd[b];
    s.len = A.len[b];
    s.n = k + 1;
    s.err = 0;
    if (k == -1 && owned >= 0) return s;   // idle
    if (k < 0 || k > A.k_max || owned < s.n || s.len < s.n || s.len > max_tokens) {
        s.err = SV_DEV_BAD_LAYOUT;
        s.n = 0;
    }
    return s;
}

// The request that owns row r of a ragged layout: the last b with row_off[b] <= r; -1 when the row
// belongs to none.  One thread, binary search.
static __device__ __noinline__ int request_of(const Batch &A, int r) {
    int lo = 0, hi = A.B;   // row_off[lo] <= r < row_off[hi], if the offsets are sound
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (A.row_off[mid] <= r) lo = mid;
        else hi = mid;
    }
    return (A.row_off[lo] <= r && r < A.row_off[lo + 1]) ? lo : -1;
}

// The request that owns row first + lane, for lanes below `rows` <= 32; -1 for a row that belongs to
// none.  One warp: a 32-way search for the request of `first`, then the rows after it count the
// offsets up to them among the next 32; where more than that many requests own no row, or `first` lies
// before them all, each lane searches for itself.
__device__ __forceinline__ int request_of_rows(const Batch &A, int first, int rows) {
    const int lane = threadIdx.x & 31;
    if (!A.row_off) return (first + lane) / (A.k_max + 1);
    int lo = 0, hi = A.B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, i = min(lo + lane * step, hi - 1);
        const uint32_t m = __ballot_sync(0xffffffffu, A.row_off[i] <= first);
        lo = min(lo + (m ? 31 - __clz(m) : 0) * step, hi - 1);
        hi = min(hi, lo + step);
    }
    const int next = lo + 1 + lane <= A.B ? A.row_off[lo + 1 + lane] : 0x7fffffff;
    bool search = A.row_off[lo] > first;
    int mine = -1;
    for (int i = 0; i < rows; i++) {
        const int later = __popc(__ballot_sync(0xffffffffu, next <= first + i));
        if (lane == i) {
            mine = lo + later < A.B ? lo + later : -1;
            search |= later == 32;
        }
    }
    if (search && lane < rows) mine = request_of(A, first + lane);
    return mine;
}

// Reports the requests whose rows, length or drafts are out of range: a request with unsound
// offsets may own no row that leads to it.  Worker i of n takes requests i, i + n, ...
__device__ __forceinline__ void check_requests(const Batch &A, int max_tokens, int32_t *hdr, int i, int n) {
    for (int b = i; b < A.B; b += n) {
        const Span s = span_of(A, max_tokens, b);
        if (s.err) record_error(hdr, s.err, b);
    }
}

template <typename E>
struct Num;
template <>
struct Num<__nv_bfloat16> {
    static __device__ __forceinline__ float2 up(uint32_t w) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
    }
    static __device__ __forceinline__ uint32_t down(float a, float b) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    static constexpr uint32_t NAN2 = 0x7fff7fffu, ONE2 = 0x3f803f80u;
    static constexpr bool BF16 = true;
};
template <>
struct Num<__half> {
    static __device__ __forceinline__ float2 up(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    static __device__ __forceinline__ uint32_t down(float a, float b) {
        const __half2 r = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    static constexpr uint32_t NAN2 = 0x7fff7fffu, ONE2 = 0x3c003c00u;
    static constexpr bool BF16 = false;
};

template <typename E>
__device__ __forceinline__ void unpack8(const uint4 &w, float x[8]) {
    const uint32_t *p = &w.x;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = Num<E>::up(p[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <typename E>
__device__ __forceinline__ uint4 pack8(const float x[8]) {
    return make_uint4(Num<E>::down(x[0], x[1]), Num<E>::down(x[2], x[3]), Num<E>::down(x[4], x[5]),
                      Num<E>::down(x[6], x[7]));
}

// --- host side ---

// Launches a kernel as a programmatic dependent of the work before it on the stream: its CTAs may be
// resident before that work ends, and wait for it (grid_wait) before their first access.
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, int cluster, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Checks shared by spec_append and spec_attention; fills the kernels' views of the arguments.
inline sv_status check_batch(const int32_t *num_drafts, const int32_t *row_offsets, const int32_t *kv_seq_len,
                             int32_t B, int32_t k_max, int32_t total_rows, int32_t num_q_heads,
                             const sv_kv_cache &c, int max_head_dim, Batch &batch, Cache &cache) {
    if (B < 1 || k_max < 0 || total_rows < 1 || !num_drafts || !kv_seq_len) return SV_ERR_INVALID_ARG;
    if (k_max > MAXK || B >= MAXB) return SV_ERR_UNSUPPORTED;
    if (!row_offsets && (long long)total_rows != (long long)B * (k_max + 1)) return SV_ERR_INVALID_ARG;
    if (c.dtype != SV_BF16 && c.dtype != SV_F16) return SV_ERR_INVALID_ARG;
    if (!c.k || !c.v || !c.block_table || c.num_pages < 1 || c.num_heads < 1 || c.max_pages < 1 || c.head_dim < 1)
        return SV_ERR_INVALID_ARG;
    if (num_q_heads < 1 || num_q_heads % c.num_heads != 0) return SV_ERR_INVALID_ARG;
    if (c.page_stride <= 0 || c.token_stride <= 0 || c.head_stride <= 0) return SV_ERR_INVALID_ARG;
    if (num_q_heads > MAXHEADS || c.head_dim % 8 != 0 || c.head_dim > max_head_dim) return SV_ERR_UNSUPPORTED;
    if (c.page_size < 8 || c.page_size > 256 || (c.page_size & (c.page_size - 1))) return SV_ERR_UNSUPPORTED;
    if (c.page_stride % 8 || c.token_stride % 8 || c.head_stride % 8 || !aligned16(c.k) || !aligned16(c.v))
        return SV_ERR_UNSUPPORTED;
    // (a tile past the last token must not overflow; a tensor map's strides have 40 bits)
    if ((long long)c.max_pages * c.page_size > 0x7ffffe00ll) return SV_ERR_UNSUPPORTED;
    if ((c.page_stride | c.token_stride | c.head_stride) >> 38) return SV_ERR_UNSUPPORTED;
    batch = Batch{num_drafts, row_offsets, kv_seq_len, B, k_max, total_rows};
    cache.k = c.k;
    cache.v = c.v;
    cache.page_stride = c.page_stride;
    cache.token_stride = c.token_stride;
    cache.head_stride = c.head_stride;
    cache.table = c.block_table;
    cache.num_pages = c.num_pages;
    cache.page_shift = __builtin_ctz((unsigned)c.page_size);
    cache.heads = c.num_heads;
    cache.D = c.head_dim;
    cache.max_pages = c.max_pages;
    return SV_OK;
}

}  // namespace svc
