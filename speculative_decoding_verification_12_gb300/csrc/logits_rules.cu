// logits_rules.cu -- spec_logits: penalties for repeated tokens, biases and grammar masks on the logits of
// a verify step.
//
// Mathematics: z -> (z > 0 ? z / r : z r) for a seen token, - (presence [c > 0] + frequency c), + bias, and -inf
// where the row's mask refuses the token; fp32, rounded once.  Masks touch every token, the other rules
// a few hundred of a row.
//
// One pass.  A CTA takes a piece of one row: it copies the piece and puts the refused tokens to -inf, 16 bytes
// at a time, or, where the output is the input, writes the refused tokens alone.  After a barrier its threads take the
// entries of the request's sorted lists that lie in the piece: a token in several of history, drafts and biases
// is the first one's, which looks it up in the others and marks it there, so every element has one writer and one
// rounding.  What the entries read again of the piece is still in L2.
//
// What bounds it: memory, and the entries: 1280 bf16 rows of 128 256 are copied in 100 us (97 % of the memory's rate), with
// 1000 tokens of history and 16 biases a request in 123, with masks on half the rows besides in 128.  (Bringing a piece's
// entries into shared memory during its copy: 134.)  Masks alone, in place, on 2048 fp32 rows: 208 us, for sectors that
// are refused in part and so come from memory and go back.  In place with lists, the 1280 rows take 77 us (masks on half of
// them) and 2500 rows of 151 937 with 1500 tokens of history each 140, four times what their sectors need, probably for the
// entries' loads in turn.  One row of 32 000: 5.8 us, latency.
#include <math.h>

#include "../../include/spec_logits.h"
#include "sv_cache.cuh"
#include "sv_tc.cuh"

namespace svc {

struct LogitArgs {
    const void *in;
    void *out;
    const int32_t *drafts;
    sv_logit_rules r;
    int32_t *hdr;
    int V;
    int penalties;   // whether any is given
    int piece;       // tokens of a row per CTA, a multiple of a pass of its threads
};

constexpr int LT = 256;       // threads per CTA
constexpr int MOST_STEPS = 16;   // of a piece that has entries: what they read again is to be in L2 still (512 requests of 1500
                                // tokens, 151 937 logits: 308, 279, 323, 354 us with 8, 16, 24, 40)
constexpr int BIASES = 256;   // of a piece that are kept in shared memory

template <typename E>
struct Logit;
template <>
struct Logit<__nv_bfloat16> {
    static constexpr int VEC = 8;
    static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
    // 16 bytes with the elements whose bit is clear put to -inf
    static __device__ __forceinline__ uint4 refuse(uint4 w, uint32_t bits) {
        uint32_t *p = &w.x;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (!(bits >> 2 * i & 1)) p[i] = (p[i] & 0xffff0000u) | 0xff80u;
            if (!(bits >> (2 * i + 1) & 1)) p[i] = (p[i] & 0xffffu) | 0xff800000u;
        }
        return w;
    }
};
template <>
struct Logit<float> {
    static constexpr int VEC = 4;
    static __device__ __forceinline__ float up(float x) { return x; }
    static __device__ __forceinline__ float down(float x) { return x; }
    static __device__ __forceinline__ uint4 refuse(uint4 w, uint32_t bits) {
        uint32_t *p = &w.x;
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (!(bits >> i & 1)) p[i] = 0xff800000u;
        return w;
    }
};

// Entries of the lists are counted without a sign: lists may hold 2^31 - 1, and steps and sums go past that.

// First index in [lo, hi) of an ascending list whose id is >= v (hi: none).  A whole warp, 32 ids at a time.
__device__ __forceinline__ uint32_t first_at(const int32_t *ids, uint32_t lo, uint32_t hi, int v) {
    const uint32_t lane = threadIdx.x & 31;
    while (lo < hi) {
        const uint32_t step = (hi - lo + 31) / 32, i = lo + lane * step;
        const uint32_t below = __popc(__ballot_sync(0xffffffffu, i < hi && ids[i] < v));   // of lo, lo + step, ...
        if (below == 0) return lo;
        hi = min(hi, lo + below * step);
        lo += (below - 1) * step + 1;
    }
    return lo;
}
// Index of v in an ascending list, or -1.  One thread.
__device__ __forceinline__ int find(const int32_t *ids, uint32_t lo, uint32_t hi, int v) {
    while (lo < hi) {
        const uint32_t mid = (lo + hi) >> 1;
        const int x = ids[mid];
        if (x == v) return (int)mid;
        if (x < v) lo = mid + 1;
        else hi = mid;
    }
    return -1;
}

// Checks a request's list [lo, hi): ascending ids in [0, V), counts (if any) >= 0.  A whole CTA.
__device__ __forceinline__ bool unsound(const int32_t *ids, const int32_t *counts, uint32_t lo, uint32_t hi, int V) {
    bool bad = false;
    for (uint32_t e = lo + threadIdx.x; e < hi; e += LT) {
        const int v = ids[e];
        bad |= v < 0 || v >= V || (e > lo && ids[e - 1] >= v) || (counts && counts[e] < 0);
    }
    return bad;
}

// SAME: the output is the input.
template <typename E, bool SAME>
__global__ void __launch_bounds__(LT, SAME ? 8 : 5) logits_kernel(const Batch A, const LogitArgs P) {
    constexpr int VEC = Logit<E>::VEC, STEP = LT * VEC;
    constexpr int NV = 4;                 // 16-byte vectors of a thread on their way at a time
    __shared__ int drafts[MAXK];
    __shared__ int range[4];              // this piece's entries of the history and of the biases
    __shared__ int ends[4];               // the request's
    __shared__ int status, mask_at, row_i, request;
    __shared__ int bias_ids[BIASES];      // this piece's biases, if they are no more
    __shared__ uint8_t draft_done[MAXK], bias_done[BIASES];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x, V = P.V;
    const int64_t row_at = (int64_t)row * V;
    // elements of the row's first 128 bytes that are not its own: the warps' accesses are whole lines
    const int lead = SAME ? 0 : (int)((((uintptr_t)P.out & 127) / sizeof(E) + row_at) % (128 / sizeof(E)));
    const int c0 = max((int)blockIdx.y * P.piece - lead, 0), c1 = (int)min((int64_t)(blockIdx.y + 1) * P.piece - lead, (int64_t)V);
    if (c0 >= c1) return;
    const E *in = static_cast<const E *>(P.in) + row_at;
    E *out = static_cast<E *>(P.out) + row_at;

    grid_wait();
    grid_launch_dependents();
    // this thread's first vectors, under way while the request is found
    uint4 x[NV];
    const int base = (int)blockIdx.y * P.piece - lead + tid * VEC;   // token of the first element
    auto whole = [&](int v) { return v >= 0 && v < c1 && v + VEC <= V; };
    auto fetch = [&](int v0) {
#pragma unroll
        for (int k = 0; k < NV; k++)
            if (whole(v0 + k * STEP)) x[k] = *reinterpret_cast<const uint4 *>(in + v0 + k * STEP);
    };
    if (!SAME) fetch(base);
    if (warp == 0) {
        // the row's request, and whether it is sound: status 0 used, 1 unused, 2 in error
        const int b = __shfl_sync(0xffffffffu, request_of_rows(A, row, 1), 0);
        int st = 1, err = 0, i = 0, first = 0, n = 0, o[4] = {0, 0, 0, 0}, mask = -1;
        if (b >= 0) {
            int owned = A.k_max + 1;
            first = b * (A.k_max + 1);
            if (A.row_off) {
                first = A.row_off[b];
                const int end = A.row_off[b + 1];
                owned = first >= 0 && end >= first && end <= A.R ? end - first : -1;
            }
            i = row - first;
            n = A.nd[b] + 1;
            if (n < 1 || n > A.k_max + 1 || owned < n) err = SV_DEV_BAD_LAYOUT, n = 0;
            // (requests without rows before this one: its drafts are not where they should be)
            if (!err && (first < b || first - b + n - 1 > A.R - A.B)) err = SV_DEV_BAD_LAYOUT, n = 0;
            if (!err && P.penalties)
                for (int j = lane; j < n - 1; j += 32) {
                    const int v = P.drafts[first - b + j];
                    drafts[j] = v;
                    if (v < 0 || v >= V) err = SV_DEV_BAD_TOKEN;
                }
            if (!err && lane < 3) {
                const float *p = lane == 0 ? P.r.repetition : lane == 1 ? P.r.presence : P.r.frequency;
                if (p && (!(fabsf(p[b]) < INFINITY) || (lane == 0 && !(p[b] > 0.f)))) err = SV_DEV_BAD_PENALTY;
            }
            if (P.r.prior_offsets) {
                o[0] = P.r.prior_offsets[b], o[1] = P.r.prior_offsets[b + 1];
                if (!err && (o[0] < 0 || o[1] < o[0] || o[1] > P.r.prior_len)) err = SV_DEV_BAD_HISTORY;
            }
            if (P.r.bias_offsets) {
                o[2] = P.r.bias_offsets[b], o[3] = P.r.bias_offsets[b + 1];
                if (!err && (o[2] < 0 || o[3] < o[2] || o[3] > P.r.bias_len)) err = SV_DEV_BAD_BIAS;
            }
            if (P.r.mask_rows)
                for (int j = lane; j < n; j += 32) {
                    const int m = P.r.mask_rows[first + j];
                    if (j == i) mask = m;
                    if (!err && (m < -1 || m >= P.r.num_masks)) err = SV_DEV_BAD_MASK;
                }
            mask = __reduce_max_sync(0xffffffffu, mask);   // (the one lane's; the others have -1)
            const unsigned bad = __ballot_sync(0xffffffffu, err != 0);
            if (bad) err = __shfl_sync(0xffffffffu, err, __ffs(bad) - 1);
            st = err ? 2 : i < n ? 0 : 1;
            if (err && lane == 0 && blockIdx.y == 0) record_error(P.hdr, err, b);
        }
        if (lane == 0) {
            status = st;
            mask_at = mask;
            row_i = i;
            request = b;
            for (int e = 0; e < 4; e++) ends[e] = o[e];
        }
    }
    __syncthreads();
    const int st = status, b = request, i = row_i;
    if (blockIdx.y == 0)   // (a request without rows has no other CTA that could report it)
        for (int64_t q = (int64_t)row * LT + tid; q < A.B; q += (int64_t)A.R * LT)
            if (A.row_off && (A.row_off[q] < 0 || A.row_off[q + 1] <= A.row_off[q] || A.row_off[q + 1] > A.R))
                record_error(P.hdr, SV_DEV_BAD_LAYOUT, (int)q);
    if (st == 1) return;
    if (st == 2) {
        for (int v = c0 + tid; v < c1; v += LT) out[v] = Logit<E>::down(NAN);
        return;
    }
    const uint32_t *mask = mask_at < 0 ? nullptr : P.r.masks + (int64_t)mask_at * P.r.mask_words;
    if (warp >= 4 && warp < 8 && (warp < 6 ? P.r.prior_offsets : P.r.bias_offsets) != nullptr) {   // (under way with the masks)
        const int e = warp - 4;
        const int at = first_at(e < 2 ? P.r.prior_tokens : P.r.bias_tokens, ends[e & 2], ends[(e & 2) + 1], e & 1 ? c1 : c0);
        if (lane == 0) range[e] = at;
    } else if (warp >= 4 && lane == 0) {
        range[warp - 4] = 0;
    }
    // the mask's words of tokens v .. v + VEC - 1, and their bits (those outside [0, V) clear or not)
    auto words = [&](int v, uint32_t &lo, uint32_t &hi) {
        lo = hi = 0xffffffffu;
        if (!mask || v >= c1 || v + VEC <= 0) return;
        const int u = max(v, 0);
        lo = mask[u >> 5];
        if ((u & 31) + VEC > 32 && (u >> 5) + 1 < P.r.mask_words) hi = mask[(u >> 5) + 1];
    };
    constexpr uint32_t ALL = (1u << VEC) - 1;
    auto allowed = [&](int v, uint32_t lo, uint32_t hi) {
        const uint32_t bits = __funnelshift_r(lo, hi, max(v, 0) & 31);
        return (v < 0 ? bits << -v : bits) & ALL;
    };
    if (SAME) {
        // Only refused logits are written: a lane has a word of the mask, and the warp an element a lane of each word in turn
        // (2048 fp32 rows of 128 256: 208 us; 16 bytes a thread, read first where a part is refused, 232).
        if (mask)
            for (int u0 = c0 + warp * 1024; u0 < c1; u0 += LT * 32) {
                const int first = u0 + lane * 32;
                uint32_t mine = first < c1 ? ~mask[first >> 5] : 0u;   // refused
                if (first + 32 > V) mine &= first < V ? 0xffffffffu >> (first + 32 - V) : 0u;
                if (!__any_sync(0xffffffffu, mine != 0)) continue;
                E *const at = out + u0 + lane;
#pragma unroll
                for (int k = 0; k < 32; k++)
                    if (__shfl_sync(0xffffffffu, mine, k) >> lane & 1) at[k * 32] = Logit<E>::down(-INFINITY);
            }
    } else {
        uint32_t lo[NV], hi[NV];   // of the next vectors
#pragma unroll
        for (int k = 0; k < NV; k++) words(base + k * STEP, lo[k], hi[k]);
#pragma unroll 1
        for (int v0 = base; v0 < c1; v0 += NV * STEP) {
            uint32_t bits[NV];
#pragma unroll
            for (int k = 0; k < NV; k++) {
                bits[k] = allowed(v0 + k * STEP, lo[k], hi[k]);
                words(v0 + (NV + k) * STEP, lo[k], hi[k]);
            }
#pragma unroll
            for (int k = 0; k < NV; k++) {
                const int v = v0 + k * STEP;
                if (v >= c1 || v + VEC <= 0) continue;
                if (whole(v)) {
                    *reinterpret_cast<uint4 *>(out + v) = bits[k] == ALL ? x[k] : Logit<E>::refuse(x[k], bits[k]);
                } else {
                    for (int e = 0; e < VEC; e++) {
                        if (v + e < 0 || v + e >= V) continue;
                        if (!(bits[k] >> e & 1)) out[v + e] = Logit<E>::down(-INFINITY);
                        else out[v + e] = in[v + e];
                    }
                }
            }
            fetch(v0 + NV * STEP);
        }
    }
    __syncthreads();

    // the entries of this piece
    const float rep = P.r.repetition ? P.r.repetition[b] : 1.f, presence = P.r.presence ? P.r.presence[b] : 0.f,
                frequency = P.r.frequency ? P.r.frequency[b] : 0.f;
    // (p0 <= p1 and b0 <= b1 also in lists that do not ascend: what first_at counts can only grow with v)
    const int p0 = range[0], p1 = range[1], b0 = range[2], b1 = range[3];
    const int nd = P.penalties ? i : 0;
    const bool kept = b1 - b0 <= BIASES;
    if (kept && tid < b1 - b0) bias_ids[tid] = P.r.bias_tokens[b0 + tid], bias_done[tid] = 0;
    if (tid < nd) draft_done[tid] = 0;
    __syncthreads();
    // token v with logit z, its count in the history (-1: not in it) and its place among the biases (-2: to be looked up)
    auto put = [&](int v, float z, int prior, int bias) {
        const bool refused = mask && !(mask[v >> 5] >> (v & 31) & 1);
        uint32_t count = max(prior, 0);   // (drafts may take it past 2^31)
        bool seen = prior >= 0;
        for (int j = 0; j < nd; j++)
            if (drafts[j] == v) count++, seen = true, draft_done[j] = 1;
        if (bias == -2) {
            bias = kept ? find(bias_ids, 0, b1 - b0, v) : find(P.r.bias_tokens, b0, b1, v);
            if (kept && bias >= 0) {
                bias_done[bias] = 1;
                bias += b0;
            }
        }
        if (refused) return;
        if (seen) {
            z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
            z = __fsub_rn(z, __fadd_rn(count > 0 ? presence : 0.f, __fmul_rn(frequency, (float)count)));
        }
        if (bias >= 0) z = __fadd_rn(z, P.r.bias_values[bias]);
        out[v] = Logit<E>::down(z);
    };
    auto here = [&](int v) { return v >= c0 && v < c1; };
    for (uint32_t e = p0 + tid; e < (uint32_t)p1; e += 4 * LT) {   // (four entries' loads at a time: 512 requests of 1500 tokens 363 us one by one)
        int v[4], count[4];
        float z[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            v[k] = e + k * LT < (uint32_t)p1 ? P.r.prior_tokens[e + k * LT] : -1;
            count[k] = e + k * LT < (uint32_t)p1 ? max(P.r.prior_counts[e + k * LT], 0) : 0;
        }
#pragma unroll
        for (int k = 0; k < 4; k++) z[k] = here(v[k]) ? Logit<E>::up(in[v[k]]) : 0.f;
#pragma unroll
        for (int k = 0; k < 4; k++)
            if (here(v[k])) put(v[k], z[k], count[k], -2);
    }
    __syncthreads();
    // drafts that the history has not got, each by its first occurrence
    bool mine = tid < nd && !draft_done[tid];
    for (int j = 0; mine && j < tid; j++) mine = drafts[j] != drafts[tid];
    __syncthreads();
    if (mine && here(drafts[tid])) put(drafts[tid], Logit<E>::up(in[drafts[tid]]), -1, -2);
    __syncthreads();
    for (uint32_t e = b0 + tid; e < (uint32_t)b1; e += LT) {
        const int v = kept ? bias_ids[e - b0] : P.r.bias_tokens[e];
        bool other = kept && bias_done[e - b0];
        if (!kept) {
            for (int j = 0; j < nd && !other; j++) other = drafts[j] == v;
            other = other || find(P.r.prior_tokens, p0, p1, v) >= 0;
        }
        if (!other && here(v)) put(v, Logit<E>::up(in[v]), -1, (int)e);
    }
    // the request's first row reports what is wrong with its lists
    if (i == 0 && blockIdx.y == 0) {
        if (P.r.prior_offsets && unsound(P.r.prior_tokens, P.r.prior_counts, ends[0], ends[1], V))
            record_error(P.hdr, SV_DEV_BAD_HISTORY, b);
        if (P.r.bias_offsets && unsound(P.r.bias_tokens, nullptr, ends[2], ends[3], V)) record_error(P.hdr, SV_DEV_BAD_BIAS, b);
    }
}

template <typename E>
static cudaError_t launch_logits(const Batch &A, LogitArgs P, cudaStream_t st) {
    constexpr int VEC = Logit<E>::VEC, STEP = LT * VEC;
    int dev = 0, nsm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // pieces of a row: about 4 waves of CTAs, 8 a multiprocessor, where the rows are fewer than that
    const int steps = (int)((P.V + 128 / sizeof(E) - 1 + STEP - 1) / STEP);   // (a row may begin anywhere in 128 bytes)
    const long long want = 32ll * nsm;
    const int pieces = (int)(A.R >= want ? 1 : (want + A.R - 1) / A.R < steps ? (want + A.R - 1) / A.R : steps);
    int per = (steps + pieces - 1) / pieces;
    if ((P.r.prior_offsets || P.r.bias_offsets) && per > MOST_STEPS) per = MOST_STEPS;
    P.piece = per * STEP;
    const dim3 grid(A.R, (steps + per - 1) / per);
    return P.in == P.out ? launch_dependent(logits_kernel<E, true>, grid, dim3(LT), 1, st, A, P)
                         : launch_dependent(logits_kernel<E, false>, grid, dim3(LT), 1, st, A, P);
}

}  // namespace svc

using namespace svc;

extern "C" sv_status spec_logits(const void *logits, sv_dtype dtype, const int32_t *draft_tokens, const int32_t *num_drafts,
                                 const int32_t *row_offsets, int32_t B, int32_t k_max, int32_t V, int32_t total_rows,
                                 sv_logit_rules rules, void *out, void *workspace, void *stream) {
    const sv_logit_rules &r = rules;
    if (B < 1 || k_max < 0 || V < 1 || total_rows < 1 || !logits || !out || !num_drafts || !workspace)
        return SV_ERR_INVALID_ARG;
    if (dtype != SV_BF16 && dtype != SV_F32) return SV_ERR_INVALID_ARG;
    if (k_max > MAXK || B >= MAXB || V > 1 << 21) return SV_ERR_UNSUPPORTED;
    if (!row_offsets && (long long)total_rows != (long long)B * (k_max + 1)) return SV_ERR_INVALID_ARG;
    const bool penalties = r.repetition || r.presence || r.frequency;
    if (penalties && k_max > 0 && total_rows > B && !draft_tokens) return SV_ERR_INVALID_ARG;
    if (r.prior_offsets && (r.prior_len < 0 || (r.prior_len && (!r.prior_tokens || !r.prior_counts)))) return SV_ERR_INVALID_ARG;
    if (r.bias_offsets && (r.bias_len < 0 || (r.bias_len && (!r.bias_tokens || !r.bias_values)))) return SV_ERR_INVALID_ARG;
    if (r.mask_rows && (r.num_masks < 0 || (r.num_masks && (!r.masks || r.mask_words < (V + 31) / 32)))) return SV_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(out)) return SV_ERR_UNSUPPORTED;
    if ((uintptr_t)workspace & 255) return SV_ERR_WORKSPACE;
    const uintptr_t from = (uintptr_t)logits, to = (uintptr_t)out, bytes = (uintptr_t)total_rows * V * (dtype == SV_F32 ? 4 : 2);
    if (from != to && from < to + bytes && to < from + bytes) return SV_ERR_INVALID_ARG;   // (partly the same)
    const Batch A{num_drafts, row_offsets, nullptr, B, k_max, total_rows};
    LogitArgs P{logits, out, draft_tokens, rules, static_cast<int32_t *>(workspace), V, penalties};
    if (!penalties) P.r.prior_offsets = nullptr;   // (nothing looks at the history)
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SV_BF16 ? launch_logits<__nv_bfloat16>(A, P, st) : launch_logits<float>(A, P, st);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
