// cache_pages.cu -- page bookkeeping of the paged KV cache: reserve, rollback, fork, release, compact, copy.
//
// The only record of what is free is ref_count itself (0: free), and pages are taken lowest id
// first, in request order: rank r of the free pages goes to the r-th page asked for.  Both ranks
// are prefix sums, so a call is two scans joined by rank: one thread-block cluster counts the
// free pages of its warps' slices, exchanges the counts through distributed shared memory, and
// writes the first pages asked for as a list; its first CTA then walks the requests.  Nothing
// depends on the order of atomics, and no free list has to be kept consistent between calls.
// These kernels move a few hundred KB at most and are bound by latency (launch, two dependent
// passes over the counts, one cluster barrier): fork, copy, reserve, rollback and release together take
// 17.6 us on the GPU for 8 requests and 30 for 512 with 81 920 pages, 2 to 4 us a kernel; a caller that
// issues them one by one waits longer for its own launches (3 us each).  Doing the children's tables
// inside the fork's cluster instead of in a second launch gained nothing (18.0 of then 18.0, and 31.4 of 30.5).  Only
// spec_page_copy is bound by bandwidth.
#include <cooperative_groups.h>
#include <limits.h>

#include "sv_cache.cuh"
#include "sv_tc.cuh"

namespace cg = cooperative_groups;

namespace svc {

constexpr int PT = 1024;              // threads per bookkeeping CTA
constexpr int PW = PT / 32;
constexpr int PAGES_PER_CTA = 4096;   // cluster CTAs: one per so many pages, at most 8

struct PageState {
    int32_t *len, *table, *ref;
    int B, max_pages, num_pages, page_size;
    int32_t *hdr;
    int32_t *list;      // workspace: num_pages entries
    int32_t *result;    // workspace: B entries (reserve: pages asked for; fork: the child's length, or -1; < 0: an error)
    int32_t *used;      // workspace: pages in use (compact)
};

struct PageWs {
    size_t list, result, used, total;
};
static inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
static inline PageWs page_ws(int B, int num_pages) {
    PageWs L;
    L.used = HEADER;
    L.list = 2 * HEADER;
    L.result = up256(L.list + (size_t)num_pages * 4);
    L.total = up256(L.result + (size_t)B * 4);
    return L;
}

__device__ __forceinline__ int warp_sum(int x) { return __reduce_add_sync(0xffffffffu, x); }

// Inclusive prefix sum over the warp.
template <typename T>
__device__ __forceinline__ T warp_scan(T x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if ((int)(threadIdx.x & 31) >= o) x += y;
    }
    return x;
}

// Exclusive prefix sum over the CTA; *total receives the sum.  tmp: PW + 1 words.
__device__ __forceinline__ long long cta_scan(long long x, long long *tmp, long long *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long inc = warp_scan(x);
    __syncthreads();
    if (lane == 31) tmp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const long long w = tmp[lane];
        const long long s = warp_scan(w);
        tmp[lane] = s - w;
        if (lane == 31) tmp[PW] = s;
    }
    __syncthreads();
    *total = tmp[PW];
    return tmp[warp] + inc - x;
}

// A warp's slice of the pool: [lo, hi), a multiple of 128 pages long except at the pool's end.
struct Slice {
    int lo, hi;
};
__device__ __forceinline__ Slice slice_of(int num_pages, int rank, int nranks) {
    const int warp = rank * PW + (int)(threadIdx.x >> 5), nw = nranks * PW;
    const long long per = (((long long)num_pages + nw - 1) / nw + 127) / 128 * 128;
    Slice s;
    s.lo = (int)min((long long)num_pages, per * warp);
    s.hi = (int)min((long long)num_pages, per * (warp + 1));
    return s;
}

// Bits 0..3: which of the lane's 4 pages at i (within the slice) are in use; `have`: which exist.
__device__ __forceinline__ int used4(const int32_t *ref, int i, int hi, int &have) {
    int v[4] = {0, 0, 0, 0};
    have = 0;
    if (i + 4 <= hi && ((uintptr_t)(ref + i) & 15) == 0) {
        const int4 w = *reinterpret_cast<const int4 *>(ref + i);
        v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
        have = 15;
    } else {
        for (int t = 0; t < 4; t++)
            if (i + t < hi) v[t] = ref[i + t], have |= 1 << t;
    }
    int m = 0;
    for (int t = 0; t < 4; t++) m |= (v[t] != 0) << t;
    return m;
}

// Which pages of a warp's slice are in use: 4 bits a lane for each 128 pages.  The first 1024 pages of
// a slice stay in a register (a pool of 262 144 pages in a cluster of 8), the rest are read again.
struct Used {
    const int32_t *ref;
    Slice s;
    uint32_t head;
    __device__ __forceinline__ void read() {
        head = 0;
        if (((uintptr_t)ref & 15) == 0) {   // (slices begin at multiples of 128: the eight loads go out together)
            int4 w[8];
#pragma unroll
            for (int k = 0; k < 8; k++)
                w[k] = page(k) + 4 <= s.hi ? *reinterpret_cast<const int4 *>(ref + page(k)) : make_int4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 8; k++)
                head |= (uint32_t)((w[k].x != 0) | (w[k].y != 0) << 1 | (w[k].z != 0) << 2 | (w[k].w != 0) << 3) << (4 * k);
        }
#pragma unroll 1
        for (int k = 0; k < 8 && s.lo + 128 * k < s.hi; k++) {   // the pool's last few pages, or an odd base
            int have;
            if (((uintptr_t)ref & 15) || (page(k) < s.hi && page(k) + 4 > s.hi))
                head |= (uint32_t)used4(ref, page(k), s.hi, have) << (4 * k);
        }
    }
    __device__ __forceinline__ int groups() const { return (s.hi - s.lo + 127) / 128; }
    __device__ __forceinline__ int page(int k) const { return s.lo + 128 * k + 4 * (int)(threadIdx.x & 31); }
    // the lane's four pages of group k: in use, and existing
    __device__ __forceinline__ int get(int k, int &have) const {
        const int left = s.hi - page(k);
        have = left >= 4 ? 15 : left > 0 ? (1 << left) - 1 : 0;
        if (k < 8) return head >> (4 * k) & 15;
        return used4(ref, page(k), s.hi, have);
    }
};

// Exclusive prefix of this warp's count over all warps of the cluster, and the total.
// counts: this CTA's PW + 1 shared words.  Contains cluster barriers.
template <typename T>
__device__ __forceinline__ T cluster_prefix(T count, T *counts, T *total) {
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) counts[warp] = count;
    __syncthreads();
    if (warp == 0) {
        const T c = counts[lane];
        const T s = warp_scan(c);
        __syncwarp();
        counts[lane] = s - c;
        if (lane == 31) counts[PW] = s;
    }
    cl.sync();
    T before = 0, all = 0;
    for (unsigned r = 0; r < cl.num_blocks(); r++) {
        const T c = cl.map_shared_rank(counts, r)[PW];
        all += c;
        if (r < cl.block_rank()) before += c;
    }
    *total = all;
    return before + counts[warp];
}

constexpr int NEAR = 2048;   // lists up to this stay in the first CTA's shared memory

// Lists the lowest `want` free pages in ascending order -- in the cluster's first CTA's `near` (NEAR
// entries) if they fit, which saves the fence and the round trip of S.list -- and returns how many free
// pages there are; the list is there for the first CTA on return.
__device__ __forceinline__ int list_free(const PageState &S, const Used &U, long long want, int *counts, int *near) {
    int *const first = cg::this_cluster().map_shared_rank(near, 0);
    const int groups = U.groups();
    int count = 0, have;
    for (int k = 0; k < groups; k++) {
        const int m = U.get(k, have);
        count += __popc(have & ~m);
    }
    int total;
    int at = cluster_prefix(warp_sum(count), counts, &total);
    for (int k = 0; k < groups && at < want; k++) {
        const int m = U.get(k, have);
        const int f = have & ~m, c = __popc(f);
        const int inc = warp_scan(c);
        int r = at + inc - c;
#pragma unroll
        for (int t = 0; t < 4; t++)
            if (f >> t & 1) {
                if (r < want) (want <= NEAR ? first : S.list)[r] = U.page(k) + t;
                r++;
            }
        at += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (want > NEAR) __threadfence();
    cg::this_cluster().sync();
    return total;
}

// ---------------------------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------------------------

// Pages that hold len >= 0 tokens.
__device__ __forceinline__ int pages_of(const PageState &S, int len) {
    return len / S.page_size + (len % S.page_size != 0);
}

struct Want {
    int err, have, grown;
    long long need;
};

// Of request b with k drafts and length len.
__device__ __forceinline__ Want want_of(const PageState &S, int b, int k, int len) {
    Want w = {0, 0, 0, 0};
    if (k == -1) return w;
    const long long grown = (long long)len + k + 1;
    if (k < -1 || len < 0 || grown > (long long)S.max_pages * S.page_size) {
        w.err = SV_DEV_BAD_LAYOUT;
        return w;
    }
    w.have = pages_of(S, len);
    w.grown = (int)grown;
    w.need = (grown + S.page_size - 1) / S.page_size - w.have;
    if (len % S.page_size) {   // the partly filled page: this request's alone
        const int p = S.table[(int64_t)b * S.max_pages + w.have - 1];
        if (p < 0 || p >= S.num_pages) w.err = SV_DEV_BAD_PAGE;
        else if (S.ref[p] != 1) w.err = S.ref[p] > 1 ? SV_DEV_SHARED_PAGE : SV_DEV_BAD_PAGE;
        if (w.err) w.need = 0;
    }
    return w;
}

__global__ void __launch_bounds__(PT) reserve_kernel(const PageState S, const int32_t *nd) {
    __shared__ int places[PT], rows[PT];   // of the requests looked at: their first page in the list and the table
    __shared__ int counts[PW + 1], near[NEAR];
    __shared__ long long tmp[PW + 1];
    grid_wait();
    grid_launch_dependents();
    Used U;
    U.ref = S.ref;
    U.s = slice_of(S.num_pages, cg::this_cluster().block_rank(), cg::this_cluster().num_blocks());
    // the first PT requests are looked at once, their first loads together with the pool's
    const bool in0 = (int)threadIdx.x < S.B;
    const int k0 = in0 ? nd[threadIdx.x] : -1, len0 = in0 ? S.len[threadIdx.x] : 0;
    U.read();
    const Want w0 = want_of(S, threadIdx.x, k0, len0);
    long long sum = w0.need, want = 0;
    const bool decides = cg::this_cluster().block_rank() == 0;
    for (int b = threadIdx.x + PT; b < S.B; b += PT) {
        const Want w = want_of(S, b, nd[b], S.len[b]);
        sum += w.need;
        if (decides) S.result[b] = w.err ? -w.err : (int)w.need;   // (kept: a later look would see pages that this call grants)
    }
    const long long at0 = cta_scan(sum, tmp, &want);   // (of PT requests at most: their places too)
    const long long free = list_free(S, U, want, counts, near);
    if (!decides) return;
    const int32_t *list = want <= NEAR ? near : S.list;
    long long before = 0;
    for (int b0 = 0; b0 < S.B; b0 += PT) {
        const int b = b0 + (int)threadIdx.x;
        const bool in = b < S.B;
        Want w = w0;
        long long at = at0, base = before, total = want;
        if (b0) {
            w = {0, 0, 0, 0};
            if (in && nd[b] != -1) {
                const int r = S.result[b], len = S.len[b];
                if (r < 0) w.err = -r;
                else w = {0, pages_of(S, len), len + nd[b] + 1, r};
            }
        }
        if (S.B > PT) {
            long long all;
            at = before + cta_scan(w.need, tmp, &all);
            before += all;
            total = all;
        }
        if (w.need > 0 && at + w.need > free) {
            w.err = SV_DEV_NO_PAGES;
            w.need = 0;
        }
        if (in && w.err) {
            record_error(S.hdr, w.err, b);
            if (S.len[b] >= 0) S.len[b] = -1 - S.len[b];
        } else if (in && nd[b] >= 0) {
            S.len[b] = w.grown;
        }
        int32_t *row = S.table + (int64_t)b * S.max_pages + w.have;
        const int small = w.need <= 4 ? (int)w.need : 0;
        for (int i = 0; i < small; i++) {
            const int p = list[at + i];
            row[i] = p;
            S.ref[p] = 1;
        }
        // longer ones (a prompt's pages) by the whole CTA, a page a thread: the list's i-th page is the last
        // request's whose place is at or before i (8 prompts of 8192 pages by a warp each: 530 us)
        places[threadIdx.x] = (int)(at - base);
        rows[threadIdx.x] = w.need > 4 ? w.have : -1;
        const int end = (int)max(min(total, free - base), 0ll);   // (what is granted ends before the free pages do)
        if (__syncthreads_or(w.need > 4)) {
#pragma unroll 2
            for (int i = threadIdx.x; i < end; i += PT) {
                int r = 0;
#pragma unroll
                for (int step = PT / 2; step; step >>= 1)
                    if (places[r + step] <= i) r += step;
                if (rows[r] < 0) continue;
                const int p = list[base + i];
                S.table[(int64_t)(b0 + r) * S.max_pages + rows[r] + (i - places[r])] = p;
                S.ref[p] = 1;
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------------------------------------
// rollback
// ---------------------------------------------------------------------------------------------

constexpr int BT = 256;

// One pass over three words a request: bound by the launch.
__global__ void __launch_bounds__(BT) rollback_kernel(int32_t *len, const int32_t *accept, const int32_t *nd, int B,
                                                      int32_t *hdr) {
    grid_wait();
    grid_launch_dependents();
    const int b = blockIdx.x * BT + (int)threadIdx.x;
    if (b >= B) return;
    const int k = nd[b], a = accept[b], L = len[b];
    if (k == -1) return;
    const long long kept = (long long)L - k + a;
    if (k < 0 || a < 0 || a > k || kept < 0) record_error(hdr, SV_DEV_BAD_LAYOUT, b);   // (kept <= L: a <= k)
    else len[b] = (int)kept;
}

// ---------------------------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------------------------

struct ForkArgs {
    const int32_t *parents, *children, *fork_len;   // fork_len may be NULL
    int32_t *src, *dst;
    int F;
};

// The error of a fork of n tokens of p (or all) to c as the state was before the call, its length and its
// partly filled page.
__device__ __forceinline__ int fork_check(const PageState &S, int p, int c, bool all, int &n, int &tail) {
    tail = -1;
    if (p < 0 || p >= S.B || c < 0 || c >= S.B || S.len[c] != 0) return SV_DEV_BAD_LAYOUT;
    const int len = S.len[p];
    if (all) n = len;
    if (n < 1 || n > len || (long long)n > (long long)S.max_pages * S.page_size) return SV_DEV_BAD_LAYOUT;
    if (n % S.page_size) {
        tail = S.table[(int64_t)p * S.max_pages + n / S.page_size];
        if (tail < 0 || tail >= S.num_pages || S.ref[tail] < 1) return SV_DEV_BAD_PAGE;
    }
    return 0;
}

// Decides every fork, takes the fresh pages and sets the children's lengths (fork_share does the
// tables).  An empty child goes to the lowest f that names it: that f's claim is the smallest
// value INT_MIN + f left in its length.
__global__ void __launch_bounds__(PT) fork_kernel(const PageState S, const ForkArgs K) {
    __shared__ int counts[PW + 1], near[NEAR];
    __shared__ long long tmp[PW + 1];
    grid_wait();
    grid_launch_dependents();
    Used U;
    U.ref = S.ref;
    U.s = slice_of(S.num_pages, cg::this_cluster().block_rank(), cg::this_cluster().num_blocks());
    // the first PT forks' first loads go out together with the pool's
    int p = -1, c = -1, len = 0;
    auto load = [&](int f) { p = K.parents[f], c = K.children[f], len = K.fork_len ? K.fork_len[f] : 0; };
    const bool decides = cg::this_cluster().block_rank() == 0;
    if (decides && (int)threadIdx.x < K.F) load(threadIdx.x);
    U.read();
    if (decides) {
        for (int f = threadIdx.x; f < K.F; f += PT) {
            if (f >= PT) load(f);
            int n = len, tail;
            const int err = fork_check(S, p, c, !K.fork_len, n, tail);
            const bool claims = c >= 0 && c < S.B && S.len[c] == 0;
            S.result[f] = err ? -err : n;
            K.src[f] = tail;
            K.dst[f] = claims ? 1 : 0;
        }
        __syncthreads();   // every length is read before one changes
        for (int f = threadIdx.x; f < K.F; f += PT)
            if (K.dst[f]) atomicMin(S.len + K.children[f], INT_MIN + f);
    }
    const int free = list_free(S, U, K.F, counts, near);   // (and a barrier: every claim is made)
    if (cg::this_cluster().block_rank() != 0) return;
    const int32_t *list = K.F <= NEAR ? near : S.list;
    long long before = 0;
    for (int f0 = 0; f0 < K.F; f0 += PT) {
        const int f = f0 + (int)threadIdx.x;
        const bool in = f < K.F;
        int n = 0, tail = -1, err = 0;
        bool mine = false;
        if (in) {
            n = S.result[f];
            err = n < 0 ? -n : 0;
            tail = K.src[f];
            mine = K.dst[f] && __ldcg(S.len + K.children[f]) == INT_MIN + f;
            if (!mine && !err) err = SV_DEV_BAD_LAYOUT;
        }
        const int need = (in && !err && tail >= 0) ? 1 : 0;
        long long all;
        const long long at = before + cta_scan(need, tmp, &all);
        before += all;
        int fresh = -1;
        if (need) {
            if (at >= free) err = SV_DEV_NO_PAGES;
            else fresh = list[at];
        }
        if (in) {
            if (err) record_error(S.hdr, err, f);
            if (mine) S.len[K.children[f]] = err ? -1 : n;
            if (fresh >= 0) S.ref[fresh] = 1;
            S.result[f] = err ? -1 : n;
            K.src[f] = fresh >= 0 ? tail : -1;
            K.dst[f] = fresh;
        }
    }
    __syncthreads();   // (the list has been read)
    for (int f = threadIdx.x; f < K.F; f += PT) {   // list[page taken] = the fork that took it, for fork_share
        const int fresh = K.dst[f];
        if (fresh >= 0) S.list[fresh] = f;
    }
}

constexpr int ST = 256, SPT = 4;   // threads per CTA, table entries per thread

// The children's tables, and a count more for each shared page.  A page that no request held before the
// call is not shared: its count is 0, which nothing here changes, or 1 because fork_kernel took it, which
// its entry of the list tells (whatever else the list holds there names no fork that took it).
__global__ void __launch_bounds__(ST) fork_share(const PageState S, const ForkArgs K) {
    grid_wait();
    grid_launch_dependents();
    const int f = blockIdx.x;
    const int n = S.result[f];
    if (n < 0) return;
    const int32_t *from = S.table + (int64_t)K.parents[f] * S.max_pages;
    int32_t *to = S.table + (int64_t)K.children[f] * S.max_pages;
    const int full = n / S.page_size, fresh = K.dst[f];
    int p[SPT], count[SPT], taker[SPT];
    const int j0 = blockIdx.y * SPT * ST + threadIdx.x;
#pragma unroll
    for (int t = 0; t < SPT; t++) {
        const int j = j0 + t * ST;
        p[t] = j < full ? from[j] : -1;
    }
#pragma unroll
    for (int t = 0; t < SPT; t++) {
        const bool is = p[t] >= 0 && p[t] < S.num_pages;
        count[t] = is ? __ldcg(S.ref + p[t]) : 0;
        taker[t] = is ? S.list[p[t]] : -1;
    }
#pragma unroll
    for (int t = 0; t < SPT; t++) {
        const int j = j0 + t * ST;
        if (j >= S.max_pages) break;
        if (count[t] > 0 && !(taker[t] >= 0 && taker[t] < K.F && K.dst[taker[t]] == p[t])) {
            atomicAdd(S.ref + p[t], 1);
        } else if (p[t] != -1) {   // not a page, or one that no request holds
            record_error(S.hdr, SV_DEV_BAD_PAGE, f);
            p[t] = -1;
        }
        to[j] = j == full ? fresh : p[t];
    }
}

// ---------------------------------------------------------------------------------------------
// release
// ---------------------------------------------------------------------------------------------

constexpr int RELEASE_CTAS = 16;   // per request at most
// Rows of up to so many entries are read 4 at a time by each thread, longer ones 16: 8 and 512 requests of
// 2048 entries take 1.5 and 2.3 us with 4, 1.6 and 2.2 with 16; of 8192 entries 1.4 and 5.2, and 1.7 and 3.3.
constexpr int RELEASE_NARROW = 2048;

// Gives back every entry past the request's length and, with a window, every one of pages that no later
// row sees.  Where a row's held entries end cannot be told from a part of it: releases under a window leave
// a gap of any width between the first tokens' pages and the window's, and the gap lies past the length once
// the request has ended.  So every entry outside what stays is read.  512 running requests with nothing to
// give back take 1.8 us for rows of 1024 entries, 3.3 for 8192 and 21 for 65 536 (134 MB, 6.5 TB/s).
template <int N>   // table entries per thread and step
__global__ void __launch_bounds__(ST) release_kernel(const PageState S, int window, int sinks) {
    grid_wait();
    grid_launch_dependents();
    const int b = blockIdx.x;
    const int len = S.len[b];
    if (len < 0) return;
    int32_t *row = S.table + (int64_t)b * S.max_pages;
    const int keep = pages_of(S, len);
    if (keep > S.max_pages) {
        if (threadIdx.x == 0 && blockIdx.y == 0) record_error(S.hdr, SV_DEV_BAD_LAYOUT, b);
        return;
    }
    // pages [from, to): all tokens >= sinks and <= len - window
    int from = 0, to = 0;
    if (window) {
        const long long gone = (long long)len - window + 1;
        from = sinks / S.page_size + (sinks % S.page_size != 0);
        to = gone > 0 ? (int)(gone / S.page_size) : 0;
    }
    for (int i0 = blockIdx.y * ST * N; i0 < S.max_pages; i0 += gridDim.y * ST * N) {
        const int first = i0 + (int)threadIdx.x;
        int p[N];
        bool any = false;
#pragma unroll
        for (int t = 0; t < N; t++) {
            const int i = first + t * ST;
            p[t] = i < S.max_pages && (i >= keep || (i >= from && i < to)) ? row[i] : -1;
        }
#pragma unroll
        for (int t = 0; t < N; t++) any |= p[t] != -1;
        if (!any) continue;
#pragma unroll
        for (int t0 = 0; t0 < N; t0 += 4) {
            int count[4];
#pragma unroll
            for (int t = 0; t < 4; t++) {
                const int page = p[t0 + t];
                count[t] = 1;
                if (page == -1) continue;
                row[first + (t0 + t) * ST] = -1;
                count[t] = page >= 0 && page < S.num_pages ? atomicSub(S.ref + page, 1) : 0;
            }
#pragma unroll
            for (int t = 0; t < 4; t++)
                if (count[t] < 1) {   // not a page, or one that no request holds
                    const int page = p[t0 + t];
                    if (page >= 0 && page < S.num_pages) atomicAdd(S.ref + page, 1);
                    record_error(S.hdr, SV_DEV_BAD_PAGE, b);
                }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------------------------

// The r-th used page at or above U (pages in use) pairs with the r-th free page below U; there
// are equally many.  S.list becomes the map from page to page for ids >= U.
__global__ void __launch_bounds__(PT) compact_kernel(const PageState S, int32_t *src, int32_t *dst, int cap) {
    __shared__ int counts[PW + 1];
    __shared__ long long counts2[PW + 1];
    grid_wait();
    grid_launch_dependents();
    cg::cluster_group cl = cg::this_cluster();
    Used P;
    P.ref = S.ref;
    P.s = slice_of(S.num_pages, cl.block_rank(), cl.num_blocks());
    P.read();
    const int groups = P.groups();
    int count = 0, have, U;
    for (int k = 0; k < groups; k++) count += __popc(P.get(k, have));
    cluster_prefix(warp_sum(count), counts, &U);
    auto below = [&](int i) { return U <= i ? 0 : (U >= i + 4 ? 15 : (1 << (U - i)) - 1); };   // ids < U of i .. i + 3
    int up = 0, down = 0;
    for (int k = 0; k < groups; k++) {
        const int m = P.get(k, have), lo = below(P.page(k));
        up += __popc(m & ~lo);
        down += __popc(have & ~m & lo);
    }
    long long both;   // movers in the low half, holes in the high half
    const long long at = cluster_prefix((long long)warp_sum(up) | (long long)warp_sum(down) << 32, counts2, &both);
    int at_up = (int)at, at_down = (int)(at >> 32);
    const int moves = (int)both;
    for (int k = 0; k < groups; k++) {
        const int i = P.page(k), m = P.get(k, have), lo = below(i);
        const int fu = m & ~lo, fd = have & ~m & lo, free_above = have & ~m & ~lo;
        const int iu = warp_scan(__popc(fu)), id = warp_scan(__popc(fd));
        int ru = at_up + iu - __popc(fu), rd = at_down + id - __popc(fd);
#pragma unroll
        for (int t = 0; t < 4; t++) {
            if (fu >> t & 1) {
                if (ru < cap) src[ru] = i + t;
                else S.list[i + t] = i + t;   // past the capacity: stays
                ru++;
            }
            if (fd >> t & 1) {
                if (rd < cap) dst[rd] = i + t;
                rd++;
            }
            if (free_above >> t & 1) S.list[i + t] = i + t;
        }
        at_up += __shfl_sync(0xffffffffu, iu, 31);
        at_down += __shfl_sync(0xffffffffu, id, 31);
    }
    __threadfence();
    cl.sync();
    const int n = min(moves, cap), step = cl.num_blocks() * PT;
    for (int r = cl.block_rank() * PT + threadIdx.x; r < cap; r += step) {
        if (r < n) {
            const int a = __ldcg(src + r), d = __ldcg(dst + r);
            S.ref[d] = S.ref[a];
            S.ref[a] = 0;
            S.list[a] = d;
        } else {
            src[r] = dst[r] = -1;
        }
    }
    if (cl.block_rank() == 0 && threadIdx.x == 0) *S.used = U;
    cl.sync();   // no CTA leaves while another may still read its counts
}

__global__ void __launch_bounds__(ST) remap_kernel(const PageState S) {
    grid_wait();
    grid_launch_dependents();
    const int U = *S.used;
    const long long total = (long long)S.B * S.max_pages;
    for (long long j = (long long)blockIdx.x * ST + threadIdx.x; j < total; j += (long long)gridDim.x * ST) {
        const int p = S.table[j];
        if (p < U) continue;
        const int to = p < S.num_pages ? S.list[p] : p;
        if (p >= S.num_pages || (to == p && S.ref[p] == 0)) record_error(S.hdr, SV_DEV_BAD_PAGE, (int)(j / S.max_pages));
        else S.table[j] = to;
    }
}

// ---------------------------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------------------------

struct CopyArgs {
    char *k, *v;
    const int32_t *src, *dst;
    int64_t page_bytes, page_stride, layer_stride;
    int32_t *hdr;
    int num_pages, layers, n;
};

constexpr int CT = 256, CU = 4;   // threads per CTA, 16-byte loads in flight per thread

// An item is one pair in one layer's keys or values; a CTA takes every gridDim.x-th, and looks up 256 of
// them at once, so that the pairs' latency is paid once and an absent pair costs next to nothing.
// Bound by the memory: 16 KB pages move at 6.6 TB/s read and write together, 8 CTAs an SM.
__global__ void __launch_bounds__(CT) copy_kernel(const CopyArgs A) {
    __shared__ int2 pairs[CT];
    grid_wait();
    grid_launch_dependents();
    const long long per_pair = (long long)A.layers * (A.v ? 2 : 1), items = per_pair * A.n;
    const int words = (int)(A.page_bytes / 16);
    for (long long base = blockIdx.x; base < items; base += (long long)CT * gridDim.x) {
        const long long mine = base + (long long)threadIdx.x * gridDim.x;
        int2 x = make_int2(-1, -1);
        if (mine < items) {
            const int i = (int)(mine / per_pair);
            x = make_int2(A.src[i], A.dst[i]);
            if (x.x < 0 || x.y < 0) {
                x.x = -1;
            } else if (x.x >= A.num_pages || x.y >= A.num_pages) {
                record_error(A.hdr, SV_DEV_BAD_PAGE, i);
                x.x = -1;
            }
        }
        __syncthreads();
        pairs[threadIdx.x] = x;
        __syncthreads();
        const int count = (int)min((long long)CT, (items - base + gridDim.x - 1) / gridDim.x);
        for (int j = 0; j < count; j++) {
            const int2 p = pairs[j];
            if (p.x < 0) continue;
            const int part = (int)((base + (long long)j * gridDim.x) % per_pair);
            char *at = (part >= A.layers ? A.v : A.k) + (part >= A.layers ? part - A.layers : part) * A.layer_stride;
            const uint4 *from = reinterpret_cast<const uint4 *>(at + p.x * A.page_stride);
            uint4 *to = reinterpret_cast<uint4 *>(at + p.y * A.page_stride);
            for (int w0 = threadIdx.x; w0 < words; w0 += CT * CU) {
                uint4 v[CU];
#pragma unroll
                for (int u = 0; u < CU; u++)
                    if (w0 + u * CT < words) v[u] = __ldcs(from + w0 + u * CT);
#pragma unroll
                for (int u = 0; u < CU; u++)
                    if (w0 + u * CT < words) __stcs(to + w0 + u * CT, v[u]);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------------

static sv_status check_pages(int32_t B, const void *table, int32_t max_pages, const void *ref, int32_t num_pages,
                             int32_t page_size, const void *ws) {
    if (B < 1 || max_pages < 1 || num_pages < 1 || page_size < 1 || !table || !ref || !ws) return SV_ERR_INVALID_ARG;
    if (B >= MAXB || max_pages > (1 << 20) || num_pages >= (1 << 28) || (long long)B * max_pages >= (1ll << 40) ||
        (long long)max_pages * page_size > 0x7fffffffll)
        return SV_ERR_UNSUPPORTED;
    if ((uintptr_t)ws & 255) return SV_ERR_WORKSPACE;
    return SV_OK;
}

static PageState page_state(int32_t *len, int32_t B, int32_t *table, int32_t max_pages, int32_t *ref,
                            int32_t num_pages, int32_t page_size, void *ws) {
    const PageWs L = page_ws(B, num_pages);
    char *w = static_cast<char *>(ws);
    return PageState{len, table, ref, B, max_pages, num_pages, page_size, reinterpret_cast<int32_t *>(w),
                     reinterpret_cast<int32_t *>(w + L.list), reinterpret_cast<int32_t *>(w + L.result),
                     reinterpret_cast<int32_t *>(w + L.used)};
}

// A bookkeeping kernel as one cluster.
template <typename... P, typename... A>
static cudaError_t launch_cluster(void (*kernel)(P...), int num_pages, cudaStream_t st, A... args) {
    int ctas = 1;
    while (ctas < 8 && (long long)ctas * PAGES_PER_CTA < num_pages) ctas *= 2;
    return launch_dependent(kernel, dim3(ctas), dim3(PT), ctas, st, args...);
}

}  // namespace svc

using namespace svc;

extern "C" size_t sv_page_workspace_bytes(int32_t B, int32_t num_pages) {
    if (B < 1 || num_pages < 1 || B >= MAXB || num_pages >= (1 << 28)) return 0;
    return page_ws(B, num_pages).total;
}

extern "C" sv_status spec_page_reserve(const int32_t *num_drafts, int32_t *kv_seq_len, int32_t B,
                                       int32_t *block_table, int32_t max_pages, int32_t *ref_count, int32_t num_pages,
                                       int32_t page_size, void *workspace, size_t workspace_bytes, void *stream) {
    const sv_status bad = check_pages(B, block_table, max_pages, ref_count, num_pages, page_size, workspace);
    if (bad != SV_OK) return bad;
    if (!num_drafts || !kv_seq_len) return SV_ERR_INVALID_ARG;
    if (workspace_bytes < page_ws(B, num_pages).total) return SV_ERR_WORKSPACE;
    const PageState S = page_state(kv_seq_len, B, block_table, max_pages, ref_count, num_pages, page_size, workspace);
    return launch_cluster(reserve_kernel, num_pages, static_cast<cudaStream_t>(stream), S, num_drafts) == cudaSuccess
               ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status spec_cache_rollback(int32_t *kv_seq_len, const int32_t *accept_len, const int32_t *num_drafts,
                                         int32_t B, void *workspace, void *stream) {
    if (B < 1 || !kv_seq_len || !accept_len || !num_drafts || !workspace) return SV_ERR_INVALID_ARG;
    if (B >= MAXB) return SV_ERR_UNSUPPORTED;
    if ((uintptr_t)workspace & 255) return SV_ERR_WORKSPACE;
    return launch_dependent(rollback_kernel, dim3((B + BT - 1) / BT), dim3(BT), 1, static_cast<cudaStream_t>(stream), kv_seq_len,
                            accept_len, num_drafts, (int)B, static_cast<int32_t *>(workspace)) == cudaSuccess
               ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status spec_page_fork(const int32_t *parents, const int32_t *children, const int32_t *fork_len,
                                    int32_t num_forks, int32_t *kv_seq_len, int32_t B, int32_t *block_table,
                                    int32_t max_pages, int32_t *ref_count, int32_t num_pages, int32_t page_size,
                                    int32_t *copy_src, int32_t *copy_dst, void *workspace, size_t workspace_bytes,
                                    void *stream) {
    const sv_status bad = check_pages(B, block_table, max_pages, ref_count, num_pages, page_size, workspace);
    if (bad != SV_OK) return bad;
    if (!kv_seq_len || num_forks < 1 || !parents || !children || !copy_src || !copy_dst) return SV_ERR_INVALID_ARG;
    if (num_forks > B) return SV_ERR_UNSUPPORTED;
    if (workspace_bytes < page_ws(B, num_pages).total) return SV_ERR_WORKSPACE;
    const PageState S = page_state(kv_seq_len, B, block_table, max_pages, ref_count, num_pages, page_size, workspace);
    const ForkArgs K{parents, children, fork_len, copy_src, copy_dst, num_forks};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_cluster(fork_kernel, num_pages, st, S, K) != cudaSuccess) return SV_ERR_CUDA;
    return launch_dependent(fork_share, dim3(num_forks, (max_pages + ST * SPT - 1) / (ST * SPT)), dim3(ST), 1, st, S, K) ==
                   cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status spec_page_release(const int32_t *kv_seq_len, int32_t B, int32_t *block_table, int32_t max_pages,
                                       int32_t *ref_count, int32_t num_pages, int32_t page_size, int32_t window,
                                       int32_t sinks, void *workspace, void *stream) {
    const sv_status bad = check_pages(B, block_table, max_pages, ref_count, num_pages, page_size, workspace);
    if (bad != SV_OK) return bad;
    if (!kv_seq_len || window < 0 || sinks < 0) return SV_ERR_INVALID_ARG;
    const PageState S = page_state(const_cast<int32_t *>(kv_seq_len), B, block_table, max_pages, ref_count, num_pages,
                                   page_size, workspace);
    const int per_thread = max_pages <= RELEASE_NARROW ? 4 : 16, chunks = (max_pages + ST * per_thread - 1) / (ST * per_thread);
    return launch_dependent(per_thread == 4 ? release_kernel<4> : release_kernel<16>,
                            dim3(B, chunks < RELEASE_CTAS ? chunks : RELEASE_CTAS), dim3(ST), 1,
                            static_cast<cudaStream_t>(stream), S, window, sinks) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status spec_page_compact(int32_t B, int32_t *block_table, int32_t max_pages, int32_t *ref_count,
                                       int32_t num_pages, int32_t *copy_src, int32_t *copy_dst, int32_t capacity,
                                       void *workspace, size_t workspace_bytes, void *stream) {
    const sv_status bad = check_pages(B, block_table, max_pages, ref_count, num_pages, 1, workspace);
    if (bad != SV_OK) return bad;
    if (capacity < 1 || !copy_src || !copy_dst) return SV_ERR_INVALID_ARG;
    if (workspace_bytes < page_ws(B, num_pages).total) return SV_ERR_WORKSPACE;
    const PageState S = page_state(nullptr, B, block_table, max_pages, ref_count, num_pages, 1, workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_cluster(compact_kernel, num_pages, st, S, copy_src, copy_dst, capacity) != cudaSuccess)
        return SV_ERR_CUDA;
    const long long blocks = ((long long)B * max_pages + ST * 4 - 1) / (ST * 4);
    return launch_dependent(remap_kernel, dim3((unsigned)(blocks < 1216 ? blocks : 1216)), dim3(ST), 1, st, S) == cudaSuccess
               ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status spec_page_copy(void *k, void *v, int64_t page_bytes, int64_t page_stride, int32_t num_layers,
                                    int64_t layer_stride, int32_t num_pages, const int32_t *copy_src,
                                    const int32_t *copy_dst, int32_t n, void *workspace, void *stream) {
    if (!k || !copy_src || !copy_dst || !workspace || n < 1 || num_pages < 1 || num_layers < 1 || page_bytes < 1 ||
        page_stride < page_bytes || layer_stride < 0 || (num_layers > 1 && layer_stride == 0))
        return SV_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || (page_bytes | page_stride | layer_stride) % 16 || page_bytes > (1ll << 34))
        return SV_ERR_UNSUPPORTED;
    if ((uintptr_t)workspace & 255) return SV_ERR_WORKSPACE;
    const CopyArgs A{static_cast<char *>(k), static_cast<char *>(v), copy_src, copy_dst, page_bytes, page_stride,
                     layer_stride, static_cast<int32_t *>(workspace), num_pages, num_layers, n};
    const long long items = (long long)n * num_layers * (v ? 2 : 1);
    return launch_dependent(copy_kernel, dim3((unsigned)(items < 1216 ? items : 1216)), dim3(CT), 1,
                            static_cast<cudaStream_t>(stream), A) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
