// cache_attention.cu -- spec_attention: the new tokens' rows attend over the paged cache under a
// causal mask with an optional sliding window and first tokens that stay visible.
//
// One pass over the keys with the running maximum m and sum l of the softmax: for each tile of 128
// tokens S = Q K^T, p = 2^(c S - c m), O += p V, l += sum p, with c = scale log2(e); a part's result
// is (O / l, m, l), and parts join by their log-sums.
//
// Query rows.  The n rows of a request and the G query heads of one key/value head share every key,
// so M = n G rows make one tile of up to 128, or two of 128 (256 rows in all) that share each loaded
// tile of keys; more rows make more row tiles.  Keys and values are then read once per 256 rows,
// and the products run on the tensor cores whatever M is: the padded rows cost nothing that the
// load of a key tile (64 KB, 1.5 us of one SM's share of the memory) does not hide.
//
// Work.  The unit of work is one key tile of one (request, key head, row tile).  All units of the
// batch, in that order, are cut into one equal range per CTA, from the lengths on the device: ragged
// batches, one long request and windows need no other schedule.  A row tile whose keys lie in several
// CTAs' ranges leaves a part per CTA in the workspace, and the second kernel joins them in order.
//
// A CTA: one producer warp (tensor copies of pages into a ring of K and V tiles), one warp that
// issues the matrix instructions (S and O in tensor memory, P back in tensor memory as an operand),
// and two groups of 4 warps, a thread per row, for softmax and epilogue.  With one row tile the
// groups take alternate key tiles, each with its own m, l and O, joined at the end; with two, each
// has its own.
#include <math.h>

#include <atomic>

#include "sv_cache.cuh"
#include "sv_tc.cuh"

namespace svc {

constexpr int TILE = 128;                // tokens per key tile, rows per row tile
constexpr int BLK = TILE * 128;          // bytes of 128 rows x 64 elements
constexpr int NTHREADS = 320;            // 2 x 4 softmax warps, producer, matrix issue
constexpr int W_LOAD = 8, W_MMA = 9;
constexpr int MAX_CTAS = 160;
constexpr int PART_ROWS = 256;           // rows of a part
constexpr int MAX_STAGES = 14;

struct AttnArgs {
    const void *q;
    int64_t q_stride;
    void *out;
    float *lse;
    int32_t *hdr;
    int4 *desc;        // workspace, per CTA: the row tile whose first part, but not last, it holds
    float *part_lse;   // workspace, [2 * MAX_CTAS][PART_ROWS]: log2 of the part's sum
    float *part_o;     // workspace, [2 * MAX_CTAS][DP / 4][PART_ROWS][4]
    float c;           // |scale| log2(e)
    uint32_t qflip;    // sign flip of two queries (scale < 0)
    int qzero;         // scale == 0
    int Hq, G, window, sinks, q_tiles, stages;
};

struct AttnWs {
    size_t desc, lse, o, total;
};
__host__ __device__ inline AttnWs attn_ws(int D) {
    AttnWs L;
    L.desc = HEADER;
    L.lse = L.desc + MAX_CTAS * sizeof(int4);
    L.o = L.lse + (size_t)2 * MAX_CTAS * PART_ROWS * 4;
    L.total = L.o + (size_t)2 * MAX_CTAS * PART_ROWS * (D <= 64 ? 64 : 128) * 4;
    return L;
}

// What a request asks of the kernel.
struct Req {
    int row0, n, len, M, mt;   // rows n, M = n G of them per key head in mt row tiles
    int lo;                    // first token that the window leaves to any row
    int w0, ns, nt;            // first window tile, sink tiles before it, tiles in all
};

__device__ __forceinline__ Req req_of(const Batch &A, const Cache &C, const AttnArgs &P, int b) {
    const Span s = span_of(A, C.max_pages << C.page_shift, b);
    Req r;
    r.row0 = s.row0;
    r.n = s.n;
    r.len = s.len;
    r.M = s.n * P.G;
    r.mt = r.M <= TILE ? 1 : (r.M + 2 * TILE - 1) / (2 * TILE);
    r.lo = P.window ? max(0, s.len - s.n - P.window + 1) : 0;
    r.w0 = r.lo / TILE;
    r.ns = P.window ? min((min(P.sinks, s.len) + TILE - 1) / TILE, r.w0) : 0;
    r.nt = s.n ? r.ns + (s.len + TILE - 1) / TILE - r.w0 : 0;
    return r;
}
__device__ __forceinline__ long long units_of(const Req &r, int heads) { return (long long)r.nt * r.mt * heads; }

// A CTA's share of one row tile: key tiles [t0, t1) of [0, nt).
struct Seg : Req {
    int b, kvh, m, t0, t1;
    long long first;   // global index of the row tile's first unit
    __device__ __forceinline__ int base(int t) const { return (t < ns ? t : w0 + t - ns) * TILE; }
    __device__ __forceinline__ bool two() const { return M > TILE; }
};

// Walks over a CTA's range of units.  Every role walks by itself.
struct Walk {
    long long pos, hi, pre;   // next unit, end, units before request b
    int b;
    Req r;
    __device__ __forceinline__ bool next(const Batch &A, const Cache &C, const AttnArgs &P, Seg &s) {
        if (pos >= hi) return false;
        long long w = units_of(r, C.heads);
        while (pos >= pre + w) {
            pre += w;
            b++;
            r = req_of(A, C, P, b);
            w = units_of(r, C.heads);
        }
        const int u = (int)((pos - pre) / r.nt);   // row tile within the request
        s.row0 = r.row0, s.n = r.n, s.len = r.len, s.M = r.M, s.mt = r.mt, s.lo = r.lo, s.w0 = r.w0, s.ns = r.ns;
        s.nt = r.nt;
        s.b = b;
        s.kvh = u / r.mt;
        s.m = u % r.mt;
        s.first = pre + (long long)u * r.nt;
        s.t0 = (int)(pos - s.first);
        s.t1 = (int)min((long long)r.nt, hi - s.first);
        pos = s.first + s.t1;
        return true;
    }
};

// Whether the row at position pos sees token j.
__device__ __forceinline__ bool sees(const AttnArgs &P, int pos, int j) {
    return j <= pos && (!P.window || j > pos - P.window || j < P.sinks);
}
// The same for tokens j .. j + 31, a bit each.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t seen_mask(const AttnArgs &P, int pos, int j) {
    uint32_t m = low_bits(pos + 1 - j);
    if (P.window) m &= ~low_bits(pos - P.window + 1 - j) | low_bits(P.sinks - j);
    return m;
}
__device__ __forceinline__ bool seen_by_all(const AttnArgs &P, const Req &s, int j) {
    return j <= s.len - s.n && (!P.window || j > s.len - 1 - P.window || j < P.sinks);
}
__device__ __forceinline__ bool seen_by_any(const AttnArgs &P, const Req &s, int j) {
    return j < s.len && (j >= s.lo || j < P.sinks);
}
// Whether every row sees all 128 tokens from base on.
__device__ __forceinline__ bool whole_tile(const AttnArgs &P, const Req &s, int base) {
    return base + TILE - 1 <= s.len - s.n && (!P.window || base > s.len - 1 - P.window || base + TILE - 1 < P.sinks);
}

// Places in the ring of a row tile's K and V tiles, in the order they are used: K0, K1, V0, K2, V1, ...
__device__ __forceinline__ uint32_t k_item(int t) { return t ? 2 * t - 1 : 0; }
__device__ __forceinline__ uint32_t v_item(int t, int nt) { return t < nt - 1 ? 2 * t + 2 : 2 * t + 1; }

struct Ring {
    uint32_t base, full, empty;   // shared addresses: tiles, barriers
    uint32_t count;               // items before the current row tile
    int stages;
    uint32_t stage, phase;
    __device__ __forceinline__ void at(uint32_t item) {
        const uint32_t i = count + item, round = i / stages;
        stage = i - round * stages;
        phase = round & 1;
    }
};

template <typename E>
__device__ __forceinline__ bool finite16(uint32_t h) {
    const uint32_t ex = sizeof(E) == 2 && Num<E>::BF16 ? 0x7f80u : 0x7c00u;
    return (h & ex) != ex;
}

// Tokens of a boundary tile whose value must not reach the product as it is: thread `tok` of a group
// clears a value row that no row sees (a slot never written may hold NaN, and 0 * NaN is NaN), and
// the non-finite elements of one that only some rows see (the epilogue gives those to the rows that
// do).  Returns whether it took any of the latter.
template <typename E, int DP>
__device__ __forceinline__ bool clean_values(const AttnArgs &P, const Req &s, int base, int tok, char *tile) {
    const int j = base + tok;
    if (seen_by_all(P, s, j)) return false;
    const bool any = seen_by_any(P, s, j);
    bool took = false;
    for (int blk = 0; blk < DP / 64; blk++) {
        uint4 *row = reinterpret_cast<uint4 *>(tile + blk * BLK + tok * 128);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if (!any) {
                row[i] = make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            uint4 w = row[i];
            uint32_t *p = &w.x;
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if (!finite16<E>(p[e] & 0xffffu)) p[e] &= 0xffff0000u, hit = true;
                if (!finite16<E>(p[e] >> 16)) p[e] &= 0xffffu, hit = true;
            }
            if (hit) row[i] = w, took = true;
        }
    }
    return took;
}

// The non-finite elements that clean_values took, for the row at position pos: columns
// [col, col + 16) of the tokens in this segment that the row sees and another does not.
template <typename E>
__device__ __noinline__ void add_non_finite(const Cache &C, const AttnArgs &P, const Seg &s, int pos, int col, float *o) {
    for (int side = 0; side < 2; side++) {
        const int from = side ? s.lo : s.len - s.n + 1, to = side ? min(s.len, s.lo + s.n - 1) : s.len;
        for (int j = from; j < to; j++) {
            if (side && (!P.window || j > s.len - s.n)) break;   // (the causal side has it)
            const int tile = j / TILE, t = tile >= s.w0 ? tile - s.w0 + s.ns : tile;
            if (t < s.t0 || t >= s.t1 || seen_by_all(P, s, j) || !sees(P, pos, j)) continue;
            const int page = __ldg(C.table + (int64_t)s.b * C.max_pages + (j >> C.page_shift));
            if (page < 0 || page >= C.num_pages) continue;
            const E *v = static_cast<const E *>(C.v) + page * C.page_stride +
                         (j & ((1 << C.page_shift) - 1)) * C.token_stride + s.kvh * C.head_stride;
            for (int i = 0; i < 16 && col + i < C.D; i++) {
                const float x = (float)v[col + i];
                if (!(fabsf(x) < INFINITY)) o[i] += x;
            }
        }
    }
}

// Barrier of the 256 softmax threads; whether any of them passed true.
__device__ __forceinline__ bool softmax_barrier_or(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "tcgen05.fence::before_thread_sync;\n\t"
        "barrier.cta.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((uint32_t)x) : "memory");
    return r != 0;
}

template <typename E, int DP>
__global__ void __launch_bounds__(NTHREADS, 1)
attention_kernel(const Batch A, const Cache C, const AttnArgs P, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v) {
    constexpr int NB = DP / 64, STAGE = NB * BLK;
    // weights are held times 2^BIAS: half precision then keeps 22 bits below the largest one
    constexpr float BIAS = Num<E>::BF16 ? 0.f : 8.f;
    // the running maximum may lag by this many powers of two before O is scaled down
    constexpr float LAG = Num<E>::BF16 ? 8.f : 6.f;
    extern __shared__ __align__(1024) char smem[];
    // [Q tiles][ring][barriers and small state]
    char *const ring_p = smem + P.q_tiles * STAGE;
    char *const small = ring_p + P.stages * STAGE;
    uint64_t *const bars = reinterpret_cast<uint64_t *>(small);              // 2 MAX_STAGES + 8
    float2 *const ex = reinterpret_cast<float2 *>(small + 512);              // [2][128] (m, l)
    long long *const scan = reinterpret_cast<long long *>(ex);               // the set-up's scratch, before ex is used
    int *const ctl = reinterpret_cast<int *>(small + 256 + 128 + 64);        // dead, tmem, patched[2], bad[8]
    const uint32_t bar0 = smem_addr(bars);
    const uint32_t full = bar0, empty = bar0 + 8 * MAX_STAGES, s_full = bar0 + 16 * MAX_STAGES, p_full = s_full + 16,
                   o_done = p_full + 16, q_full = o_done + 16, drained = q_full + 8;
    volatile int *const dead = ctl;
    volatile int *const patched = ctl + 2, *const bad = ctl + 4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < P.stages; i++) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
        for (int g = 0; g < 2; g++) mbar_init(s_full + 8 * g, 1), mbar_init(p_full + 8 * g, 4), mbar_init(o_done + 8 * g, 1);
        mbar_init(q_full, 8);
        mbar_init(drained, 1);
        ctl[0] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W_MMA) tmem_alloc(smem_addr(ctl + 1), 512);
    grid_wait();   // the work before this on the stream may still be writing what follows

    // the batch's units, and where this CTA's range begins
    constexpr int NW = NTHREADS / 32;
    long long &start_pre = scan[NW], &total_units = scan[NW + 1], &start_b = scan[NW + 2];
    long long sum = 0;
    for (int b = tid; b < A.B; b += NTHREADS) sum += units_of(req_of(A, C, P, b), C.heads);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) scan[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        long long t = 0;
        for (int w = 0; w < NW; w++) t += scan[w];
        total_units = t;
    }
    __syncthreads();
    const long long T = total_units;
    const int nc = (int)min((long long)gridDim.x, T), cta = blockIdx.x;
    const long long lo = cta < nc ? T * cta / nc : 0, hi = cta < nc ? T * (cta + 1) / nc : 0;
    if (lo < hi) {   // (the whole CTA)
        long long before = 0;
        for (int b0 = 0; before <= lo; b0 += NTHREADS) {
            const int b = b0 + tid;
            const long long w = b < A.B ? units_of(req_of(A, C, P, b), C.heads) : 0;
            long long inc = w;
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            __syncthreads();
            if (lane == 31) scan[warp] = inc;
            __syncthreads();
            long long pre = before + inc - w, all = 0;
            for (int i = 0; i < NW; i++) {
                if (i < warp) pre += scan[i];
                all += scan[i];
            }
            if (pre <= lo && lo < pre + w) start_b = b, start_pre = pre;
            before += all;
            if (b0 + NTHREADS >= A.B) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(ctl + 1);
    grid_launch_dependents();

    Walk walk;
    Seg s;
    walk.pos = lo, walk.hi = hi;
    if (lo < hi) {
        walk.pre = start_pre;
        walk.b = (int)start_b;
        walk.r = req_of(A, C, P, walk.b);
    }
    Ring ring{smem_addr(ring_p), full, empty, 0, P.stages, 0, 0};

    if (warp == W_LOAD) {
        const int P_ = 1 << C.page_shift, box = min(P_, TILE), npg = TILE / box;
        uint32_t stage = 0, phase = 1, loads = 0;   // the first round finds every stage empty
        bool ok = true;
        for (int seg = 0; ok && walk.next(A, C, P, s); seg++) {
            if (lane == 0) bad[seg & 7] = 0;
            __syncwarp();
            // this lane's page of a key tile, or -1
            auto page_of = [&](int t) {
                const int j = s.base(t) + lane * box;
                if (lane >= npg || j >= s.len || !(j + box > s.lo || j < P.sinks)) return -1;
                const int id = __ldg(C.table + (int64_t)s.b * C.max_pages + (j >> C.page_shift));
                if (id >= 0 && id < C.num_pages) return id;
                bad[seg & 7] = 1;
                record_error(P.hdr, SV_DEV_BAD_PAGE, s.b);
                return -1;
            };
            auto load = [&](const CUtensorMap *map, int t, int id) {
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * box * 128 * NB;
                __syncwarp();   // (a bad page noted by any lane, before the arrival that publishes it)
                ok = warp_wait(empty + 8 * stage, phase, dead);
                if (!ok) return;
                loads++;
                if (lane == 0) mbar_expect(full + 8 * stage, bytes);
                __syncwarp();
                if (id >= 0) {
                    const uint32_t dst = ring.base + stage * STAGE + lane * box * 128;
                    for (int blk = 0; blk < NB; blk++)
                        tma_load_4d(dst + blk * BLK, map, full + 8 * stage, blk * 64, s.base(t) & (P_ - 1) & ~(box - 1),
                                    s.kvh, id);
                }
                if (++stage == (uint32_t)P.stages) stage = 0, phase ^= 1;
            };
            int id = page_of(s.t0);
            load(&map_k, s.t0, id);
            for (int t = s.t0; ok && t < s.t1; t++) {
                int nid = -1;
                if (t + 1 < s.t1) {
                    nid = page_of(t + 1);
                    load(&map_k, t + 1, nid);
                }
                if (ok) load(&map_v, t, id);
                id = nid;
            }
        }
        if (!ok) {   // let the copies in flight land before the CTA may end
            const unsigned long long t0 = now_ns();
            for (uint32_t i = loads > (uint32_t)P.stages ? loads - P.stages : 0; i < loads; i++)
                while (!mbar_try(full + 8 * (i % P.stages), i / P.stages & 1) && now_ns() - t0 < WAIT_NS) {}
        }
    } else if (warp == W_MMA) {
        if (lane == 0) {
            constexpr uint32_t idesc_s = mma_idesc(Num<E>::BF16, TILE, TILE, false);
            constexpr uint32_t idesc_o = mma_idesc(Num<E>::BF16, TILE, DP, true);
            const uint64_t qd = smem_desc(smem_addr(smem), 16);
            uint32_t np[2] = {0, 0};   // P tiles taken, per group
            bool ok = true;
            for (int seg = 0; ok && walk.next(A, C, P, s); seg++) {
                const int nt = s.t1 - s.t0, two = s.two(), nv = nt << two;
                auto scores = [&](int v) {
                    const int t = v >> two, g = v & 1;
                    ring.at(k_item(t));
                    if (!mbar_wait(full + 8 * ring.stage, ring.phase, dead)) return false;
                    tc_fence_after();
                    const uint64_t kd = smem_desc(ring.base + ring.stage * STAGE, 16);
                    const uint64_t qg = qd + (uint64_t)((two ? g : 0) * STAGE >> 4);
#pragma unroll
                    for (int k = 0; k < DP / 16; k++) {
                        const uint64_t step = (uint64_t)(((k >> 2) * BLK + (k & 3) * 32) >> 4);
                        mma_ss(tmem + g * TILE, qg + step, kd + step, idesc_s, k > 0);
                    }
                    mma_commit(s_full + 8 * g);
                    if (!two || (v & 1)) mma_commit(empty + 8 * ring.stage);
                    return true;
                };
                auto outputs = [&](int v) {
                    const int t = v >> two, g = v & 1;
                    if (!mbar_wait(p_full + 8 * g, np[g]++ & 1, dead)) return false;
                    ring.at(v_item(t, nt));
                    if (!mbar_wait(full + 8 * ring.stage, ring.phase, dead)) return false;
                    tc_fence_after();
                    const uint64_t vd = smem_desc(ring.base + ring.stage * STAGE, BLK);
#pragma unroll
                    for (int k = 0; k < TILE / 16; k++)
                        mma_ts(tmem + 2 * TILE + g * TILE, tmem + g * TILE + k * 8, vd + (uint64_t)(k * 2048 >> 4),
                               idesc_o, v >= 2 || k > 0);
                    mma_commit(o_done + 8 * g);
                    if (!two || (v & 1)) mma_commit(empty + 8 * ring.stage);
                    return true;
                };
                ok = mbar_wait(q_full, seg & 1, dead);
                tc_fence_after();
                for (int v = 0; ok && v < min(2, nv); v++) ok = scores(v);
                for (int v = 0; ok && v < nv; v++) {
                    ok = outputs(v);
                    if (ok && v + 2 < nv) ok = scores(v + 2);
                }
                ring.count += 2 * nt;
            }
            if (!ok) {   // wait for the matrix instructions in flight before tensor memory is given back
                mma_commit(drained);
                const unsigned long long t0 = now_ns();
                while (!mbar_try(drained, 0) && now_ns() - t0 < WAIT_NS) {}
            }
        }
        __syncwarp();
    } else {
        const int g = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // this warp's 32 lanes of tensor memory
        const uint32_t t_s = tmem + g * TILE + lanes, t_o = tmem + 2 * TILE + lanes;
        const int D = C.D, Hq = P.Hq;
        uint32_t ns_ = 0;   // S tiles taken
        bool ok = true;
        for (int seg = 0; ok && walk.next(A, C, P, s); seg++) {
            const int nt = s.t1 - s.t0;
            const bool two = s.two();
            const int rows = min(s.M - s.m * 2 * TILE, 2 * TILE);   // of this row tile
            // queries, swizzled as the matrix instruction reads them
            for (int i = tid; i < rows * (DP / 8); i += 256) {
                const int r = i / (DP / 8), ch = i % (DP / 8);
                const int rr = s.m * 2 * TILE + r, tok = rr / P.G;
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (ch * 8 < D && !P.qzero)
                    w = *reinterpret_cast<const uint4 *>(static_cast<const E *>(P.q) + (s.row0 + tok) * P.q_stride +
                                                         (int64_t)(s.kvh * P.G + rr - tok * P.G) * D + ch * 8);
                w.x ^= P.qflip, w.y ^= P.qflip, w.z ^= P.qflip, w.w ^= P.qflip;
                char *to = smem + (r >> 7) * STAGE + (ch >> 3) * BLK + (r & 127) * 128 + (((ch & 7) ^ (r & 7)) << 4);
                *reinterpret_cast<uint4 *>(to) = w;
            }
            fence_proxy_async();
            if (tid == 0) patched[seg & 1] = 0;   // (last read before the previous segment's barrier)
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);

            const int rt = two ? g * TILE + row : row;             // this thread's row of the row tile
            const bool active = rt < rows;
            const bool warp_on = (two ? g * TILE : 0) + (warp & 3) * 32 < rows;
            const int rr = s.m * 2 * TILE + rt, tok = rr / P.G;
            const int pos = s.len - s.n + tok;
            float m = -INFINITY, l = 0.f;
            bool any_tile = false;
            for (int t = two ? 0 : g; t < nt; t += two ? 1 : 2) {
                if (!warp_wait(s_full + 8 * g, ns_++ & 1, dead)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int base = s.base(s.t0 + t);
                const bool whole = whole_tile(P, s, base);
                if (!whole && (!two || g == 0)) {
                    ring.at(v_item(t, nt));
                    if (!warp_wait(full + 8 * ring.stage, ring.phase, dead)) {
                        ok = false;
                        break;
                    }
                    if (clean_values<E, DP>(P, s, base, row, ring_p + ring.stage * STAGE)) patched[seg & 1] = 1;
                    fence_proxy_async();
                    __syncwarp();
                }
                if (warp_on) {
                    // S comes in four times 32 columns, twice (maximum, then weights): a thread's 128
                    // scores at once would leave no registers
                    uint32_t x[2][32];
                    auto masked = [&](int i) {
                        if (whole) return;
                        const uint32_t see = seen_mask(P, pos, base + 32 * i);
#pragma unroll
                        for (int k = 0; k < 32; k++)
                            x[i & 1][k] = (see >> k & 1) ? x[i & 1][k] : 0xff800000u;   // -inf
                    };
                    float top[4] = {m, m, m, m};
                    tmem_ld32(t_s, x[0]);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        tmem_wait_ld();
                        after_wait32(x[i & 1]);
                        if (i < 3) tmem_ld32(t_s + 32 * (i + 1), x[(i + 1) & 1]);
                        masked(i);
#pragma unroll
                        for (int k = 0; k < 32; k++) top[k & 3] = fmaxf(top[k & 3], __uint_as_float(x[i & 1][k]));
                    }
                    const float new_m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    // lift the running maximum, and scale O and l down, only where it lags too far
                    const bool lift = active && (m == -INFINITY ? new_m > m : (new_m - m) * P.c > LAG);
                    if (__any_sync(0xffffffffu, lift)) {
                        const float f = lift ? ex2((m - new_m) * P.c) : 1.f;
                        if (lift) m = new_m;
                        if (any_tile) {
                            l *= f;
                            // the group's last product is complete before O changes
                            if (!warp_wait(o_done + 8 * g, (ns_ - 2) & 1, dead)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll
                            for (int i = 0; i < DP; i += 32) {
                                uint32_t o[32];
                                tmem_ld32(t_o + g * TILE + i, o);
                                tmem_wait_ld();
                                after_wait32(o);
#pragma unroll
                                for (int k = 0; k < 32; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                tmem_st32(t_o + g * TILE + i, o);
                            }
                        }
                    }
                    const float off = BIAS - (m == -INFINITY ? 0.f : m * P.c);
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    tmem_ld32(t_s, x[0]);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        uint32_t w[16];
                        tmem_wait_ld();
                        after_wait32(x[i & 1]);
                        if (i < 3) tmem_ld32(t_s + 32 * (i + 1), x[(i + 1) & 1]);
                        masked(i);
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const float a = ex2(fmaf(__uint_as_float(x[i & 1][k]), P.c, off));
                            const float b = ex2(fmaf(__uint_as_float(x[i & 1][k + 1]), P.c, off));
                            sum[k & 3] += a;
                            sum[(k & 3) + 1] += b;
                            w[k / 2] = Num<E>::down(a, b);
                        }
                        tmem_st16(t_s + 16 * i, w);   // over columns already read
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_wait_st();
                }
                any_tile = true;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * g);
            }
            if (ok && any_tile) ok = warp_wait(o_done + 8 * g, (ns_ - 1) & 1, dead);
            if (!two) ex[g * TILE + row] = make_float2(m, l);
            // both groups are through; whether a wait ran out is decided once for all 8 warps
            ok = !softmax_barrier_or(!ok || *dead);
            tc_fence_after();
            if (!ok) break;
            const bool patch = patched[seg & 1] != 0, broken = bad[seg & 7] != 0;
            const bool direct = s.t0 == 0 && s.t1 == s.nt;
            if (warp_on) {
                // the part's maximum and sum, and the factors of the (up to) two sums O
                float f0 = 1.f, f1 = 0.f;
                if (!two && nt > 1) {
                    const float2 a = ex[row], b = ex[TILE + row];
                    m = fmaxf(a.x, b.x);
                    f0 = a.x == m ? 1.f : ex2((a.x - m) * P.c);
                    f1 = b.x == m ? 1.f : ex2((b.x - m) * P.c);
                    l = a.y * f0 + b.y * f1;
                } else if (!two) {
                    const float2 a = ex[row];
                    m = a.x;
                    l = a.y;
                }
                if (broken) l = NAN;
                const float inv = (l == 0.f && !direct) ? 0.f : 1.f / l;
                f0 *= inv;
                f1 *= inv;
                const float lse2 = l == 0.f ? -INFINITY : m * P.c + log2f(l) - BIAS;
                const int slot = 2 * cta + (s.t0 > 0 ? 0 : 1);
                const int head = s.kvh * P.G + rr - tok * P.G;
                const int64_t orow = (int64_t)(s.row0 + tok) * Hq + head;
                const uint32_t t0_ = two ? t_o + g * TILE : t_o;
                const int c0 = two ? 0 : g * (DP / 2), c1 = two ? DP : c0 + DP / 2;
                for (int c = c0; c < c1; c += 16) {
                    uint32_t a[16], b[16];
                    float o[16];
                    tmem_ld16(t0_ + c, a);
                    if (!two && nt > 1) tmem_ld16(t0_ + TILE + c, b);
                    tmem_wait_ld();
                    after_wait16(a);
                    after_wait16(b);
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        o[i] = __uint_as_float(a[i]) * f0;
                        if (!two && nt > 1) o[i] += __uint_as_float(b[i]) * f1;
                    }
                    if (active) {
                        if (patch) add_non_finite<E>(C, P, s, pos, c, o);
                        if (direct) {
                            E *to = static_cast<E *>(P.out) + orow * D + c;
                            if (c < D) *reinterpret_cast<uint4 *>(to) = pack8<E>(o);
                            if (c + 8 < D) *reinterpret_cast<uint4 *>(to + 8) = pack8<E>(o + 8);
                        } else {
                            float4 *to = reinterpret_cast<float4 *>(P.part_o) + ((int64_t)slot * (DP / 4) + c / 4) * PART_ROWS + rt;
#pragma unroll
                            for (int i = 0; i < 4; i++) to[i * PART_ROWS] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                    }
                    __syncwarp();
                }
                if (active && c0 == 0) {
                    if (!direct) P.part_lse[slot * PART_ROWS + rt] = lse2;
                    else if (P.lse) P.lse[orow] = lse2 * 0.6931471805599453f;
                }
            }
            tc_fence_before();
            ring.count += 2 * nt;
        }
        if (tid == 0) {
            // the last segment, if it begins here and ends elsewhere, is this CTA's to describe
            int4 d = make_int4(-1, 0, 0, 0);
            if (lo < hi && s.t0 == 0 && s.t1 < s.nt) {
                const long long last = s.first + s.nt;   // the CTA that holds unit last - 1
                d = make_int4(s.b, s.kvh, s.m, (int)((last * nc + T - 1) / T) - 1);
            }
            P.desc[cta] = d;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *dead) record_error(P.hdr, SV_DEV_TIMEOUT, 0);
    if (warp == W_MMA) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

// Joins the parts of the row tiles that several CTAs hold, in order of the CTAs, and sets the rows
// that no request uses.  Block (c, y): rows [32 y, 32 y + 32) of the row tile that begins in CTA c.
template <typename E, int DP>
__global__ void __launch_bounds__(256) join_kernel(const Batch A, const Cache C, const AttnArgs P) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nblocks = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
    grid_wait();
    const int4 d = P.desc[blockIdx.x];
    if (d.x >= 0) {
        const Req s = req_of(A, C, P, d.x);
        const int rows = min(s.M - d.z * 2 * TILE, 2 * TILE);
        const int rt = blockIdx.y * 32 + lane;
        if (rt < rows) {
            const int first = blockIdx.x, last = d.w;
            float top = -INFINITY;
            bool nan = false;
            for (int c = first; c <= last; c++) {
                const float v = P.part_lse[(2 * c + (c == first)) * PART_ROWS + rt];
                nan |= v != v;
                top = fmaxf(top, v);
            }
            float sum = 0.f;
            float4 o[DP / 32];
#pragma unroll
            for (int i = 0; i < DP / 32; i++) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = first; c <= last; c++) {
                const int slot = 2 * c + (c == first);
                const float f = ex2(P.part_lse[slot * PART_ROWS + rt] - top);
                sum += f;
                const float4 *from = reinterpret_cast<const float4 *>(P.part_o) + ((int64_t)slot * (DP / 4) + warp) * PART_ROWS + rt;
#pragma unroll
                for (int i = 0; i < DP / 32; i++) {
                    const float4 x = from[(int64_t)i * 8 * PART_ROWS];
                    o[i].x += f * x.x, o[i].y += f * x.y, o[i].z += f * x.z, o[i].w += f * x.w;
                }
            }
            if (nan) sum = NAN;
            const float inv = 1.f / sum;
            const int rr = d.z * 2 * TILE + rt, tok = rr / P.G;
            const int64_t orow = (int64_t)(s.row0 + tok) * P.Hq + d.y * P.G + rr - tok * P.G;
#pragma unroll
            for (int i = 0; i < DP / 32; i++) {
                const int col = (i * 8 + warp) * 4;
                if (col < C.D)
                    *reinterpret_cast<uint2 *>(static_cast<E *>(P.out) + orow * C.D + col) =
                        make_uint2(Num<E>::down(o[i].x * inv, o[i].y * inv), Num<E>::down(o[i].z * inv, o[i].w * inv));
            }
            if (P.lse && warp == 0) P.lse[orow] = (top + log2f(sum)) * 0.6931471805599453f;
        }
    }
    // unused rows: zeros; the rows of a request in error: NaN
    for (int b0 = (me * 8 + warp) * 32; b0 < A.B; b0 += nblocks * 256) {
        const int b = b0 + lane;
        int from = 0, to = 0, err = 0, head = 0, tail = 0;
        if (b < A.B) {
            const Span s = span_of(A, C.max_pages << C.page_shift, b);
            err = s.err;
            if (err) record_error(P.hdr, err, b);
            int end = s.row0 + A.k_max + 1;
            if (A.row_off) {
                end = __ldg(A.row_off + b + 1);
                if (b == 0) head = min(max(s.row0, 0), A.R);                       // rows before the first request
                if (b == A.B - 1) tail = A.R - min(max(end, 0), A.R);              // and after the last
            }
            from = s.row0 + s.n;
            to = end;
            if (from < 0 || to > A.R || to < from) from = to = 0;
        }
        for (unsigned m = __ballot_sync(0xffffffffu, to > from || head || tail); m; m &= m - 1) {
            const int l = __ffs(m) - 1;
            const int f = __shfl_sync(0xffffffffu, from, l), t = __shfl_sync(0xffffffffu, to, l);
            const int h = __shfl_sync(0xffffffffu, head, l), e = A.R - __shfl_sync(0xffffffffu, tail, l);
            const bool er = __shfl_sync(0xffffffffu, err, l) != 0;
            auto fill = [&](int r0, int r1, bool nan) {
                const uint32_t w = nan ? Num<E>::NAN2 : 0u;
                const int64_t n = (int64_t)(r1 - r0) * P.Hq * C.D / 8, hn = (int64_t)(r1 - r0) * P.Hq;
                uint4 *o = reinterpret_cast<uint4 *>(static_cast<E *>(P.out) + (int64_t)r0 * P.Hq * C.D);
                for (int64_t i = lane; i < n; i += 32) o[i] = make_uint4(w, w, w, w);
                if (P.lse)
                    for (int64_t i = lane; i < hn; i += 32) P.lse[(int64_t)r0 * P.Hq + i] = nan ? NAN : 0.f;
            };
            fill(f, t, er);
            fill(0, h, false);
            fill(e, A.R, false);
        }
    }
}

// cuTensorMapEncodeTiled, looked up once (the library does not link the driver).
typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeFn encode_fn() {
    static std::atomic<void *> fn{nullptr};
    void *f = fn.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeFn>(f);
}

// Tensor map of a cache: (element, slot, head, page), boxes of 64 elements x the slots of one page
// that fit a key tile.  Elements past head_dim read as zero, which pads odd widths.
static bool encode(CUtensorMap *map, const sv_kv_cache &c, void *ptr) {
    EncodeFn f = encode_fn();
    if (!f) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_heads, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride * 2, (cuuint64_t)c.head_stride * 2, (cuuint64_t)c.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(c.page_size < TILE ? c.page_size : TILE), 1, 1}, one[4] = {1, 1, 1, 1};
    return f(map, c.dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, ptr, dims,
             strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int SMEM_MAX = 232448, SMALL = 512 + 2 * TILE * 8;

template <typename E, int DP>
static sv_status launch_attention(const Batch &A, const Cache &C, AttnArgs P, const sv_kv_cache &cache, cudaStream_t st) {
    constexpr int STAGE = DP / 64 * BLK;
    CUtensorMap mk, mv;
    if (!encode(&mk, cache, cache.k) || !encode(&mv, cache, cache.v)) return SV_ERR_CUDA;
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return SV_ERR_CUDA;
    P.q_tiles = (A.k_max + 1) * P.G > TILE ? 2 : 1;
    P.stages = (SMEM_MAX - SMALL - P.q_tiles * STAGE) / STAGE;
    if (P.stages > MAX_STAGES) P.stages = MAX_STAGES;
    const int smem = (P.q_tiles + P.stages) * STAGE + SMALL;
    // no more CTAs than the batch can have units
    const long long most = (long long)A.B * C.heads * (((long long)(A.k_max + 1) * P.G + 2 * TILE - 1) / (2 * TILE)) *
                           ((((long long)C.max_pages << C.page_shift) + TILE - 1) / TILE);
    int ctas = nsm < MAX_CTAS ? nsm : MAX_CTAS;
    if (most < ctas) ctas = (int)most;
    if (cudaFuncSetAttribute(attention_kernel<E, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return SV_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, attention_kernel<E, DP>, A, C, P, mk, mv) != cudaSuccess) return SV_ERR_CUDA;
    const int most_rows = (A.k_max + 1) * P.G;
    cfg.gridDim = dim3(ctas, (min(most_rows, PART_ROWS) + 31) / 32);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join_kernel<E, DP>, A, C, P) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace svc

using namespace svc;

extern "C" size_t sv_attention_workspace_bytes(int32_t head_dim) {
    if (head_dim < 8 || head_dim > 128 || head_dim % 8) return 0;
    return attn_ws(head_dim).total;
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
    const AttnWs L = attn_ws(cache.head_dim);
    if (((uintptr_t)workspace & 255) || workspace_bytes < L.total) return SV_ERR_WORKSPACE;
    char *w = static_cast<char *>(workspace);
    AttnArgs P;
    P.q = q;
    P.q_stride = q_stride;
    P.out = out;
    P.lse = out_lse;
    P.hdr = reinterpret_cast<int32_t *>(w);
    P.desc = reinterpret_cast<int4 *>(w + L.desc);
    P.part_lse = reinterpret_cast<float *>(w + L.lse);
    P.part_o = reinterpret_cast<float *>(w + L.o);
    P.c = (scale == 0.f ? 1.f : fabsf(scale)) * 1.4426950408889634f;
    P.qflip = scale < 0.f ? 0x80008000u : 0u;
    P.qzero = scale == 0.f;
    P.Hq = num_q_heads;
    P.G = num_q_heads / cache.num_heads;
    P.window = window;
    P.sinks = sinks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = cache.head_dim > 64;
    if (cache.dtype == SV_BF16)
        return wide ? launch_attention<__nv_bfloat16, 128>(A, C, P, cache, st) : launch_attention<__nv_bfloat16, 64>(A, C, P, cache, st);
    return wide ? launch_attention<__half, 128>(A, C, P, cache, st) : launch_attention<__half, 64>(A, C, P, cache, st);
}
