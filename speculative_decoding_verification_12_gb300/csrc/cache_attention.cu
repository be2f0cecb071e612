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
// Work.  The unit of work is one key tile of one (key head, request, row tile).  All units of the
// batch, in that order, are cut into one equal range per CTA, from the lengths on the device: ragged
// batches, one long request and windows need no other schedule.  Heads come first so that the heads of
// a request run at the same time, CTAs / heads apart: where they lie beside each other in a token's
// row and are not whole 128-byte lines wide, the lines that two of them share are then read once
// (64 requests of 4096 keys, 8 heads of 80 columns: 178 us request by request, 123 us).  A row tile
// whose keys lie in several CTAs' ranges leaves a part per CTA in the workspace, and the second kernel
// joins them in order.
//
// A CTA: a front warp that turns the CTA's range into segments (a row tile and its key tiles here) and
// loads their queries, a warp for K and one for V (tensor copies of pages into two rings of tiles),
// one that issues the matrix instructions (S and O in tensor memory, P back in tensor memory as an
// operand), and two groups of 4 warps, a thread per row, for softmax and epilogue.  With one row tile
// the groups take alternate key tiles, each with its own m, l and O, joined at the end; with two, each
// has its own.
//
// What bounds it.  Few rows per key (a verify step): the cache's bytes; 256 requests of 5 rows over 4096
// keys of 8 heads of 128 read 4.3 GB in 633 to 661 us by run, 6.5 to 6.8 TB/s, one request over 131 071
// keys 0.54 GB in 90 us.  Many rows (16 requests of 65 rows, 8 query heads per key head, 8192 keys): the
// chain of a product, its softmax and the next product on the 512 columns of tensor memory; 162 us in a
// graph (166 issued), 860 TFLOP/s, the tensor pipe active in 50 % of the cycles.  Small calls: the chain of
// launch, lengths, table, first tile, epilogue and join, 10.5 us for one request of 2049 keys.  Short
// segments: the change from one to the next, about 2 us where both groups share them (512 one-row requests
// of 8 heads under a window of 64 keys: 27 segments a CTA, 151 us).  Many rows of one request: one warp
// loads up to 256 rows' queries, into one buffer where there are two row tiles (65 rows, 32 on 8 heads,
// over 65 keys: 18.9 us).
#include <math.h>

#include <atomic>

#include "sv_cache.cuh"
#include "sv_launch.h"
#include "sv_tc.cuh"

namespace svc {

constexpr int TILE = 128;                // tokens per key tile, rows per row tile
constexpr int BLK = TILE * 128;          // bytes of 128 rows x 64 elements
constexpr int NTHREADS = 384;            // 2 x 4 softmax warps, then one warp for each of:
constexpr int W_K = 9, W_V = 10, W_MMA = 11;   // keys, values, matrix instructions; 8 is the front warp
constexpr int MAX_CTAS = 160;
constexpr int PART_ROWS = 256;           // rows of a part
constexpr int MAX_STAGES = 7;            // of each of the two rings
constexpr int MAX_QBUFS = 4;

struct AttnArgs {
    const void *q;
    int64_t q_stride;
    void *out;
    float *lse;
    int32_t *hdr;
    int4 *desc;        // workspace, per CTA: the row tile whose first part, but not last, it holds (its request's
                       // first row, or -1: none; key head; number; last part's CTA and 256 M)
    float *part_lse;   // workspace, [2 * MAX_CTAS][PART_ROWS]: log2 of the part's sum
    float *part_o;     // workspace, [2 * MAX_CTAS][PART_ROWS][DP]
    float c;           // |scale| log2(e)
    int negative, zero;   // scale < 0, scale == 0
    int withhold;         // testing aid: no CTA loads its first K tile
    int Hq, G, window, sinks;
    int k_stages, v_stages;
    int overhead;      // cost of a row tile beside its key tiles, in key tiles
    int weighted;      // whether a key tile costs more for more than 128 rows
    int q_tiles;       // row tiles of 128 that a request may have at a time: 1 or 2
    int q_rows, q_bufs;   // rows of a query buffer (a multiple of 8), and how many there are
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

template <int V>
struct Const {
    static constexpr int N = V;
};

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
// What a key tile costs for up to 128 rows, and for more.  16 requests of 65 rows on 8192 keys, 8 query heads
// per key head, whose third row tile has the last 8 of 520 rows: 180 us at 1 to 1, 168 at 3 to 4, 166 at
// 2 to 3, 175 at 1 to 2; 64 ragged requests of up to 17 rows: 185, 175, 175 and 175 us.
constexpr int W_ONE = 2, W_TWO = 3;
__device__ __forceinline__ uint32_t over_weight(uint32_t x, int w) {
    return w == 1 ? x : w == W_ONE ? x / W_ONE : x / W_TWO;
}

// The cost of a key tile for row tile m of a request, and the request's cost per key head.
__device__ __forceinline__ int weight_of(const AttnArgs &P, const Req &r, int m) {
    return !P.weighted ? 1 : r.M - m * 2 * TILE > TILE ? W_TWO : W_ONE;
}
__device__ __forceinline__ long long units_of(const AttnArgs &P, const Req &r) {
    const int weight = (r.mt - 1) * (P.weighted ? W_TWO : 1) + weight_of(P, r, r.mt - 1);
    return r.nt ? (long long)(r.nt + P.overhead) * weight : 0;
}

// A segment, as the front warp hands it out (64 bytes): key tiles [t0, t1) of the nt of row tile m of
// key head kvh of request b.  nt == 0 ends the list.
struct __align__(16) Seg {
    int row0, n, len, M, lo, w0, ns, nt;   // as in Req
    int b, kvh, m, t0, t1, solo, pad[2];   // solo: one group takes all its tiles
    __device__ __forceinline__ int base(int t) const { return (t < ns ? t : w0 + t - ns) * TILE; }
    __device__ __forceinline__ bool two() const { return M - m * 2 * TILE > TILE; }
};
constexpr int SEGS = 32;                 // segments in flight between the front warp and the others
// Narrow heads: key tiles of a segment that one group takes alone.  512 x 8 segments of 3 tiles take 150 us
// shared and 129 alone; 1024 x 8 of 8 tiles 422 shared and 440 alone (the last one leaves a group idle).
constexpr int SOLO_TILES = 4;
constexpr int SMALL_BATCH = 16;          // requests that the front warp looks at together
constexpr int SEG_READERS = 11;          // warps that take each of them

// a / b for a >= 0, b > 0: nearly always in 32 bits, where it takes a tenth of the time.
__device__ __forceinline__ long long quotient(long long a, int b) {
    return (a >> 32) ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

__device__ __forceinline__ long long quotient64(long long a, long long b) {
    return ((a | b) >> 32) ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

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
__device__ __forceinline__ bool seen_by_all(const AttnArgs &P, const Seg &s, int j) {
    return j <= s.len - s.n && (!P.window || j > s.len - 1 - P.window || j < P.sinks);
}
__device__ __forceinline__ bool seen_by_any(const AttnArgs &P, const Seg &s, int j) {
    return j < s.len && (j >= s.lo || j < P.sinks);
}
// Whether every row sees all 128 tokens from base on.
__device__ __forceinline__ bool whole_tile(const AttnArgs &P, const Seg &s, int base) {
    return base + TILE - 1 <= s.len - s.n && (!P.window || base > s.len - 1 - P.window || base + TILE - 1 < P.sinks);
}

// A position in a ring of tiles: the stage, and the parity of its turn.
struct Place {
    uint32_t stage, parity;
    __device__ __forceinline__ void advance(uint32_t stages) {
        if (++stage == stages) stage = 0, parity ^= 1;
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
__device__ __forceinline__ bool clean_values(const AttnArgs &P, const Seg &s, int base, int tok, char *tile) {
    const int j = base + tok;
    if (seen_by_all(P, s, j)) return false;
    // (a different 16 bytes of the row per lane: no two of 8 lanes share a bank)
    auto at = [&](int i) {
        return reinterpret_cast<uint4 *>(tile + (i >> 3) * BLK + tok * 128 + (((i ^ tok) & 7) << 4));
    };
    if (!seen_by_any(P, s, j)) {
#pragma unroll 8
        for (int i = 0; i < DP / 8; i++) *at(i) = make_uint4(0u, 0u, 0u, 0u);
        return false;
    }
    bool took = false;
#pragma unroll 1
    for (int i = 0; i < DP / 8; i++) {
        uint4 w = *at(i);
        uint32_t *p = &w.x;
        bool hit = false;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            if (!finite16<E>(p[e] & 0xffffu)) p[e] &= 0xffff0000u, hit = true;
            if (!finite16<E>(p[e] >> 16)) p[e] &= 0xffffu, hit = true;
        }
        if (!hit) continue;
        took = true;
        *at(i) = w;
    }
    return took;
}

// The non-finite elements that clean_values took, for the row at position pos, added to its result
// after it was stored: `put(d, x)` adds x to element d, for d in [c0, c1).
template <typename E, typename F>
__device__ __forceinline__ void add_non_finite(const Cache &C, const AttnArgs &P, const Seg &s, int pos, int c0, int c1,
                                               F put) {
#pragma unroll 1
    for (int side = 0; side < 2; side++) {
        const int from = side ? s.lo : s.len - s.n + 1, to = side ? min(s.len, s.lo + s.n - 1) : s.len;
#pragma unroll 1
        for (int j = from; j < to; j++) {
            if (side && (!P.window || j > s.len - s.n)) break;   // (the causal side has it)
            const int tile = j / TILE, t = tile >= s.w0 ? tile - s.w0 + s.ns : tile;
            if (t < s.t0 || t >= s.t1 || seen_by_all(P, s, j) || !sees(P, pos, j)) continue;
            const int page = C.table[(int64_t)s.b * C.max_pages + (j >> C.page_shift)];
            if (page < 0 || page >= C.num_pages) continue;
            const E *v = static_cast<const E *>(C.v) + page * C.page_stride +
                         (j & ((1 << C.page_shift) - 1)) * C.token_stride + s.kvh * C.head_stride;
#pragma unroll 1
            for (int d = c0; d < c1; d++) {
                const float x = (float)v[d];
                if (!(fabsf(x) < INFINITY)) put(d, x);
            }
        }
    }
}

// Barriers, flags and the groups' exchange, at the start of shared memory.
constexpr int SMALL = 5120;
// Narrow heads, up to 32 rows: group 1 takes its rows to the third quarter of tensor memory, so that the
// groups' one busy warp each sits on a scheduler of its own, and hands its O to group 0 through shared
// memory.
constexpr int FEW_ROWS = 32, DOWN = 64;   // rows, and how far down group 1 has them
__host__ __device__ constexpr int hand_over(int DP) {   // (9216: 1024-byte steps)
    return DP == 64 ? FEW_ROWS * (64 + 4) * 4 + 512 : 0;
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
    constexpr int NW = NTHREADS / 32;
    // With narrow heads O leaves room for P beside it, so that a group's next S can be made as soon as
    // its scores are in registers; with wide ones P lies over S, and S waits for P V.
    constexpr bool APART = DP == 64;
    constexpr int P_COL = APART ? 2 * TILE + 64 : TILE / 2;   // P of group g at column g * 128 + P_COL
    extern __shared__ __align__(1024) char smem[];
    // [barriers and small state][group 1's O][ring of K tiles][query buffers][ring of V tiles]; the matrix
    // instruction reads 128 rows around a query buffer whatever they hold: the rows outside it are other
    // bytes of this memory, and reach only rows of S, P and O that nothing uses
    const int q_block = P.q_rows * 128, q_buffer = NB * q_block;
    float *const handed = reinterpret_cast<float *>(smem + SMALL);           // [FEW_ROWS][DP + 4]
    char *const k_p = smem + SMALL + hand_over(DP), *const q_p = k_p + P.k_stages * STAGE;
    char *const v_p = q_p + P.q_bufs * P.q_tiles * q_buffer;
    int *const ctl = reinterpret_cast<int *>(smem + 400);                    // dead, tmem, -, -, patched[2][4], bad[16]
    float2 *const ex = reinterpret_cast<float2 *>(smem + 512);               // [2][128] (m, l)
    long long *const scan = reinterpret_cast<long long *>(ex);               // the set-up's scratch, before ex is used
    Seg *const segs = reinterpret_cast<Seg *>(smem + 2560);                  // [SEGS]
    const uint32_t seg_full = smem_addr(smem + 4608), seg_empty = seg_full + 8 * SEGS;
    const uint32_t k_full = smem_addr(smem), k_empty = k_full + 8 * MAX_STAGES, v_full = k_empty + 8 * MAX_STAGES,
                   v_empty = v_full + 8 * MAX_STAGES, s_full = v_empty + 8 * MAX_STAGES, p_full = s_full + 16,
                   o_done = p_full + 16, both = o_done + 16, s_free = both + 16, drained = s_free + 16,
                   q_full = drained + 24, q_empty = q_full + 8 * MAX_QBUFS;
    volatile int *const dead = ctl, *const patched = ctl + 4, *const bad = ctl + 12;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t k_stages = P.k_stages, v_stages = P.v_stages, q_bufs = P.q_bufs;

    // one thread per barrier: the rings and pairs in a row from k_full, then the segments'
    constexpr int NBARS = 4 * MAX_STAGES + 13 + 2 * MAX_QBUFS;
    if (tid < NBARS) {
        // pairs: s_full, p_full (4 warps), o_done, both (8 warps), s_free (4 warps); then the rest
        const int p = (tid - 4 * MAX_STAGES) >> 1;
        const bool frees_v = tid >= 3 * MAX_STAGES && tid < 4 * MAX_STAGES;
        mbar_init(k_full + 8 * tid, p == 1 || p == 4 ? 4 : p == 3 ? 8 : APART && frees_v ? 2 : 1);
    } else if (tid >= 128 && tid < 128 + 2 * SEGS) {
        mbar_init(seg_full + 8 * (tid - 128), tid < 128 + SEGS ? 1 : SEG_READERS);
    } else if (tid >= 256 && tid < 256 + 28 && tid != 257) {   // (1 is the tensor memory's address)
        ctl[tid - 256] = tid >= 260 && tid < 268 ? -1 : 0;   // patched: -1
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (warp == W_MMA) tmem_alloc(smem_addr(ctl + 1), 512);
    grid_wait();   // the work before this on the stream may still be writing what follows

    // The batch's units, and where this CTA's range begins: prefix sums over the requests, NTHREADS at a
    // time (a batch of up to that many is looked at once).  Only the front warp needs them, and finds those
    // of a small batch by itself, a request a lane.
    long long &start_pre = scan[NW], &start_b = scan[NW + 1];
    long long W = 0, T = 0, lo = 0, hi = 0, before = 0;   // units of one key head, of all, and this CTA's range
    int nc = 0, kvh0 = 0;
    const int cta = blockIdx.x;
    auto range = [&]() {   // [T cta / nc, T (cta + 1) / nc), and the head that it begins in
        T = W * C.heads;
        nc = (int)min((long long)gridDim.x, P.weighted ? T / W_TWO : T);   // (a key tile at least for each)
        if (T && !nc) nc = 1;
        if (cta < nc) {
            const long long q = quotient(T, nc);
            const int rest = (int)(T - q * nc);
            lo = q * cta + rest * cta / nc;
            hi = q * (cta + 1) + rest * (cta + 1) / nc;
            if (lo < hi) kvh0 = (int)quotient64(lo, W);
        }
    };
    if (A.B > SMALL_BATCH) {
        __syncthreads();   // (barriers and flags are set)
#pragma unroll 1
        for (int pass = A.B <= NTHREADS; pass < 2; pass++) {   // pass 0 sums, pass 1 finds
            before = 0;
#pragma unroll 1
            for (int b0 = 0; b0 < A.B; b0 += NTHREADS) {
                const int b = b0 + tid;
                Req r = {};
                if (b < A.B) r = req_of(A, C, P, b);
                const long long w = units_of(P, r);
                long long inc = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                if (b0) __syncthreads();
                if (lane == 31) scan[warp] = inc;
                __syncthreads();
                long long pre = before + inc - w, all = 0;
#pragma unroll
                for (int i = 0; i < NW; i++) {
                    const long long x = scan[i];
                    if (i < warp) pre += x;
                    all += x;
                }
                before += all;
                if (pass == 0) continue;
                if (b0 == 0) {
                    if (A.B <= NTHREADS) W = all;
                    range();
                }
                const long long at = lo - kvh0 * W;
                if (lo < hi && pre <= at && at < pre + w) start_b = b, start_pre = pre;
            }
            if (pass == 0) W = before;
            __syncthreads();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(ctl + 1);
    grid_launch_dependents();

    // Takes segment k into registers; false at the end of the list, or when a wait ran out (ok).
    bool ok = true;
    auto take = [&](int k, Seg &s, bool release_now) {
        const int slot = k & (SEGS - 1);
        ok = warp_wait(seg_full + 8 * slot, k / SEGS & 1, dead);
        if (!ok) return false;
        int4 *to = reinterpret_cast<int4 *>(&s);
        const int4 *from = reinterpret_cast<const int4 *>(segs + slot);
#pragma unroll
        for (int i = 0; i < 4; i++) to[i] = from[i];
        __syncwarp();
        if (release_now && lane == 0) mbar_arrive(seg_empty + 8 * slot);
        return s.nt > 0;
    };
    auto release = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty + 8 * (k & (SEGS - 1)));
    };

    // S of group g from the queries and keys at the given places, and P V into the group's O (one lane each)
    const int steps = (C.D + 15) / 16;                              // of 16 columns: nothing past head_dim
    auto issue_s = [&](uint32_t g, uint32_t q_at, uint32_t k_stage, bool down) {
        const uint32_t idesc = mma_idesc(Num<E>::BF16, TILE, TILE, false) | (uint32_t)P.negative << 13;
        const uint64_t qd = smem_desc(smem_addr(q_p) + q_at * q_buffer - (down ? DOWN * 128 : 0), 16);
        const uint64_t kd = smem_desc(smem_addr(k_p) + k_stage * STAGE, 16);
        const uint32_t q_step = q_block >> 4;
        auto run = [&](auto n) {
#pragma unroll
            for (int k = 0; k < decltype(n)::N; k++)
                mma_ss(tmem + g * TILE, qd + (uint64_t)((k >> 2) * q_step + (k & 3) * 2),
                       kd + (uint64_t)((k >> 2) * (BLK >> 4) + (k & 3) * 2), idesc, k > 0);
        };
        if (DP == 64) run(Const<4>());
        else if (steps == 8) run(Const<8>());
        else if (steps == 5) run(Const<5>());
        else if (steps == 6) run(Const<6>());
        else run(Const<7>());
    };
    auto issue_o = [&](uint32_t g, uint32_t v_stage, bool add) {
        const uint32_t idesc = mma_idesc(Num<E>::BF16, TILE, 0, true) | (uint32_t)(steps * 2) << 17;
        const uint64_t vd = smem_desc(smem_addr(v_p) + v_stage * STAGE, BLK);
#pragma unroll
        for (int k = 0; k < TILE / 16; k++)
            mma_ts(tmem + 2 * TILE + g * TILE, tmem + g * TILE + P_COL + k * 8, vd + (uint64_t)(k * 2048 >> 4), idesc,
                   add || k > 0);
    };

    if (warp >= 8) {
        regs_down<88>();   // to the softmax warps: 2 x 208 + 88 = 3 x 168
        if (warp == W_K || warp == W_V) {
            // Keys, or values, of each segment's tiles.
            const bool is_v = warp == W_V;
            const CUtensorMap *const map = is_v ? &map_v : &map_k;
            const uint32_t ring = smem_addr(is_v ? v_p : k_p), full = is_v ? v_full : k_full, empty = is_v ? v_empty : k_empty,
                           stages = is_v ? v_stages : k_stages;
            Seg s;
            const int P_ = 1 << C.page_shift, box = min(P_, TILE), npg = TILE / box, tpl = 32 / npg;
            const int sub = lane & (npg - 1), lane_tile = lane / npg;
            Place at{0, 1};   // the first round finds every stage empty
            uint32_t loads = 0;
            for (int seg = 0; ok && take(seg, s, true); seg++) {
                // a lane's page of `tpl` tiles from t on (npg lanes a tile), or -1: one load of the table
                // serves several tiles, and is issued that many tiles ahead of its use
                const int32_t *table = C.table + (int64_t)s.b * C.max_pages;
                auto fetch = [&](int t) {
                    t += lane_tile;
                    const int j = s.base(t) + sub * box;
                    if (t >= s.t1 || j >= s.len || !(j + box > s.lo || j < P.sinks)) return -1;
                    return (int)min((uint32_t)table[j >> C.page_shift], (uint32_t)C.num_pages);   // (num_pages: not a page)
                };
                int ids = -1, ahead = fetch(s.t0), t_ids = s.t0 - tpl;
#pragma unroll 1
                for (int t = s.t0; t < s.t1; t++) {
                    if (t == t_ids + tpl) {
                        ids = ahead;
                        t_ids = t;
                        ahead = fetch(t + tpl);
                    }
                    // this lane's page of tile t (lanes below npg), or -1
                    int id = __shfl_sync(0xffffffffu, ids, (t - t_ids) * npg + sub);
                    if (lane >= npg) id = -1;
                    if (id == C.num_pages) {
                        bad[seg & 15] = seg + 1;
                        record_error(P.hdr, SV_DEV_BAD_PAGE, s.b);
                        id = -1;
                    }
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * box * 128 * NB;
                    __syncwarp();   // (a bad page noted by any lane, before the arrival that publishes it)
                    ok = warp_wait(empty + 8 * at.stage, at.parity, dead);
                    if (!ok) break;
                    if (P.withhold && !is_v && loads == 0) {   // (its waits then run out, as they are meant to)
                        ok = false;
                        break;
                    }
                    loads++;
                    if (lane == 0) mbar_expect(full + 8 * at.stage, bytes);
                    __syncwarp();
                    if (id >= 0) {
                        const uint32_t dst = ring + at.stage * STAGE + sub * box * 128;
                        for (int blk = 0; blk < NB; blk++)
                            tma_load_4d(dst + blk * BLK, map, full + 8 * at.stage, blk * 64, s.base(t) & (P_ - 1) & ~(box - 1),
                                        s.kvh, id);
                    }
                    __syncwarp();
                    at.advance(stages);
                }
            }
            if (!ok) {   // let the copies in flight land before the CTA may end
                const uint32_t t0 = now_ns32();
                for (uint32_t i = loads > stages ? loads - stages : 0; i < loads; i++)
                    while (!mbar_try(full + 8 * (i % stages), i / stages & 1) && now_ns32() - t0 < WAIT_NS) {}
            }
        } else if (APART && warp == W_MMA) {
            // Scores, with P apart: each as soon as its group has the last ones in registers.
            const bool leader = elect();
            Place ks{0, 0}, qs{0, 0};
            uint32_t g = 0, nf = 3;   // the group whose turn it is; parities of each one's free S
            Seg s;
            for (int seg = 0; ok && take(seg, s, true); seg++) {
                const int two = s.two(), nv = (s.t1 - s.t0) << two;
                ok = warp_wait(q_full + 8 * qs.stage, qs.parity, dead);
#pragma unroll 1
                for (int v = 0; ok && v < nv; v++) {
                    ok = warp_wait(s_free + 8 * g, nf >> g & 1, dead) && warp_wait(k_full + 8 * ks.stage, ks.parity, dead);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        issue_s(g, two ? v & 1 : qs.stage, ks.stage, g && s.M <= FEW_ROWS);
                        mma_commit(s_full + 8 * g);
                        if (v == nv - 1) mma_commit(q_empty + 8 * qs.stage);
                    }
                    __syncwarp();
                    nf ^= 1u << g;
                    if (!s.solo || v == nv - 1) g ^= 1;
                    if (!two || (v & 1)) ks.advance(k_stages);
                }
                qs.advance(q_bufs);
            }
            if (!ok) {   // wait for the matrix instructions in flight before tensor memory is given back
                if (leader) mma_commit(drained);
                const uint32_t t0 = now_ns32();
                while (!mbar_try(drained, 0) && now_ns32() - t0 < WAIT_NS) {}
            }
            __syncwarp();
        } else if (warp == W_MMA) {
            // Matrix instructions, with P over S.  Over all segments the row tiles' products come in one
            // sequence: tile v of a segment, or, with two row tiles, row tile v & 1 of key tile v >> 1.  The
            // groups take it in turn, S runs two ahead of P V, and so the next segment's scores are ready
            // while this one's last tiles are still with the groups.  The whole warp runs this; one lane
            // issues.  The path from a group's weights to its next scores is the kernel's longest chain, so
            // P V and that S are issued together, the commits after both.  A commit costs the issuing lane
            // 70 to 140 cycles: there are two a product, S is there (the softmax group then frees the K tile)
            // and the V tile is free.  A group learns of its last product of a segment by o_done; earlier
            // ones are complete when a later S is.
            const bool leader = elect();
            int sseg = 0, oseg = 0;                                     // segments opened
            int sv = 0, snv = 0, stwo = 0, ov = 0, onv = 0, otwo = 0;   // product, products and kind of the current ones
            auto open = [&](int &k, int &v, int &nv, int &two, bool release) {
                Seg s;
                v = nv = 0;
                if (!take(k++, s, release)) return;
                two = s.two();
                nv = (s.t1 - s.t0) << two;
            };
            open(sseg, sv, snv, stwo, false);
            if (ok) open(oseg, ov, onv, otwo, true);
            Place ks{0, 0}, vs{0, 0}, qs{0, 0};
            uint32_t gs = 0, go = 0, np = 0;   // groups whose turn it is; parity of each one's next P
            int lead = 0;                      // products whose S, but not P V, is issued: at most 2
            uint32_t polls = 0, idle_since = 0;
#pragma unroll 1
            while (ok && onv) {
                // all that may be waited for is asked at once; every lane has to have seen it
                uint32_t there = 0;
                if (snv) {   // the next S: its queries and its keys
                    there = sv || mbar_test(q_full + 8 * qs.stage, qs.parity);
                    there |= (uint32_t)mbar_test(k_full + 8 * ks.stage, ks.parity) << 1;
                }
                if (lead) {
                    there |= (uint32_t)mbar_test(p_full + 8 * go, np >> go & 1) << 2;
                    there |= (uint32_t)mbar_test(v_full + 8 * vs.stage, vs.parity) << 3;
                }
                there = __reduce_and_sync(0xffffffffu, there);
                const bool do_o = there >> 2 == 3, do_s = (there & 3) == 3 && (lead < 2 || do_o);
                if (!do_o && !do_s) {
                    if (++polls & 255) continue;
                    const uint32_t now = now_ns32() | 1;
                    if (!idle_since) idle_since = now;
                    const bool late = *dead || now - idle_since > WAIT_NS;
                    if (__any_sync(0xffffffffu, late)) {
                        *dead = 1;
                        ok = false;
                    }
                    continue;
                }
                idle_since = 0;
                tc_fence_after();
                const bool last_use = !otwo || (ov & 1);
                if (leader) {
                    if (do_o) issue_o(go, vs.stage, ov >= 2);
                    if (do_s) {
                        issue_s(gs, stwo ? sv & 1 : qs.stage, ks.stage, false);
                        mma_commit(s_full + 8 * gs);
                        if (sv == snv - 1) mma_commit(q_empty + 8 * qs.stage);
                    }
                    if (do_o) {
                        if (last_use) mma_commit(v_empty + 8 * vs.stage);
                        if (ov >= onv - 2) mma_commit(o_done + 8 * go);
                    }
                }
                __syncwarp();
                if (do_o) {
                    if (last_use) vs.advance(v_stages);
                    np ^= 1u << go;
                    go ^= 1;
                    lead--;
                    if (++ov == onv) open(oseg, ov, onv, otwo, true);
                }
                if (do_s && ok) {
                    if (!stwo || (sv & 1)) ks.advance(k_stages);
                    gs ^= 1;
                    lead++;
                    if (++sv == snv) {
                        qs.advance(q_bufs);
                        open(sseg, sv, snv, stwo, false);
                    }
                }
            }
            if (!ok) {   // wait for the matrix instructions in flight before tensor memory is given back
                if (leader) mma_commit(drained);
                const uint32_t t0 = now_ns32();
                while (!mbar_try(drained, 0) && now_ns32() - t0 < WAIT_NS) {}
            }
            __syncwarp();
        } else {
            // Front: the segments of this CTA's range, in order, and their queries, swizzled as the matrix
            // instruction reads them.  A lane looks at one of 16 requests at a time.
            uint32_t pushed = 0, issued = 0, done = 0;   // segments handed out, their queries' copies begun, and there
            Req r = {};
            long long first = 0, sum = 0;                // this lane's request's first unit, all 16's units
            bool fresh = true;
            auto look = [&](int b) {                     // at requests b .. b + 15: first and sum from this head's start
                r.nt = r.mt = 0;
                if (lane < SMALL_BATCH && b + lane < A.B) r = req_of(A, C, P, b + lane);
                const long long w = units_of(P, r);
                sum = w;
#pragma unroll
                for (int o = 1; o < SMALL_BATCH; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                first = sum - w;
                sum = __shfl_sync(0xffffffffu, sum, SMALL_BATCH - 1);
            };
            if (A.B <= SMALL_BATCH) {
                look(0);
                W = sum;
                range();
            }
            int kvh = kvh0, b_base = A.B > SMALL_BATCH && lo < hi ? (int)start_b : 0, m = 0;
            long long pre = A.B > SMALL_BATCH && lo < hi ? start_pre : 0;   // units of this head before request b_base
            Place at{0, 1}, out{0, 0};   // query buffers to fill, and filling
            if (lane == 0) P.desc[cta] = make_int4(-1, 0, 0, 0);
            __syncwarp();
            auto push = [&](uint32_t k, const Seg &s) {   // (any subset of lanes, each its own k)
                const uint32_t slot = k & (SEGS - 1);
                const bool free = mbar_wait(seg_empty + 8 * slot, (k / SEGS & 1) ^ 1, dead);
                if (free) {
                    segs[slot] = s;
                    mbar_arrive(seg_full + 8 * slot);
                }
                return free;
            };
#pragma unroll 1
            for (bool more = lo < hi, ended = false; ok;) {
#pragma unroll 1
                while (ok && more && pushed - done < 12) {
                    if (fresh) {
                        if (A.B > SMALL_BATCH) look(b_base);
                        m = 0;
                        fresh = false;
                    }
                    // row tile m of each of them, as far as it lies in [lo, hi)
                    const int w = weight_of(P, r, m);
                    const int per = (r.nt + P.overhead) * w;
                    const long long mine =
                        kvh * W + pre + first + (long long)m * (r.nt + P.overhead) * (P.weighted ? W_TWO : 1);
                    Seg s;
                    s.row0 = r.row0, s.n = r.n, s.len = r.len, s.M = r.M, s.lo = r.lo, s.w0 = r.w0, s.ns = r.ns, s.nt = r.nt;
                    s.b = b_base + lane;
                    s.kvh = kvh;
                    s.m = m;
                    // (a key tile is its last unit's: the CTA of the row tile's last unit has its last key tile)
                    s.t0 = max((int)over_weight((uint32_t)min(max(lo - mine, 0ll), (long long)per), w) - P.overhead, 0);
                    s.t1 = (int)over_weight((uint32_t)min(max(hi - mine, 0ll), (long long)per), w) - P.overhead;
                    // a short segment among others is one group's alone: the groups then work on two segments at
                    // a time, and neither waits for the other at the end
                    s.solo = APART && s.M <= TILE && s.t1 - s.t0 <= SOLO_TILES && hi - lo >= 4 * per;
                    const bool any = r.nt && m < r.mt && s.t1 > s.t0;   // (else nothing, or the overhead alone)
                    const uint32_t mask = __ballot_sync(0xffffffffu, any);
                    if (any) {
                        ok = push(pushed + __popc(mask & ((1u << lane) - 1)), s);
                        if (s.t0 == 0 && s.t1 < s.nt) {   // begins here and ends elsewhere: in the CTA of its last unit
                            const long long last = mine + per;
                            P.desc[cta] = make_int4(s.row0, s.kvh, s.m, s.M << 8 | ((int)((last * nc + T - 1) / T) - 1));
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok);
                    pushed += __popc(mask);
                    if (__any_sync(0xffffffffu, ++m < r.mt)) continue;
                    fresh = true;
                    pre += sum;
                    b_base += SMALL_BATCH;
                    more = kvh * W + pre < hi;
                    if (b_base >= A.B) {
                        kvh++;
                        b_base = 0;
                        pre = 0;
                        more = kvh * W < hi;
                    }
                }
                if (!more && !ended && ok) {
                    Seg s = {};
                    if (lane == 0) ok = push(pushed, s);
                    ok = __all_sync(0xffffffffu, ok);
                    ended = true;
                }
                if (!ok) break;
                // two segments' copies under way where there are buffers; else finish the older one first
                const bool room = issued < pushed && issued - done < min(q_bufs, 2u);
                if (room && (done == issued ? warp_wait(q_empty + 8 * at.stage, at.parity, dead)
                                            : warp_try(q_empty + 8 * at.stage, at.parity))) {
                    const Seg &s = segs[issued & (SEGS - 1)];   // (not written again before its queries are there)
                    const int row0 = s.m * 2 * TILE, rows = min(s.M - row0, 2 * TILE);
                    const bool two = s.two();
                    constexpr int CH = DP / 8, RPW = 32 / CH;   // 16-byte pieces of a row, rows per warp step
                    const int ch = lane % CH;
                    int row = lane / CH, tok = (row0 + row) / P.G, head = row0 + row - tok * P.G;
                    const E *q = static_cast<const E *>(P.q) + s.row0 * P.q_stride + (int64_t)s.kvh * P.G * C.D +
                                 (ch * 8 < C.D ? ch * 8 : 0);
                    const uint32_t bytes = ch * 8 < C.D && !P.zero ? 16 : 0;
                    const uint32_t base = smem_addr(q_p) + (two ? 0 : at.stage) * q_buffer + (ch >> 3) * q_block;
#pragma unroll 2
                    for (; row < rows; row += RPW) {
                        copy16(base + (row >> 7) * q_buffer + (row & 127) * 128 + (((ch & 7) ^ (row & 7)) << 4),
                               q + tok * P.q_stride + (int64_t)head * C.D, bytes);
                        head += RPW;
                        while (head >= P.G) head -= P.G, tok++;
                    }
                    copies_commit();
                    issued++;
                    at.advance(q_bufs);
                } else if (done < issued) {
                    if (issued - done == 2) copies_wait<1>();
                    else copies_wait<0>();
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(q_full + 8 * out.stage);
                    done++;
                    out.advance(q_bufs);
                } else {
                    if (room) ok = false;   // the wait ran out
                    break;                  // (nothing is left)
                }
            }
            copies_wait<0>();
        }
    } else {
        regs_up<208>();
        // Softmax and epilogue: group g, a thread per row.
        Seg s;
        const int g = warp >> 2, lane_row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // this warp's 32 lanes of tensor memory
        const uint32_t t_s = tmem + g * TILE + lanes, t_o = tmem + 2 * TILE + lanes;
        const int D = C.D, Hq = P.Hq;
        const bool leader = elect();
        // S tiles taken; products, key tiles, epilogues; barriers of both groups
        uint32_t ns_ = 0, turn = 0, tiles = 0, parts = 0, joint = 0, pairs = 0;
#pragma unroll 1
        for (int seg = 0; ok && take(seg, s, false); release(seg++)) {
            const Seg &all = segs[seg & (SEGS - 1)];   // what only the ends of a segment need stays there
            const int nt = s.t1 - s.t0;
            const bool two = s.two();
            const int mine = (g ^ turn) & 1;      // this group's row tile, or its first key tile
            const uint32_t tile0 = tiles;
            turn += s.solo ? 1 : nt << two;
            tiles += nt;
            const bool alone = two || s.solo;     // this group's rows are its own
            if (!two && mine >= (s.solo ? 1 : nt)) continue;   // the other group's turn
            const bool pair = !alone && nt > 1;   // both groups hold a part of every row
            const bool few = APART && s.M <= FEW_ROWS;
            const int row = lane_row ^ (few && g ? DOWN : 0);
            const int rows = min(s.M - s.m * 2 * TILE, 2 * TILE);   // of this row tile
            const int rt = two ? mine * TILE + row : row;           // this thread's row of it
            const bool active = rt < rows;
            const bool warp_on = (two ? mine * TILE : 0) + (((warp & 3) * 32) ^ (few && g ? DOWN : 0)) < rows;
            const int pos = s.len - s.n + (s.m * 2 * TILE + rt) / P.G;
            float m = -INFINITY, l = 0.f;
            bool any_tile = false;
#pragma unroll 1
            for (int t = alone ? 0 : mine; t < nt; t += alone ? 1 : 2) {
                const int base = s.base(s.t0 + t);
                const bool whole = whole_tile(P, s, base);
                if (!whole && (!two || mine == 0)) {   // (while this tile's scores are made)
                    const uint32_t round = (tile0 + t) / v_stages, stage = tile0 + t - round * v_stages;
                    if (!warp_wait(v_full + 8 * stage, round & 1, dead)) {
                        ok = false;
                        break;
                    }
                    if (clean_values<E, DP>(P, s, base, row, v_p + stage * STAGE)) patched[4 * g + (seg & 3)] = seg;
                    fence_proxy_async();
                    __syncwarp();
                }
                if (!warp_wait(s_full + 8 * g, ns_++ & 1, dead)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if ((warp & 3) == 0 && lane == 0 && (!two || mine)) mbar_arrive(k_empty + 8 * ((tile0 + t) % k_stages));
                if (APART && two && !whole) {   // the other group's product reads this V tile too
                    if (lane == 0) mbar_arrive(both);
                    if (!warp_wait(both, joint++ & 1, dead)) {
                        ok = false;
                        break;
                    }
                }
                if (warp_on) {
                    uint32_t x[4][32];   // a thread's 128 scores
                    if (!whole) {   // hide what this row does not see, in place: one copy of the code, off the main path
#pragma unroll 1
                        for (int i = 0; i < TILE; i += 32) {
                            const uint32_t see = seen_mask(P, pos, base + i);
                            tmem_ld32(t_s + i, x[0]);
                            tmem_wait_ld();
                            after_wait32(x[0]);
#pragma unroll
                            for (int k = 0; k < 32; k++) x[0][k] = (see >> k & 1) ? x[0][k] : 0xff800000u;   // -inf
                            tmem_st32(t_s + i, x[0]);
                        }
                        tmem_wait_st();
                    }
                    float top[4] = {m, m, m, m};
                    auto largest = [&](const uint32_t *v) {
#pragma unroll
                        for (int k = 0; k < 32; k += 2)
                            top[k / 2 & 3] = max3(top[k / 2 & 3], __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                    };
#pragma unroll
                    for (int i = 0; i < 4; i++) tmem_ld32(t_s + 32 * i, x[i]);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; i++) after_wait32(x[i]);
                    if (APART) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(s_free + 8 * g);
                    }
#pragma unroll
                    for (int i = 0; i < 4; i++) largest(x[i]);
                    if (APART && any_tile) {
                        if (!warp_wait(o_done + 8 * g, ns_ & 1, dead)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    const float new_m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    // lift the running maximum, and scale O and l down, only where it lags too far
                    const bool lift = active && (m == -INFINITY ? new_m > m : (new_m - m) * P.c > LAG);
                    if (__any_sync(0xffffffffu, lift)) {
                        const float f = lift ? ex2((m - new_m) * P.c) : 1.f;
                        if (lift) m = new_m;
                        if (any_tile) {
                            l *= f;
                            // (the group's last product is complete: with P apart waited for above,
                            // else issued before this S)
#pragma unroll 1
                            for (int i = 0; i < D; i += 32) {
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
                    const uint64_t cc = pair_of(P.c, P.c), offs = pair_of(off, off);
                    // (l is the fp32 weights' own sum; for the product with v they are rounded to the cache's
                    // type, the only operand that the matrix instruction takes beside such a v.  The outputs'
                    // error against 64 bits is then 0.0022 relative in bf16 and 0.00021 in fp16, where weights
                    // of 32 bits, as a plain form has them, leave 0.0017 and 0.00018: the output's rounding.)
                    uint64_t sum[2] = {0, 0};
                    auto weights = [&](const uint32_t *v, int i) {
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            float a, b;
                            split(fma2(pair_of(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), cc, offs), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            sum[k / 2 & 1] = add2(sum[k / 2 & 1], pair_of(a, b));
                            w[k / 2] = Num<E>::down(a, b);
                        }
                        tmem_st16(t_s + P_COL + 16 * i, w);
                    };
#pragma unroll
                    for (int i = 0; i < 4; i++) weights(x[i], i);
                    float s0, s1;
                    split(add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1;
                    tmem_wait_st();
                }
                if (APART && !warp_on) {
                    // a warp without rows keeps step: a second arrival while another warp still owes its
                    // first would pass for that one's
                    if (lane == 0) mbar_arrive(s_free + 8 * g);
                    if (any_tile && !warp_wait(o_done + 8 * g, ns_ & 1, dead)) {
                        ok = false;
                        break;
                    }
                }
                // the group's last product is through with its weights, which these replace, and its V tile
                // (two arrivals free a tile: one of each group, or both of the one that used it)
                if (APART && any_tile && (warp & 3) == 0 && lane == 0)
                    mbar_arrive(v_empty + 8 * ((tile0 + t - (alone ? 1 : 2)) % v_stages), two ? 1 : 2);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * g);
                // with P apart the group issues its P V itself: its last warp, which has no rows of its own
                // unless the row tile has more than 96
                if (APART && (warp & 3) == 3) {
                    const uint32_t round = (tile0 + t) / v_stages, stage = tile0 + t - round * v_stages;
                    ok = warp_wait(p_full + 8 * g, (ns_ - 1) & 1, dead) && warp_wait(v_full + 8 * stage, round & 1, dead);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        issue_o(g, stage, any_tile);
                        mma_commit(o_done + 8 * g);
                    }
                    __syncwarp();
                }
                any_tile = true;
            }
            // (what the epilogue needs of the segment, while the last product runs)
            const int rr = all.m * 2 * TILE + rt, tok = pos - all.len + all.n;
            const bool direct = all.t0 == 0 && all.t1 == all.nt;
            const int slot = 2 * cta + (all.t0 > 0 ? 0 : 1);
            const int64_t orow = (int64_t)(all.row0 + tok) * Hq + all.kvh * P.G + rr - tok * P.G;
            if (ok) ok = warp_wait(o_done + 8 * g, APART ? (ns_ - 1) & 1 : parts & 1, dead);
            parts++;
            if (APART && ok && (warp & 3) == 0 && lane == 0) {
                const int last = alone ? nt - 1 : nt - 1 - ((nt - 1 - mine) & 1);   // this group's last key tile
                mbar_arrive(v_empty + 8 * ((tile0 + last) % v_stages), two ? 1 : 2);
            }
            if (ok && pair) {   // the other group's maxima, sums and O
                ex[g * TILE + row] = make_float2(m, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(both);
                ok = warp_wait(both, joint++ & 1, dead);
            }
            if (!ok) break;
            tc_fence_after();
            float2 part0 = {}, part1 = {};   // the groups' (m, l) of this row
            if (pair) part0 = ex[row], part1 = ex[TILE + row];
            if (pair && few) {   // (the barrier that ends a pair: group 1's part is handed over, and both have read ex, before it)
                if (g && warp_on) {
                    const float f = part1.x == fmaxf(part0.x, part1.x) ? 1.f : ex2((part1.x - part0.x) * P.c);
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(t_o + TILE + c, o);
                        tmem_wait_ld();
                        after_wait32(o);
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(handed + row * (DP + 4) + c + i) =
                                make_float4(__uint_as_float(o[i]) * f, __uint_as_float(o[i + 1]) * f, __uint_as_float(o[i + 2]) * f,
                                            __uint_as_float(o[i + 3]) * f);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(both + 8);
                ok = warp_wait(both + 8, pairs++ & 1, dead);
                if (!ok) break;
                if (g) continue;
            }
            const bool patch = patched[seg & 3] == seg || patched[4 + (seg & 3)] == seg, broken = bad[seg & 15] == seg + 1;
            if (warp_on) {
                // the part's maximum and sum, and the factors of the (up to) two sums O
                float f0 = 1.f, f1 = 0.f;
                if (pair) {
                    m = fmaxf(part0.x, part1.x);
                    f0 = part0.x == m ? 1.f : ex2((part0.x - m) * P.c);
                    f1 = part1.x == m ? 1.f : ex2((part1.x - m) * P.c);
                    l = part0.y * f0 + part1.y * f1;
                }
                if (broken) l = NAN;
                const float inv = (l == 0.f && !direct) ? 0.f : rcp(l);
                f0 *= inv;
                f1 *= inv;
                const float lse2 = l == 0.f ? -INFINITY : m * P.c + lg2(l) - BIAS;
                const uint32_t t0_ = pair ? t_o : t_o + g * TILE;
                const bool halves = pair && !few;
                const int c0 = halves ? g * (DP / 2) : 0, c1 = min(D, halves ? c0 + DP / 2 : DP);
#pragma unroll 1
                for (int c = c0; c < c1; c += 32) {
                    uint32_t a[32], b[32];
                    tmem_ld32(t0_ + c, a);
                    if (halves) tmem_ld32(t0_ + TILE + c, b);
                    tmem_wait_ld();
                    after_wait32(a);
                    after_wait32(b);
                    float o[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) o[i] = __uint_as_float(a[i]) * f0;
                    if (halves) {
#pragma unroll
                        for (int i = 0; i < 32; i++) o[i] = fmaf(__uint_as_float(b[i]), f1, o[i]);
                    } else if (pair) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 x = *reinterpret_cast<const float4 *>(handed + row * (DP + 4) + c + i);
                            o[i] += x.x * inv, o[i + 1] += x.y * inv, o[i + 2] += x.z * inv, o[i + 3] += x.w * inv;
                        }
                    }
                    if (active) {
                        if (direct) {
                            E *to = static_cast<E *>(P.out) + orow * D + c;
#pragma unroll
                            for (int i = 0; i < 32; i += 8)
                                if (c + i < c1) *reinterpret_cast<uint4 *>(to + i) = pack8<E>(o + i);
                        } else {
                            float4 *to = reinterpret_cast<float4 *>(P.part_o + ((int64_t)slot * PART_ROWS + rt) * DP + c);
#pragma unroll
                            for (int i = 0; i < 8; i++)
                                if (c + i * 4 < c1) to[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                    }
                    __syncwarp();
                }
                if (patch && active) {
                    add_non_finite<E>(C, P, all, pos, c0, c1, [&](int d, float x) {
                        if (direct) {
                            E &y = static_cast<E *>(P.out)[orow * D + d];
                            y = (E)((float)y + x);
                        } else {
                            P.part_o[((int64_t)slot * PART_ROWS + rt) * DP + d] += x;
                        }
                    });
                }
                if (active && c0 == 0) {
                    if (!direct) P.part_lse[slot * PART_ROWS + rt] = lse2;
                    else if (P.lse) P.lse[orow] = lse2 * 0.6931471805599453f;
                }
            }
            tc_fence_before();
            if (pair && !few) {   // neither group's next product may overwrite an O that the other still reads
                __syncwarp();
                if (lane == 0) mbar_arrive(both + 8);
                ok = warp_wait(both + 8, pairs++ & 1, dead);
            }
        }
        if (APART && !ok && (warp & 3) == 3) {   // as the matrix warp does
            if (leader) mma_commit(drained + 8 + 8 * g);
            const uint32_t t0 = now_ns32();
            while (!mbar_try(drained + 8 + 8 * g, 0) && now_ns32() - t0 < WAIT_NS) {}
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

// Four columns (from 4 sub on) of a joined row, and its lse.
template <typename E>
__device__ __forceinline__ void store_joined(const AttnArgs &P, const Cache &C, int4 d, int rt, int sub, float4 o, float sum,
                                             float top) {
    if (sub * 4 >= C.D) return;
    const float inv = 1.f / sum;
    const int rr = d.z * 2 * TILE + rt, tok = rr / P.G;
    const int64_t orow = (int64_t)(d.x + tok) * P.Hq + d.y * P.G + rr - tok * P.G;
    *reinterpret_cast<uint2 *>(static_cast<E *>(P.out) + orow * C.D + sub * 4) =
        make_uint2(Num<E>::down(o.x * inv, o.y * inv), Num<E>::down(o.z * inv, o.w * inv));
    if (P.lse && sub == 0) P.lse[orow] = (top + log2f(sum)) * 0.6931471805599453f;
}

// Joins the parts of the row tiles that several CTAs hold, in order of the CTAs, and sets the rows
// that no request uses.  Blocks (c, y): rows y, y + ny, ... of the row tile that begins in CTA c; the last y
// has the rows that no request uses.
// Many rows of few parts (long draft chains): a row per DP / 4 lanes.  Else a row's parts are spread over
// the block, 16 bytes of a part per thread, and the thread groups' sums are added in shared memory: one
// long request's parts (19 for 131 072 keys) then come in one round trip.
template <typename E, int DP>
__global__ void __launch_bounds__(256) join_kernel(const Batch A, const Cache C, const AttnArgs P) {
    constexpr int TPP = DP / 4, LANES = 256 / TPP;   // threads per part, parts at a time
    __shared__ float weight[MAX_CTAS];
    __shared__ float4 sums[LANES][TPP];
    __shared__ float red[2][8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ny = gridDim.y - 1;
    grid_wait();
    if ((int)blockIdx.y < ny) {
        const int4 d = P.desc[blockIdx.x];
        if (d.x < 0) return;
        const int rows = min((d.w >> 8) - d.z * 2 * TILE, 2 * TILE), first = blockIdx.x, parts = (d.w & 255) - first + 1;
        auto slot = [&](int p) { return 2 * (first + p) + (p == 0); };
        if (parts <= TPP && rows > 2 * ny) {
            const int sub = lane % TPP;
            for (int r0 = blockIdx.y * LANES; r0 < rows; r0 += ny * LANES) {   // (the whole warp)
                const int rt = r0 + tid / TPP;
                const bool on = rt < rows;
                const float v = on && sub < parts ? P.part_lse[slot(sub) * PART_ROWS + rt] : -INFINITY;
                const float4 *from = reinterpret_cast<const float4 *>(P.part_o + (int64_t)rt * DP) + sub;
                auto part = [&](int p) {
                    return on ? from[(int64_t)slot(p) * PART_ROWS * (DP / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
                };
                const float4 x0 = part(0), x1 = part(1);   // (there are two at least: under way with the weights)
                float top = v;
#pragma unroll
                for (int o = TPP / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float f = v == -INFINITY ? 0.f : ex2(v - top);
                float sum = f;
#pragma unroll
                for (int o = TPP / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                auto add = [&](int p, float4 x) {
                    const float w = __shfl_sync(0xffffffffu, f, lane - sub + p);
                    o.x += w * x.x, o.y += w * x.y, o.z += w * x.z, o.w += w * x.w;
                };
                add(0, x0);
                add(1, x1);
#pragma unroll 2
                for (int p = 2; p < parts; p++) add(p, part(p));
                if (on) store_joined<E>(P, C, d, rt, sub, o, sum, top);
            }
        } else for (int rt = blockIdx.y; rt < rows; rt += ny) {
            const float *lse = P.part_lse + rt;
            const float v = tid < parts ? lse[slot(tid) * PART_ROWS] : -INFINITY;   // (parts <= MAX_CTAS < 256)
            const float *from = P.part_o + (int64_t)rt * DP + (tid % TPP) * 4;
            float4 x[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {   // the first parts' values, under way while the weights come together
                const int p = tid / TPP + i * LANES;
                x[i] = p < parts ? *reinterpret_cast<const float4 *>(from + (int64_t)slot(p) * PART_ROWS * DP)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float top = v;
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (lane == 0) red[0][warp] = top;
            __syncthreads();
            top = red[0][0];
            for (int i = 1; i < 8; i++) top = fmaxf(top, red[0][i]);
            float f = v == -INFINITY ? 0.f : ex2(v - top);   // (NaN where a part is)
            if (tid < parts) weight[tid] = f;
            for (int o = 16; o; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
            if (lane == 0) red[1][warp] = f;
            __syncthreads();
            float sum = 0.f;
            for (int i = 0; i < 8; i++) sum += red[1][i];
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int p0 = tid / TPP; p0 < parts; p0 += 4 * LANES) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int p = p0 + i * LANES;
                    if (p >= parts) break;
                    if (p0 >= LANES) x[i] = *reinterpret_cast<const float4 *>(from + (int64_t)slot(p) * PART_ROWS * DP);
                    const float w = weight[p];
                    o.x += w * x[i].x, o.y += w * x[i].y, o.z += w * x[i].z, o.w += w * x[i].w;
                }
            }
            sums[tid / TPP][tid % TPP] = o;
            __syncthreads();
            if (tid < TPP && tid * 4 < C.D) {
                for (int i = 1; i < LANES; i++) {
                    const float4 y = sums[i][tid];
                    o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
                }
                store_joined<E>(P, C, d, rt, tid, o, sum, top);
            }
            __syncthreads();
        }
        return;
    }
    // unused rows: zeros; the rows of a request in error: NaN.  A warp looks at 32 requests, and up to 64
    // warps share what there is to fill in them: the half of 16 requests of 65 rows that is unused took one
    // warp per 32 requests 150 us.
    const int nb = gridDim.x, groups = (A.B + 31) / 32, shares = max(1, min(64, nb * 8 / groups));
    for (int i = warp * nb + blockIdx.x; i < groups * shares; i += nb * 8) {
        const int share = i / groups, b = (i - share * groups) * 32 + lane;
        int from = 0, to = 0, err = 0, head = 0, tail = 0;
        if (b < A.B) {
            const Span s = span_of(A, C.max_pages << C.page_shift, b);
            err = s.err;
            if (err && share == 0) record_error(P.hdr, err, b);
            int end = s.row0 + A.k_max + 1;
            if (A.row_off) {
                end = A.row_off[b + 1];
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
#pragma unroll 1
            for (int part = 0; part < 3; part++) {   // the request's unused rows; rows before the first, after the last request
                const int r0 = part == 0 ? f : part == 1 ? 0 : e, r1 = part == 0 ? t : part == 1 ? h : A.R;
                const bool nan = part == 0 && er;
                const uint32_t w = nan ? Num<E>::NAN2 : 0u;
                const int64_t n = (int64_t)(r1 - r0) * P.Hq * C.D / 8, hn = (int64_t)(r1 - r0) * P.Hq;
                uint4 *o = reinterpret_cast<uint4 *>(static_cast<E *>(P.out) + (int64_t)r0 * P.Hq * C.D);
#pragma unroll 1
                for (int64_t j = share * 32 + lane; j < n; j += shares * 32) o[j] = make_uint4(w, w, w, w);
                if (P.lse)
#pragma unroll 1
                    for (int64_t j = share * 32 + lane; j < hn; j += shares * 32)
                        P.lse[(int64_t)r0 * P.Hq + j] = nan ? NAN : 0.f;
            }
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
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_heads,
                                (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride * 2, (cuuint64_t)c.head_stride * 2,
                                   (cuuint64_t)c.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(c.page_size < TILE ? c.page_size : TILE), 1, 1}, one[4] = {1, 1, 1, 1};
    return f(map, c.dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, ptr, dims,
             strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             c.head_dim % 64 ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int SMEM_MAX = 232448;

template <typename E, int DP>
static sv_status launch_attention(const Batch &A, const Cache &C, AttnArgs P, const sv_kv_cache &cache, cudaStream_t st) {
    constexpr int STAGE = DP / 64 * BLK;
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return SV_ERR_CUDA;
    P.q_tiles = (A.k_max + 1) * P.G > TILE ? 2 : 1;
    P.q_rows = P.q_tiles == 2 ? TILE : ((A.k_max + 1) * P.G + 7) / 8 * 8;
    P.q_bufs = P.q_tiles == 2 ? 1 : P.q_rows <= 32 ? MAX_QBUFS : 2;
    const int q_bytes = P.q_bufs * P.q_tiles * P.q_rows * DP * 2;
    // values wait longer than keys for their use: the odd stage is theirs
    const int stages = (SMEM_MAX - SMALL - hand_over(DP) - q_bytes) / STAGE;
    // A row tile costs about 4 us beside its key tiles (a first tile's latency, the epilogue, the join),
    // and a key tile 1.0 us at 64 columns, 1.6 at 128.  Ragged 96 requests at 64 columns: 93, 78, 72, 68 us
    // with 1, 2, 3, 4; ragged 64 at 128 columns, full and windowed: 69 and 46, 61 and 42, 60 and 44, 63 and 46.
    P.overhead = DP == 64 ? 4 : 2;
    P.weighted = P.q_tiles == 2;
    P.k_stages = stages / 2 < MAX_STAGES ? stages / 2 : MAX_STAGES;
    P.v_stages = stages - P.k_stages < MAX_STAGES ? stages - P.k_stages : MAX_STAGES;
    const int smem = SMALL + hand_over(DP) + q_bytes + (P.k_stages + P.v_stages) * STAGE;
    // no more CTAs than the batch can have units
    const long long most = (long long)A.B * C.heads * (((long long)(A.k_max + 1) * P.G + 2 * TILE - 1) / (2 * TILE)) *
                           ((((long long)C.max_pages << C.page_shift) + TILE - 1) / TILE + P.overhead);
    int ctas = nsm < MAX_CTAS ? nsm : MAX_CTAS;
    // heads that share lines keep step only if each has a whole number of CTAs: worth up to 5 % of them
    if (C.D * 2 % 128 && cache.head_stride * 2 % 128 && C.heads <= 16 && ctas % C.heads * 20 <= ctas)
        ctas -= ctas % C.heads;
    if (most < ctas) ctas = (int)most;
    // (one limit for every call: another thread's call may come between this and the launch)
    if (cudaFuncSetAttribute(attention_kernel<E, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX) != cudaSuccess)
        return SV_ERR_CUDA;
    // (after a runtime call that brings this host thread to the device: encoding alone does not, and fails in a new thread)
    CUtensorMap mk, mv;
    if (!encode(&mk, cache, cache.k) || !encode(&mv, cache, cache.v)) return SV_ERR_CUDA;
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
    // 8 blocks a row tile: 64 windows of 4096 keys took 61 us, 63 with 16; 16 x 65 rows 161 us, 163 with 4
    const int most_rows = (A.k_max + 1) * P.G;
    cfg.gridDim = dim3(ctas, (most_rows < 8 ? most_rows : 8) + 1);
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
    P.negative = scale < 0.f;
    P.zero = scale == 0.f;
    P.withhold = sv::withholding();
    P.Hq = num_q_heads;
    P.G = num_q_heads / cache.num_heads;
    // (a window that holds every length is none: differences of positions stay in 32 bits)
    P.window = window < (cache.max_pages << C.page_shift) ? window : 0;
    P.sinks = sinks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = cache.head_dim > 64;
    if (cache.dtype == SV_BF16)
        return wide ? launch_attention<__nv_bfloat16, 128>(A, C, P, cache, st)
                    : launch_attention<__nv_bfloat16, 64>(A, C, P, cache, st);
    return wide ? launch_attention<__half, 128>(A, C, P, cache, st) : launch_attention<__half, 64>(A, C, P, cache, st);
}
