// cache_attention8.cu -- spec_attention8: the new tokens' rows attend over a paged cache of e4m3 numbers with
// a scale per block of tokens and head.
//
// One pass over the keys with the running maximum m and sum l of the softmax, as in cache_attention.cu, and the
// same cut of the batch's key tiles into one range per CTA.  What differs is how the products are made: the stored
// numbers go to the tensor cores as they are, so nothing is widened on the way, and the 16-bit operands come to them.
//
// Products.  A key tile is the A operand, its 128 keys (for the scores) or 128 elements (for the output) the M of the
// instruction, and the rows are its N:
//     S^T[key, row] = K q^T,      O^T[element, row] += V^T P^T.
// Few rows then cost few columns, and all warps of a softmax group have work: a thread has one
// key and half of the rows, so a key's scale is a register and the sum of a row is spread over the threads until the end.
// The B operands are sums of 8-bit parts:
//   - a query row, times the power of two that brings its largest element into (224, 448], is q0 + q1 (+ q2 for fp16) with
//     q0 = RN(q) in e4m3, 4 bits, q1 = RN(q - q0) and q2 = RN(q - q0 - q1) in e5m2, 3 bits and a sign each: 4 + 1 + 3 (+ 1 + 3)
//     bits hold the 8 of a bf16 (11 of an fp16) without loss from 2^-6 on, 2^-13.8 of the row's largest.  Below, q0 has
//     steps of 2^-9, and what is left, 2^-10 or less, is held to 2^-14 (2^-17 by two parts): 2^-21.8 (2^-24.8) of the largest.
//     The parts are added up along K, in one accumulator: the keys are read twice (three times),
//     which costs less than the columns that parts side by side would take and a thread would have to add;
//   - a weight in fp16 is a sum of its top byte, the top byte of the rest, and so on: an fp16's top byte is an e5m2
//     number.  The parts lie side by side along N, so that the values are read once.  2 (3) of them and the rest rounded
//     to e5m2 hold 9 bits for bf16 (11, all, for fp16).  e5m2 spans 2^-17 to 2^15.8, and the running maximum is kept
//     between 2^12 and 2^15.5, so what is lost of a weight beside its 9 (11) bits is below 2^-28 of a row's largest.
//     (e4m3 parts would end 2^-18 below it: 131 072 small weights would lose a percent of the sum.)
// The score of a key is c ks_j qs_r S (ks: the key's scale, qs: the row's power of two), and the weight that goes to the
// product with v is p vs_j: log2 vs_j is added to the exponent, and m is the maximum of the sums.  l adds p alone.
//
// A CTA works at two ranges at once.  Each has a warp that keeps its queue of segments and loads keys and values
// (tensor copies of pages into two rings) and scales (4-byte copies), one that issues its matrix instructions, and a
// group of 8 softmax warps, which also brings its queries into parts.  While one range changes from a segment to the
// next, the other keeps the memory busy.  A group's warps decide together, at a barrier per tile, whether a maximum
// lags too far; every decision that a barrier depends on is taken that way, so a wait that runs out in one warp ends
// all of them.
//
// What bounds it.  Few rows: the cache's bytes; 256 requests of one row (4 query heads a key head) over 4096 keys of 8
// heads of 128 take 323 us, 317 at the memory's rate (620 in 16 bits).  More rows: the chain of a softmax group from a tile's
// scores to the next one's; with 5 rows a request 365 us, about 3200 cycles a tile and group, while the schedulers issue in
// 54 % of the cycles and the tensor pipe works in 18.  One request of 131 071 keys: the same chain, 27 tiles a range at 1.7 us
// of the 62.  Heads of 64 columns: the tensor copies, 16 rows of 64 bytes each with pages of 16 (one row a request: 290 us;
// 238 with pages of 256).  Long chains (16 x 65 rows, 8 query heads a key head, 8192 keys): the groups' instructions, 11 row
// tiles of 48 rows; 294 us, where the 16-bit kernel's tiles of 128 rows take 161.  Small calls: latency, 11 us.
//
// What was slower (256 x 5 rows): two groups taking the tiles of one segment in turn, 432 us at best; one warp issuing
// both ranges' matrix instructions, 459, at 2000 cycles a tile; barriers polled in tight loops, 463 for 433.  With
// 64 columns, 16-byte copies by the loading warp instead of tensor copies, 689 for 327.
#include "sv_cache8.cuh"
#include "sv_launch.h"
#include "sv_segments.cuh"
#include "sv_tc.cuh"

namespace svc {

constexpr int NTHREADS8 = 640;           // 2 x 8 softmax warps, then
constexpr int W_MMA = 18;                // 16, 17: loads of each range; 18, 19: its matrix instructions
constexpr int MAX_STAGES8 = 7;           // of a ring: keys and values of each range
constexpr int SCALES8 = 8;               // tiles whose scales are kept
constexpr int MOST_K_STAGES = SCALES8 - 2;   // with two S, scales of stages + 1 tiles are awaited or in use beside a new one's
constexpr int MAX_ROWS8 = 48;            // rows of a row tile, at most
constexpr int READERS8 = 9;              // warps that take each segment

template <typename E>
struct Parts;
template <>
struct Parts<__nv_bfloat16> {
    static constexpr int Q = 2, P = 3, ROWS = 48;   // (4 + 2 P) ROWS columns of tensor memory
};
template <>
struct Parts<__half> {
    static constexpr int Q = 3, P = 4, ROWS = 32;
};

struct Attn8Args {
    const void *q;
    int64_t q_stride;
    void *out;
    float *lse;
    int32_t *hdr;
    int4 *desc;        // as in AttnArgs, per range
    float *part_lse;   // [2 * MAX_RANGES][PART]
    float *part_o;     // [2 * MAX_RANGES][PART][pitch]
    float c;           // scale log2(e) 2^shift
    int shift;         // 64 for a scale so small that its product with a key's scale might have too few bits, else 0: rows
                       // of bf16's largest numbers, 2^127, need one of 2^-127 for scores of 1
    int withhold;
    int Hq, G, window, sinks;
    int k_stages, v_stages;   // of each range
    int overhead;      // cost of a row tile beside its key tiles, in key tiles
    int tile_rows;     // rows of a row tile at most
    int pitch;         // of part_o: 64 or 128

    // Row tiles of M rows: as few as it takes, of one height, a multiple of 8.
    static constexpr int PART = MAX_ROWS8, MAX_RANGES = 2 * MAX_CTAS, RANGE_BITS = 10;
    __device__ __forceinline__ int tiles_of(int M) const { return (M + tile_rows - 1) / tile_rows; }
    __device__ __forceinline__ int height(int M) const {
        const int mt = tiles_of(M);
        return mt <= 1 ? M : ((M + mt - 1) / mt + 7) & ~7;
    }
    __device__ __forceinline__ int first_row(int M, int m) const { return m * height(M); }
    __device__ __forceinline__ int rows_of(int M, int m) const { return min(M - m * height(M), height(M)); }
};

// What stands in shared memory before the rings; [2]: of each range.
struct Small8 {
    uint64_t k_full[2][MAX_STAGES8], k_empty[2][MAX_STAGES8], v_full[2][MAX_STAGES8], v_empty[2][MAX_STAGES8];
    uint64_t s_full[2][2], s_free[2][2], p_full[2], o_done[2], q_full[2], drained[2];
    uint64_t seg_full[2][SEGS], seg_empty[2][SEGS];
    int dead, tmem, patched[2], bad[2][16];
    int k_info[2][MAX_STAGES8], v_info[2][MAX_STAGES8];   // of a stage's tile, as the loading warp notes it: see INFO_*
    long long scan[24];
    Seg segs[2][SEGS];
    float scale[2][SCALES8][32];                  // a tile's scales of keys (16) and of values
    __align__(16) float q_scale[2][MAX_ROWS8];
    int q_place[2][MAX_ROWS8];                    // a row's token of the request << 16 | head of the group
    __align__(16) float neg_m[2][MAX_ROWS8];      // BIAS - m; 0 before a row has a maximum
    __align__(16) float lift[2][MAX_ROWS8];
    int set[2][MAX_ROWS8];                        // whether a row has a maximum
    int top[2][4][MAX_ROWS8];
    float sum[2][4][MAX_ROWS8];
    float factor[2][MAX_ROWS8];
};
constexpr int SMALL8 = (sizeof(Small8) + 1023) / 1024 * 1024;
constexpr int INFO_FIRST = 0x100;   // a segment's first tile; the low byte: columns of a part, or 0 at the end of the range

constexpr float BIAS8 = 12.f;      // log2 of the largest weight, for a maximum that does not lag
constexpr float MOST8 = 15.5f;     // and the largest that may be: 57344 is e5m2's last number

// fp32 numbers as integers of the same order.
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// Descriptor of a tile of WIDTH-byte rows, swizzled over as many bytes, for a product with the rows (K q^T) or the
// columns (V^T P^T) as M.  With 64 columns the upper half of the second's M is no columns: it reads the 8 rows after, and
// reaches only lanes of the output that nothing uses.
template <int WIDTH>
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
    if (WIDTH == 128) return smem_desc(addr, 16);
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(512 >> 4) << 16 | (uint64_t)(512 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)4 << 61;
}
// A matrix descriptor `by` bytes further on (within shared memory's 18 bits, so that nothing is carried).
__device__ __forceinline__ uint64_t further(uint64_t desc, uint32_t by) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(desc));
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo + (by >> 4)), "r"(hi));
    return d;
}

__device__ __forceinline__ uint32_t sub_half2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {   // a in the low half
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}
__device__ __forceinline__ uint32_t e5m2_of(uint32_t half2) {
    __half2_raw h;
    h.x = (unsigned short)half2;
    h.y = (unsigned short)(half2 >> 16);
    return __nv_cvt_halfraw2_to_fp8x2(h, __NV_SATFINITE, __NV_E5M2);
}

// Four fp16 weights (two pairs of rows) as P parts: part i of them in out[i].  3 parts hold 9 bits, so a weight is rounded to
// as many first, and a tie goes up or down by the key's parity (`up`: 2 or 1 in each half).  What is added has to be masked
// away again: the parts hold up to 11 bits of a weight whose bits are not all set, and keep what they can of it, which
// made every output 7e-4 to 1e-3 too large beside the sum of the weights, which are not rounded there.
template <int P>
__device__ __forceinline__ void parts_of(uint32_t a, uint32_t b, uint32_t up, uint32_t *out) {
    if (P == 3) a = (a + up) & 0xfffcfffcu, b = (b + up) & 0xfffcfffcu;
#pragma unroll
    for (int i = 0; i < P; i++) {
        out[i] = __byte_perm(a, b, 0x7531);
        if (i == P - 1) break;
        a = sub_half2(a, a & 0xff00ff00u);
        b = sub_half2(b, b & 0xff00ff00u);
    }
}

// CHUNKS: of 8 rows that a softmax warp may have; a row tile has 16 CHUNKS rows at most.  WIDTH: bytes of a key in a
// stage, 64 where head_dim allows: half the bytes leave room for twice the stages, and the memory's latency needs them
// (256 x 5 rows of 64-wide heads over 4096 keys: 341 us with 128).
template <typename E, int CHUNKS, int WIDTH>
__global__ void __launch_bounds__(NTHREADS8, 1)
attention8_kernel(const Batch A, const Cache8 C, const Attn8Args P, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
    constexpr int QP = Parts<E>::Q, PP = Parts<E>::P, ROWS = 16 * CHUNKS;
    constexpr int S_COLS = ROWS, O_COLS = PP * ROWS;   // two S and one O of each range
    static_assert(4 * S_COLS + 2 * O_COLS <= 512, "tensor memory");
    constexpr int NW = NTHREADS8 / 32;
    constexpr int STAGE8 = TILE * WIDTH, Q_BUFFER = QP * ROWS * 128, P_BUFFER = PP * ROWS * 128;
    extern __shared__ __align__(1024) char smem[];
    Small8 &sm = *reinterpret_cast<Small8 *>(smem);
    // [barriers and small state][rings of K tiles][rings of V tiles][queries of each range][weights of each range]
    char *const k_p = smem + SMALL8, *const v_p = k_p + 2 * P.k_stages * STAGE8, *const q_p = v_p + 2 * P.v_stages * STAGE8;
    char *const p_p = q_p + 2 * Q_BUFFER;
    volatile int *const dead = &sm.dead;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t k_stages = P.k_stages, v_stages = P.v_stages;
    auto bar = [&](const uint64_t &b) { return smem_addr(&b); };

    if (tid < 2) {
        const int w = tid;
        for (int i = 0; i < MAX_STAGES8; i++) {
            mbar_init(bar(sm.k_full[w][i]), 33);    // the copies' bytes, and each lane's scale
            mbar_init(bar(sm.k_empty[w][i]), 1);
            mbar_init(bar(sm.v_full[w][i]), 1);
            mbar_init(bar(sm.v_empty[w][i]), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(bar(sm.s_full[w][i]), 2);     // the products, and the matrix warp (for the scales)
            mbar_init(bar(sm.s_free[w][i]), 8);     // the group's warps
        }
        mbar_init(bar(sm.p_full[w]), 8);
        mbar_init(bar(sm.o_done[w]), 1);
        mbar_init(bar(sm.q_full[w]), 8);
        mbar_init(bar(sm.drained[w]), 1);
        if (w == 0) sm.dead = 0;
    } else if (tid >= 64 && tid < 64 + 4 * SEGS) {
        const int i = tid - 64, w = i / (2 * SEGS), k = i % (2 * SEGS);
        mbar_init(k < SEGS ? bar(sm.seg_full[w][k]) : bar(sm.seg_empty[w][k - SEGS]), k < SEGS ? 1 : READERS8);
    } else if (tid >= 256 && tid < 256 + 32) {
        sm.bad[(tid >> 4) & 1][tid & 15] = 0;
    } else if (tid >= 320 && tid < 322) {
        sm.patched[tid - 320] = -1;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (warp == W_MMA) tmem_alloc(smem_addr(&sm.tmem), 512);
    grid_wait();   // the work before this on the stream may still be writing what follows

    // The batch's units, and where this CTA's ranges begin, as in attention_kernel; range r of `nr` is the first of CTA r,
    // or the second of CTA r - gridDim.x, so that a few ranges lie on as many multiprocessors.
    auto units_of = [&](const Req &r) { return r.nt ? (long long)(r.nt + P.overhead) * r.mt : 0ll; };
    long long W = 0;          // units of one key head
    struct Range {
        long long lo, hi;
        int kvh, nr;          // the key head that it begins in, ranges in all
    };
    auto range = [&](int w) {
        const long long T = W * C.heads;
        Range R = {0, 0, 0, (int)min(2ll * gridDim.x, T)};
        const int id = w * gridDim.x + blockIdx.x;
        if (id < R.nr) {
            const long long q = quotient(T, R.nr);
            const int rest = (int)(T - q * R.nr);
            R.lo = q * id + (long long)rest * id / R.nr;
            R.hi = q * (id + 1) + (long long)rest * (id + 1) / R.nr;
            if (R.lo < R.hi) R.kvh = (int)quotient64(R.lo, W);
        }
        return R;
    };
    long long *const start_pre = sm.scan + NW, *const start_b = sm.scan + NW + 2;
    if (A.B > SMALL_BATCH) {
        __syncthreads();   // (barriers and flags are set)
#pragma unroll 1
        for (int pass = A.B <= NTHREADS8; pass < 2; pass++) {   // pass 0 sums, pass 1 finds
            long long before = 0, at[2] = {-1, -1};
#pragma unroll 1
            for (int b0 = 0; b0 < A.B; b0 += NTHREADS8) {
                const int b = b0 + tid;
                Req r = {};
                if (b < A.B) r = req_of(A, C, P, b);
                const long long u = units_of(r);
                long long inc = u;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                if (b0) __syncthreads();
                if (lane == 31) sm.scan[warp] = inc;
                __syncthreads();
                long long pre = before + inc - u, all = 0;
#pragma unroll 4
                for (int i = 0; i < NW; i++) {
                    const long long x = sm.scan[i];
                    if (i < warp) pre += x;
                    all += x;
                }
                before += all;
                if (pass == 0) continue;
                if (b0 == 0) {
                    if (A.B <= NTHREADS8) W = all;
#pragma unroll
                    for (int w = 0; w < 2; w++) {
                        const Range R = range(w);
                        if (R.lo < R.hi) at[w] = R.lo - R.kvh * W;
                    }
                }
#pragma unroll
                for (int w = 0; w < 2; w++)
                    if (at[w] >= 0 && pre <= at[w] && at[w] < pre + u) start_b[w] = b, start_pre[w] = pre;
            }
            if (pass == 0) W = before;
            __syncthreads();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile int *>(&sm.tmem);
    grid_launch_dependents();
    bool ok = true;

    if (warp >= 16) {
        if (CHUNKS == 3) regs_down<64>();   // to the softmax warps: 4 x 104 + 64 = 5 x 96
        const int w = warp & 1;   // the range
        const bool leader = elect();
        if (warp < W_MMA) {
            // A range's segments, in order, and the keys, values and scales of their tiles.  A lane looks at one of 16
            // requests at a time and hands out its segments; then their tiles are loaded.
            uint32_t pushed = 0;             // segments handed out
            Req r = {};
            long long first = 0, sum = 0;    // this lane's request's first unit, all 16's units
            auto look = [&](int b) {         // at requests b .. b + 15: first and sum from this head's start
                r.nt = r.mt = 0;
                if (lane < SMALL_BATCH && b + lane < A.B) r = req_of(A, C, P, b + lane);
                const long long u = units_of(r);
                sum = u;
#pragma unroll
                for (int o = 1; o < SMALL_BATCH; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                first = sum - u;
                sum = __shfl_sync(0xffffffffu, sum, SMALL_BATCH - 1);
            };
            if (A.B <= SMALL_BATCH) {
                look(0);
                W = sum;
            }
            const Range R = range(w);
            const int id = w * gridDim.x + blockIdx.x;
            if (lane == 0) P.desc[id] = make_int4(-1, 0, 0, 0);
            __syncwarp();
            const bool scanned = A.B > SMALL_BATCH && R.lo < R.hi;
            int kvh = R.kvh, b_base = scanned ? (int)start_b[w] : 0, m = 0;
            long long pre = scanned ? start_pre[w] : 0;   // units of this head before request b_base
            auto push = [&](uint32_t k, const Seg &s) {   // (any subset of lanes, each its own k)
                const uint32_t slot = k & (SEGS - 1);
                const bool free = mbar_wait(bar(sm.seg_empty[w][slot]), (k / SEGS & 1) ^ 1, dead);
                if (free) {
                    sm.segs[w][slot] = s;
                    mbar_arrive(bar(sm.seg_full[w][slot]));
                }
                return free;
            };
            bool fresh = true, more = R.lo < R.hi;
            auto hand_out = [&]() {   // the next segments: one more row tile of each of the 16 requests
                if (fresh) {
                    if (A.B > SMALL_BATCH) look(b_base);
                    m = 0;
                    fresh = false;
                }
                // row tile m of each of them, as far as it lies in [lo, hi)
                const int per = r.nt + P.overhead;
                const long long mine = kvh * W + pre + first + (long long)m * per;
                Seg s;
                s.row0 = r.row0, s.n = r.n, s.len = r.len, s.M = r.M, s.lo = r.lo, s.w0 = r.w0, s.ns = r.ns, s.nt = r.nt;
                s.b = b_base + lane;
                s.kvh = kvh;
                s.m = m;
                s.solo = 0;
                // (the range of the row tile's last unit has its last key tile)
                s.t0 = max((int)min(max(R.lo - mine, 0ll), (long long)per) - P.overhead, 0);
                s.t1 = (int)min(max(R.hi - mine, 0ll), (long long)per) - P.overhead;
                const bool any = r.nt && m < r.mt && s.t1 > s.t0;   // (else nothing, or the overhead alone)
                const uint32_t mask = __ballot_sync(0xffffffffu, any);
                if (any) {
                    ok = push(pushed + __popc(mask & ((1u << lane) - 1)), s);
                    if (s.t0 == 0 && s.t1 < s.nt) {   // begins here and ends elsewhere: in the range of its last unit
                        const long long last = mine + per, T = W * C.heads;
                        P.desc[id] = make_int4(s.row0, s.kvh, s.m, s.M << Attn8Args::RANGE_BITS | ((int)((last * R.nr + T - 1) / T) - 1));
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                pushed += __popc(mask);
                if (__any_sync(0xffffffffu, ++m < r.mt)) return;
                fresh = true;
                pre += sum;
                b_base += SMALL_BATCH;
                more = kvh * W + pre < R.hi;
                if (b_base >= A.B) {
                    kvh++;
                    b_base = 0;
                    pre = 0;
                    more = kvh * W < R.hi;
                }
            };
            const uint32_t k_ring = smem_addr(k_p) + w * k_stages * STAGE8, v_ring = smem_addr(v_p) + w * v_stages * STAGE8;
            const int P_ = 1 << C.page_shift, box = min(P_, TILE), npg = TILE / box, tpl = 32 / npg;
            const int sub = lane & (npg - 1), lane_tile = lane / npg;
            const int per = min(1 << C.block_shift, TILE), blocks = TILE / per;   // tokens per scale, scales per tile and side
            const int blk = lane & 15, blk_tok = blk * per, blk_page = (blk_tok / box) & (npg - 1);
            Place ka{0, 1}, va{0, 1};   // the first round finds every stage empty
            uint32_t k_loads = 0, v_loads = 0;
            for (uint32_t seg = 0; ok; seg++) {
                while (ok && more && pushed == seg) hand_out();
                __syncwarp();
                if (!ok || pushed == seg) break;
                const Seg &s = sm.segs[w][seg & (SEGS - 1)];   // (as this warp wrote it; released below)
                const int t1 = s.t1, ns = s.ns, w0 = s.w0, len = s.len, kv = s.kvh, s_lo = s.lo;
                const int columns = (P.rows_of(s.M, s.m) + 15) & ~15;
                // a lane's page of `tpl` tiles from t on (npg lanes a tile), or -1: one load of the table
                // serves several tiles, and is issued that many tiles ahead of its use
                const int32_t *table = C.table + (int64_t)s.b * C.max_pages;
                auto base_of = [&](int t) { return (t < ns ? t : w0 + t - ns) * TILE; };
                auto fetch = [&](int t) {
                    t += lane_tile;
                    const int j = base_of(t) + sub * box;
                    if (t >= t1 || j >= len || !(j + box > s_lo || j < P.sinks)) return -1;
                    return (int)min((uint32_t)table[j >> C.page_shift], (uint32_t)C.num_pages);   // (num_pages: not a page)
                };
                const int t0 = s.t0, b = s.b;
                int ids = -1, ahead = fetch(t0), t_ids = t0 - tpl;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sm.seg_empty[w][seg & (SEGS - 1)]));
#pragma unroll 1
                for (int t = t0; t < t1; t++) {
                    if (t == t_ids + tpl) {
                        ids = ahead;
                        t_ids = t;
                        ahead = fetch(t + tpl);
                    }
                    // this lane's page of tile t (lanes below npg), or -1, and its block's
                    int page = __shfl_sync(0xffffffffu, ids, (t - t_ids) * npg + sub);
                    const int of_block = __shfl_sync(0xffffffffu, ids, (t - t_ids) * npg + blk_page);
                    if (lane >= npg) page = -1;
                    if (page == C.num_pages) {
                        *reinterpret_cast<volatile int *>(&sm.bad[w][seg & 15]) = seg + 1;
                        record_error(P.hdr, SV_DEV_BAD_PAGE, b);
                        page = -1;
                    }
                    const int base = base_of(t), y = base & (P_ - 1) & ~(box - 1), info = columns | (t == t0 ? INFO_FIRST : 0);
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, page >= 0)) * box * WIDTH;
                    const uint32_t kf = bar(sm.k_full[w][ka.stage]), vf = bar(sm.v_full[w][va.stage]);
                    __syncwarp();   // (a bad page noted by any lane, before the arrival that publishes it)
                    ok = warp_wait(bar(sm.k_empty[w][ka.stage]), ka.parity, dead);
                    if (!ok) break;
                    if (P.withhold && k_loads == 0) {   // (its waits then run out, as they are meant to)
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        sm.k_info[w][ka.stage] = info;
                        mbar_expect(kf, bytes);
                    }
                    __syncwarp();
                    if (page >= 0) tma_load_4d(k_ring + ka.stage * STAGE8 + sub * box * WIDTH, &map_k, kf, 0, y, kv, page);
                    if (blk < blocks && of_block >= 0 && of_block < C.num_pages && base + blk_tok < len) {
                        const int slot = (base + blk_tok) & (P_ - 1);
                        const float *from = lane < 16 ? C.k_scale : C.v_scale;
                        copy4(smem_addr(&sm.scale[w][k_loads & (SCALES8 - 1)][lane]),
                              from + of_block * C.s_page + (slot >> C.block_shift) * C.s_block + kv * C.s_head);
                    }
                    copies_arrive(kf);
                    __syncwarp();
                    k_loads++;
                    ka.advance(k_stages);
                    ok = warp_wait(bar(sm.v_empty[w][va.stage]), va.parity, dead);
                    if (!ok) break;
                    if (lane == 0) {
                        sm.v_info[w][va.stage] = info;
                        mbar_expect(vf, bytes);
                    }
                    __syncwarp();
                    if (page >= 0) tma_load_4d(v_ring + va.stage * STAGE8 + sub * box * WIDTH, &map_v, vf, 0, y, kv, page);
                    __syncwarp();
                    v_loads++;
                    va.advance(v_stages);
                }
            }
            if (ok) {   // the end of the range, for the softmax and the matrix warps
                const Seg end = {};
                if (lane == 0) ok = push(pushed, end);
                ok = __all_sync(0xffffffffu, ok) && warp_wait(bar(sm.k_empty[w][ka.stage]), ka.parity, dead);
            }
            if (ok) {
                if (lane == 0) {
                    sm.k_info[w][ka.stage] = 0;
                    mbar_expect(bar(sm.k_full[w][ka.stage]), 0);
                }
                __syncwarp();
                copies_arrive(bar(sm.k_full[w][ka.stage]));
            }
            copies_commit();
            copies_wait<0>();
            if (!ok) {   // let the copies in flight land before the CTA may end
                const uint32_t since = now_ns32();
                for (uint32_t i = k_loads > k_stages ? k_loads - k_stages : 0; i < k_loads; i++)
                    while (!mbar_try(bar(sm.k_full[w][i % k_stages]), i / k_stages & 1) && now_ns32() - since < WAIT_NS) {}
                for (uint32_t i = v_loads > v_stages ? v_loads - v_stages : 0; i < v_loads; i++)
                    while (!mbar_try(bar(sm.v_full[w][i % v_stages]), i / v_stages & 1) && now_ns32() - since < WAIT_NS) {}
            }
        } else {
            // A range's matrix instructions: a tile's scores as soon as there is an S to put them in, its P V as soon as the
            // weights are there.
            // The whole warp runs this; one lane issues.
            const int steps = (C.D + 31) / 32;         // of 32 elements of a head
            Place ks{0, 0}, vs{0, 0};
            uint32_t n_s = 0, n_o = 0, n_q = 0;        // scores and products issued, queries taken
            bool more = true;                          // the range has not ended
            const uint64_t qd = smem_desc(smem_addr(q_p) + w * Q_BUFFER, 16),
                           pd = smem_desc_plain(smem_addr(p_p) + w * P_BUFFER, 128, 2048);
            auto scores = [&]() {
                const int info = *reinterpret_cast<volatile int *>(&sm.k_info[w][ks.stage]);
                if (info == 0) {
                    more = false;
                    return;
                }
                if (info & INFO_FIRST) {
                    // (the queries come when the segment before is done, so no product is waited for meanwhile)
                    ok = warp_wait(bar(sm.q_full[w]), n_q++ & 1, dead);
                    if (!ok) return;
                }
                tc_fence_after();
                if (leader) {
                    const int columns = info & 0xff;
                    const uint64_t kd = tile_desc<WIDTH>(smem_addr(k_p) + (w * k_stages + ks.stage) * STAGE8);
                    const uint32_t d = tmem + (2 * w + (n_s & 1)) * S_COLS;
#pragma unroll
                    for (int part = 0; part < QP; part++) {
                        const uint32_t idesc = mma8_idesc(part > 0, columns, false);
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            if (k < WIDTH / 32 && k < steps)
                                mma8_ss(d, further(kd, k * 32), further(qd, part * columns * 128 + k * 32), idesc, part > 0 || k > 0);
                    }
                    mbar_arrive(bar(sm.s_full[w][n_s & 1]));   // (it has waited for the keys, and so for the scales)
                    mma_commit(bar(sm.s_full[w][n_s & 1]));
                    mma_commit(bar(sm.k_empty[w][ks.stage]));
                }
                __syncwarp();
                n_s++;
                ks.advance(k_stages);
            };
            auto product = [&]() {
                tc_fence_after();
                const int info = *reinterpret_cast<volatile int *>(&sm.v_info[w][vs.stage]);
                if (leader) {
                    const uint32_t idesc = mma8_idesc(true, PP * (info & 0xff), true);
                    const uint64_t vd = tile_desc<WIDTH>(smem_addr(v_p) + (w * v_stages + vs.stage) * STAGE8);
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        mma8_ss(tmem + 4 * S_COLS + w * O_COLS, further(vd, k * 32 * WIDTH), further(pd, k * 512), idesc,
                                !(info & INFO_FIRST) || k > 0);
                    mma_commit(bar(sm.o_done[w]));
                    mma_commit(bar(sm.v_empty[w][vs.stage]));
                }
                __syncwarp();
                n_o++;
                vs.advance(v_stages);
            };
            uint32_t idle_since = 0, polls = 0;
#pragma unroll 1
            while (ok && (more || n_o < n_s)) {
                // both are asked at once; every lane has to have seen it.  A segment's first S waits until the products of the
                // one before are issued, since its queries come after them.
                uint32_t there = 0;
                if (more && mbar_test(bar(sm.k_full[w][ks.stage]), ks.parity) && mbar_test(bar(sm.s_free[w][n_s & 1]), (n_s >> 1 & 1) ^ 1)) there = 1;
                if (n_o < n_s && mbar_test(bar(sm.p_full[w]), n_o & 1) && mbar_test(bar(sm.v_full[w][vs.stage]), vs.parity)) there |= 2;
                there = __reduce_and_sync(0xffffffffu, there);
                if (there & 2) product();
                const bool next = (there & 1) &&
                                  (n_s == n_o || !(*reinterpret_cast<volatile int *>(&sm.k_info[w][ks.stage]) & INFO_FIRST));
                if (next) scores();
                if (next || there & 2) {
                    idle_since = 0;
                } else if (!(++polls & 255)) {
                    const uint32_t now = now_ns32() | 1;
                    if (!idle_since) idle_since = now;
                    if (__any_sync(0xffffffffu, *dead || now - idle_since > WAIT_NS)) {
                        *dead = 1;
                        ok = false;
                    }
                }
            }
            if (!ok) {   // wait for the matrix instructions in flight before tensor memory is given back
                if (leader) mma_commit(bar(sm.drained[w]));
                const uint32_t since = now_ns32();
                while (!mbar_try(bar(sm.drained[w]), 0) && now_ns32() - since < WAIT_NS) {}
            }
            __syncwarp();
        }
    } else {
        if (CHUNKS == 3) regs_up<104>();
        // Softmax and epilogue of range g: two threads per key of a tile, which have its rows by turns of 8.
        const int g = warp >> 3, half = warp >> 2 & 1, key = (warp & 3) * 32 + lane, place = tid & 255;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // this warp's 32 lanes of tensor memory
        const uint32_t t_s = tmem + 2 * g * S_COLS + lanes, t_o = tmem + 4 * S_COLS + g * O_COLS + lanes;
        const int block = key >> min(C.block_shift, 7);               // of this thread's key in a tile
        char *const q_at = q_p + g * Q_BUFFER;
        char *const p_at = p_p + g * P_BUFFER + (key >> 3) * 128 + (key & 7) * 16 + half * 8;
        const uint32_t tie = key & 1 ? 0x00020002u : 0x00010001u;      // see parts_of
        auto any_of = [&](bool x) { return barrier_any(1 + g, 256, x); };
        const float *const q_scale = sm.q_scale[g];
        const int *const q_place = sm.q_place[g];
        float *const neg_m = sm.neg_m[g], *const lift = sm.lift[g];
        uint32_t done = 0;                                            // tiles
        Place vp{0, 0};
#pragma unroll 1
        for (int seg = 0;; seg++) {
            ok = warp_wait(bar(sm.seg_full[g][seg & (SEGS - 1)]), seg / SEGS & 1, dead);
            if (any_of(!ok)) break;
            const Seg &s = sm.segs[g][seg & (SEGS - 1)];   // (its fields are read where they are needed)
            if (s.nt == 0) break;
            const int rows = P.rows_of(s.M, s.m), rp = (rows + 15) & ~15;
            const int t1 = s.t1, ns = s.ns, w0 = s.w0, shared = s.len - s.n;   // (tokens that every row sees, but for the window)
            {   // queries in parts, swizzled as the matrix instruction reads them (no product reads the last ones any more)
                const int lpr = C.D > 64 ? 16 : 8, rpp = 256 / lpr;   // lanes of a row, rows per pass of the group
                const int ch = place & (lpr - 1), row0 = P.first_row(s.M, s.m);
                const E *q = static_cast<const E *>(P.q) + s.row0 * P.q_stride + (int64_t)s.kvh * P.G * C.D + ch * 8;
                uint4 raw[CHUNKS];
                int at[CHUNKS];
#pragma unroll
                for (int i = 0; i < CHUNKS; i++) {   // (256 / 16 rows at least a pass)
                    const int row = place / lpr + i * rpp, rr = row0 + row, tok = rr / P.G, head = rr - tok * P.G;
                    raw[i] = make_uint4(0u, 0u, 0u, 0u);
                    at[i] = tok << 16 | head;
                    if (row < rows && ch * 8 < C.D) raw[i] = *reinterpret_cast<const uint4 *>(q + tok * P.q_stride + (int64_t)head * C.D);
                }
#pragma unroll
                for (int i = 0; i < CHUNKS; i++) {
                    const int row = place / lpr + i * rpp;
                    if (i * rpp >= rp) break;   // (the whole group)
                    float x[8], top = 0.f;
                    unpack8<E>(raw[i], x);
                    bool finite = true;
#pragma unroll
                    for (int e = 0; e < 8; e++) top = fmaxf(top, fabsf(x[e])), finite = finite && fabsf(x[e]) < INFINITY;
                    if (!finite) top = INFINITY;
                    for (int o = lpr / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // the power of two 2^k with top in (224, 448] 2^k, up to 2^120 for a finite top; rows below 2^-117 have
                    // 2^-126, where the last bit of a bf16, 2^-133, is 2^-7 and so exact
                    const uint32_t b = __float_as_uint(top);
                    const int k = max((int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7), -126);
                    const float inv = __uint_as_float((uint32_t)(127 - k) << 23);
                    if (row >= rp) continue;
                    if (ch == 0) {
                        // (2^-126 at least: with a shift the scores are none to speak of there)
                        sm.q_scale[g][row] = top < INFINITY ? __uint_as_float((uint32_t)max(127 + k - P.shift, 1) << 23) : NAN;
                        sm.q_place[g][row] = at[i];
                    }
#pragma unroll
                    for (int e = 0; e < 8; e++) x[e] *= inv;
#pragma unroll
                    for (int part = 0; part < QP; part++) {
                        uint32_t two[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            float2 y;
                            if (part == 0) {
                                two[e] = pack_e4m3(x[2 * e], x[2 * e + 1]);
                                y = unpack_e4m3(two[e]);
                            } else {
                                two[e] = e5m2_of(half2_of(x[2 * e], x[2 * e + 1]));   // (the rest has at most 7 bits)
                                y = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two[e], __NV_E5M2)));
                            }
                            x[2 * e] -= y.x;
                            x[2 * e + 1] -= y.y;
                        }
                        const int n = part * rp + row;
                        *reinterpret_cast<uint2 *>(q_at + n * 128 + (((ch >> 1) ^ (n & 7)) << 4) + (ch & 1) * 8) =
                            make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sm.q_full[g]));
            }
            uint64_t l[CHUNKS][4];   // pairs of rows
#pragma unroll
            for (int c = 0; c < CHUNKS; c++)
#pragma unroll
                for (int i = 0; i < 4; i++) l[c][i] = 0;
            if (place < MAX_ROWS8) neg_m[place] = 0.f, sm.set[g][place] = 0;
            any_of(false);
            bool any_tile = false, pending = true;   // whether O holds something, and a row may be without a maximum
            bool failed = false;                     // (the group's decision; `ok` is this warp's alone)
#pragma unroll 1
            for (int t = s.t0; t < t1; t++) {
                const int base = (t < ns ? t : w0 + t - ns) * TILE, j = base + key;
                const bool whole = base + TILE - 1 <= shared && (!P.window || whole_tile(P, s, base));
                if (!whole && !seen_by_all(P, s, j)) {   // a value that must not reach the product as it is
                    ok = ok && mbar_wait(bar(sm.v_full[g][vp.stage]), vp.parity, dead);
                    uint4 *const row = reinterpret_cast<uint4 *>(v_p + (g * v_stages + vp.stage) * STAGE8 + key * WIDTH);
                    constexpr int HALF = WIDTH / 32;     // 16-byte pieces of a half of it
                    // (each half of the threads has half of its bytes, a different bank per lane)
                    if (!seen_by_any(P, s, j)) {         // (a slot never written may hold NaN, and 0 * NaN is NaN)
#pragma unroll
                        for (int i = 0; i < HALF; i++) row[(HALF * half + i) ^ (key & (2 * HALF - 1))] = make_uint4(0u, 0u, 0u, 0u);
                    } else {                             // (the epilogue gives its NaN to the rows that see it)
                        bool took = false;
#pragma unroll 1
                        for (int i = HALF * half; i < HALF * half + HALF; i++) {
                            uint4 v = row[i ^ (key & (2 * HALF - 1))];
                            uint32_t *p = &v.x;
                            bool hit = false;
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const uint32_t nan = __vcmpeq4(p[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                p[e] &= ~nan;
                                hit |= nan != 0;
                            }
                            if (hit) row[i ^ (key & (2 * HALF - 1))] = v, took = true;
                        }
                        if (took) *reinterpret_cast<volatile int *>(&sm.patched[g]) = seg;
                    }
                }
                if (!whole) __syncwarp();
                // Rows lie in order of their tokens, so those that see this key are neighbours: tokens from the key's own on,
                // up to the last whose window has it.
                int from = 0, to = 0x7fffffff;
                if (!whole) {
                    const int first = j - shared, row0 = P.first_row(s.M, s.m);
                    from = min(max(first, 0), s.n) * P.G - row0;
                    // (and never the rows that fill the tile up: a slot that was not loaded must not lift anything)
                    to = P.window && j >= P.sinks ? min(min(max(first + P.window, 0), s.n) * P.G - row0, rows) : rows;
                }
                // the scores (and the scales that came with the keys) and the last product: asked at once, and waited for where they
                // are not there yet
                const uint32_t buffer = done & 1;
                uint32_t there = mbar_test(bar(sm.s_full[g][buffer]), done >> 1 & 1) |
                                 (uint32_t)mbar_test(bar(sm.o_done[g]), (done - 1) & 1) << 2;
                there = __reduce_and_sync(0xffffffffu, there);
                if (!(there & 1)) ok = warp_wait(bar(sm.s_full[g][buffer]), done >> 1 & 1, dead) && ok;
                tc_fence_after();
                const float *const scales = sm.scale[g][done & (SCALES8 - 1)];
                const float ck = P.c * clean_scale(scales[block]);
                const float lvs = lg2(clean_scale(scales[16 + block])), rvs = ex2(-lvs);
                bool waited = !any_tile;
                auto last_product = [&]() {   // the group's last product is through with its weights, its V tile and O
                    if (waited) return;
                    if (!(there & 4)) {
                        ok = warp_wait(bar(sm.o_done[g]), (done - 1) & 1, dead) && ok;
                        tc_fence_after();
                    }
                    waited = true;
                };
                // exponents of the weights: scores in powers of two, with the value's scale, from the row's maximum on.  A second
                // time where a maximum had to be lifted.
                const uint64_t cc = pair_of(ck, ck), ll = pair_of(lvs, lvs), rr = pair_of(rvs, rvs);
                uint64_t u[CHUNKS][4];   // pairs of rows
#pragma unroll 1
                for (int pass = 0;; pass++) {
                    float most = -INFINITY;
#pragma unroll
                    for (int c = 0; c < CHUNKS; c++) {
                        const int r0 = 16 * c + 8 * half;
                        if (r0 >= rows) break;
                        uint32_t x[8];
                        tmem_ld8(t_s + buffer * S_COLS + r0, x);
                        tmem_wait_ld();
                        after_wait<8>(x);
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const ulonglong2 qs = *reinterpret_cast<const ulonglong2 *>(q_scale + r0 + 2 * i),
                                             nm = *reinterpret_cast<const ulonglong2 *>(neg_m + r0 + 2 * i);
                            auto score = [&](int k) { return pair_of(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])); };
                            u[c][i] = add2(fma2(score(i), mul2(cc, qs.x), ll), nm.x);
                            u[c][i + 1] = add2(fma2(score(i + 1), mul2(cc, qs.y), ll), nm.y);
                        }
                        if (!whole) {   // rows from `from` up to `to` see this key
                            // (their comparisons stay in here: taken out of the loop they were a fifth of its instructions)
                            int f = from, e = to;
                            asm volatile("" : "+r"(f), "+r"(e));
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                float y, z;
                                split(u[c][i], y, z);
                                const int r = r0 + 2 * i;
                                u[c][i] = pair_of(r >= f && r < e ? y : -INFINITY, r + 1 >= f && r + 1 < e ? z : -INFINITY);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            float y, z;
                            split(u[c][i], y, z);
                            most = max3(most, y, z);
                        }
                    }
                    if (pass || !any_of(pending || most > MOST8 || !ok)) break;
                    if (any_of(!ok)) {
                        failed = true;
                        break;
                    }
                    // lift the maxima: of the tile's keys over the warps, then of each row by a thread
#pragma unroll
                    for (int c = 0; c < CHUNKS; c++) {
                        if (16 * c + 8 * half >= rows) break;
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            float y, z;
                            split(u[c][i / 2], y, z);
                            const int top = __reduce_max_sync(0xffffffffu, ordered(i & 1 ? z : y));
                            if (lane == 0) sm.top[g][warp & 3][16 * c + 8 * half + i] = top;
                        }
                    }
                    any_of(false);
                    bool without = false;
                    if (place < (rows + 7) / 8 * 8) {
                        int top = sm.top[g][0][place];
#pragma unroll
                        for (int q = 1; q < 4; q++) top = max(top, sm.top[g][q][place]);
                        const float m = unordered(top), was = neg_m[place];   // (m: from the last maximum on)
                        const bool set = sm.set[g][place];
                        float f = 1.f;
                        if (!(m <= INFINITY)) {   // a NaN that the row sees: it has no maximum any more
                            neg_m[place] = NAN;
                            sm.set[g][place] = 1;
                        } else if (m > (set ? BIAS8 : -INFINITY)) {
                            const float now = was + (BIAS8 - m);
                            if (set) f = ex2(now - was);
                            neg_m[place] = now;
                            sm.set[g][place] = 1;
                        } else if (!set && place < rows) {
                            without = true;
                        }
                        lift[place] = f;
                    }
                    pending = any_of(without);
                    last_product();
#pragma unroll
                    for (int c = 0; c < CHUNKS; c++) {
                        const int r0 = 16 * c + 8 * half;
                        if (r0 >= rows) break;
                        float f[8];
#pragma unroll
                        for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4 *>(f + i) = *reinterpret_cast<const float4 *>(lift + r0 + i);
#pragma unroll
                        for (int i = 0; i < 4; i++) l[c][i] = mul2(l[c][i], pair_of(f[2 * i], f[2 * i + 1]));
                        if (!any_tile) continue;
#pragma unroll 1
                        for (int part = 0; part < PP; part++) {
                            uint32_t o[8];
                            tmem_ld8(t_o + part * rp + r0, o);
                            tmem_wait_ld();
                            after_wait<8>(o);
#pragma unroll
                            for (int i = 0; i < 8; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f[i]);
                            tmem_st8(t_o + part * rp + r0, o);
                        }
                    }
                    tmem_wait_st();
                }
                if (failed) break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sm.s_free[g][buffer]));
                last_product();
                // the weights: their sum, and their parts
#pragma unroll
                for (int c = 0; c < CHUNKS; c++) {
                    const int r0 = 16 * c + 8 * half;
                    if (r0 >= rows) break;
                    uint32_t w[PP][2];
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        float d[4];
                        split(u[c][i / 2], d[0], d[1]);
                        split(u[c][i / 2 + 1], d[2], d[3]);
#pragma unroll
                        for (int e = 0; e < 4; e++) d[e] = ex2(d[e]);
                        l[c][i / 2] = fma2(pair_of(d[0], d[1]), rr, l[c][i / 2]);
                        l[c][i / 2 + 1] = fma2(pair_of(d[2], d[3]), rr, l[c][i / 2 + 1]);
                        uint32_t parts[PP];
                        parts_of<PP>(half2_of(d[0], d[1]), half2_of(d[2], d[3]), tie, parts);
#pragma unroll
                        for (int part = 0; part < PP; part++) w[part][i / 4] = parts[part];
                    }
#pragma unroll
                    for (int part = 0; part < PP; part++)
                        *reinterpret_cast<uint2 *>(p_at + ((part * rp >> 4) + c) * 2048) = make_uint2(w[part][0], w[part][1]);
                }
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sm.p_full[g]));
                done++;
                vp.advance(v_stages);
                any_tile = true;
            }
            // each row's sum over this warp's keys, while the last product runs
#pragma unroll
            for (int c = 0; c < CHUNKS; c++) {
                if (16 * c + 8 * half >= rows) break;
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; i++) split(l[c][i], x[2 * i], x[2 * i + 1]);
#pragma unroll
                for (int o = 16, n = 4; n; o >>= 1, n >>= 1)
#pragma unroll
                    for (int i = 0; i < n; i++) {
                        const bool up = lane & o;
                        const float give = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
                        x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                x[0] += __shfl_xor_sync(0xffffffffu, x[0], 2);
                x[0] += __shfl_xor_sync(0xffffffffu, x[0], 1);
                if (!(lane & 3)) sm.sum[g][warp & 3][16 * c + 8 * half + (lane >> 2)] = x[0];
            }
            if (failed) ok = false;
            if (ok) {
                ok = warp_wait(bar(sm.o_done[g]), (done - 1) & 1, dead);
            }
            if (any_of(!ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const bool direct = s.t0 == 0 && s.t1 == s.nt;
            const int slot = 2 * (g * gridDim.x + blockIdx.x) + (s.t0 > 0 ? 0 : 1);
            const int64_t orow0 = (int64_t)s.row0 * P.Hq + s.kvh * P.G;
            const bool broken = *reinterpret_cast<volatile int *>(&sm.bad[g][seg & 15]) == seg + 1;
            const bool patch = *reinterpret_cast<volatile int *>(&sm.patched[g]) == seg;
            if (place < rows) {   // the row's sum, and what its O is multiplied by
                float sum = sm.sum[g][0][place] + sm.sum[g][1][place] + sm.sum[g][2][place] + sm.sum[g][3][place];
                if (broken) sum = NAN;
                sm.factor[g][place] = sum == 0.f ? 0.f : rcp(sum);
                const float lse2 = sum == 0.f ? -INFINITY : lg2(sum) - neg_m[place];
                const int at = q_place[place];
                if (!direct) P.part_lse[slot * MAX_ROWS8 + place] = lse2;
                else if (P.lse) P.lse[orow0 + (int64_t)(at >> 16) * P.Hq + (at & 0xffff)] = lse2 * 0.6931471805599453f;
            }
            any_of(false);
#pragma unroll 1
            for (int c = 8 * half; c < rows; c += 16) {
                uint32_t x[PP][8];
#pragma unroll
                for (int part = 0; part < PP; part++) tmem_ld8(t_o + part * rp + c, x[part]);
                tmem_wait_ld();
#pragma unroll
                for (int part = 0; part < PP; part++) after_wait<8>(x[part]);
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    float a = 0.f;
#pragma unroll
                    for (int part = PP - 1; part >= 0; part--) a += __uint_as_float(x[part][i]);
                    o[i] = a * sm.factor[g][c + i];
                }
                if (patch && key < C.D) {   // NaN elements of values that some rows do not see, for those that do
#pragma unroll 1
                    for (int side = 0; side < 2; side++) {
                        const int from = side ? s.lo : s.len - s.n + 1, to = side ? min(s.len, s.lo + s.n - 1) : s.len;
#pragma unroll 1
                        for (int j = from; j < to; j++) {
                            if (side && (!P.window || j > s.len - s.n)) break;   // (the causal side has it)
                            const int tile = j / TILE, t = tile >= s.w0 ? tile - s.w0 + s.ns : tile;
                            if (t < s.t0 || t >= s.t1 || seen_by_all(P, s, j)) continue;
                            const int page = C.table[(int64_t)s.b * C.max_pages + (j >> C.page_shift)];
                            if (page < 0 || page >= C.num_pages) continue;
                            const uint8_t v = C.v[page * C.page_stride + (j & ((1 << C.page_shift) - 1)) * C.token_stride +
                                                  s.kvh * C.head_stride + key];
                            if ((v & 0x7f) != 0x7f) continue;
#pragma unroll
                            for (int i = 0; i < 8; i++)
                                if (c + i < rows && sees(P, s.len - s.n + (q_place[c + i] >> 16), j)) o[i] = NAN;
                        }
                    }
                }
                if (key < C.D) {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        if (c + i >= rows) break;
                        if (direct) {
                            const int at = q_place[c + i];
                            static_cast<E *>(P.out)[(orow0 + (int64_t)(at >> 16) * P.Hq + (at & 0xffff)) * C.D + key] = (E)o[i];
                        } else {
                            P.part_o[((int64_t)slot * MAX_ROWS8 + c + i) * P.pitch + key] = o[i];
                        }
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(sm.seg_empty[g][seg & (SEGS - 1)]));
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

// Tensor map of a cache in 8 bits: (byte, slot, head, page), boxes of `width` bytes x the slots of one page that fit a
// key tile.  Bytes past head_dim read as zero.
static bool encode8(CUtensorMap *map, const sv_kv_cache8 &c, void *ptr, int width) {
    EncodeFn f = encode_fn();
    if (!f) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_heads,
                                (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride, (cuuint64_t)c.head_stride, (cuuint64_t)c.page_stride};
    const cuuint32_t box[4] = {(cuuint32_t)width, (cuuint32_t)(c.page_size < TILE ? c.page_size : TILE), 1, 1}, one[4] = {1, 1, 1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, ptr, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             c.head_dim % 128 ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Attn8Ws {
    size_t desc, lse, o, total;
};
static Attn8Ws attn8_ws(int D) {
    Attn8Ws L;
    L.desc = HEADER;
    constexpr size_t RANGES = Attn8Args::MAX_RANGES;
    L.lse = L.desc + RANGES * sizeof(int4);
    L.o = L.lse + 2 * RANGES * MAX_ROWS8 * 4;
    L.total = L.o + 2 * RANGES * MAX_ROWS8 * (D <= 64 ? 64 : 128) * 4;
    return L;
}

constexpr int SMEM_MAX8 = 232448;

template <typename E, int CHUNKS, int WIDTH>
static sv_status launch_rows8(const Batch &A, const Cache8 &C, Attn8Args P, const sv_kv_cache8 &cache, cudaStream_t st) {
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return SV_ERR_CUDA;
    const int most_rows = (A.k_max + 1) * P.G;
    P.tile_rows = 16 * CHUNKS;
    constexpr int STAGE8 = TILE * WIDTH;
    const int other = 2 * (Parts<E>::Q + Parts<E>::P) * P.tile_rows * 128, stages = (SMEM_MAX8 - SMALL8 - other) / (2 * STAGE8);
    // A row tile costs about 4 key tiles beside its own.  96 ragged requests of 64 columns: 114, 93, 83, 79, 80 us with 1, 2, 3, 4, 6;
    // 64 of 128 columns 84, 73, 62, 57, 60; uniform batches within 1 %.
    P.overhead = 4;
    // (values wait longer than keys for their use: the odd stage is theirs)
    P.k_stages = stages / 2 < MOST_K_STAGES ? stages / 2 : MOST_K_STAGES;
    P.v_stages = stages - P.k_stages < MAX_STAGES8 ? stages - P.k_stages : MAX_STAGES8;
    const int smem = SMALL8 + other + 2 * (P.k_stages + P.v_stages) * STAGE8;
    // no more CTAs than the batch can have units
    const long long most = (long long)A.B * C.heads * (((long long)most_rows + P.tile_rows - 1) / P.tile_rows) *
                           ((((long long)C.max_pages << C.page_shift) + TILE - 1) / TILE + P.overhead);
    int ctas = nsm < MAX_CTAS ? nsm : MAX_CTAS;
    // heads that share lines keep step only if each has a whole number of CTAs: worth up to 5 % of them
    if (C.D % 128 && cache.head_stride % 128 && C.heads <= 16 && ctas % C.heads * 20 <= ctas) ctas -= ctas % C.heads;
    if (most < ctas) ctas = (int)most;
    // (one limit for every call: another thread's call may come between this and the launch)
    if (cudaFuncSetAttribute(attention8_kernel<E, CHUNKS, WIDTH>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX8) != cudaSuccess)
        return SV_ERR_CUDA;
    // (after a runtime call that brings this host thread to the device)
    CUtensorMap mk, mv;
    if (!encode8(&mk, cache, cache.k, WIDTH) || !encode8(&mv, cache, cache.v, WIDTH)) return SV_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(NTHREADS8);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, attention8_kernel<E, CHUNKS, WIDTH>, A, C, P, mk, mv) != cudaSuccess) return SV_ERR_CUDA;
    cfg.gridDim = dim3(2 * ctas, (most_rows < 8 ? most_rows : 8) + 1);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return (P.pitch == 128 ? cudaLaunchKernelEx(&cfg, join_kernel<E, 128, Cache8, Attn8Args>, A, C, P)
                           : cudaLaunchKernelEx(&cfg, join_kernel<E, 64, Cache8, Attn8Args>, A, C, P)) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

template <typename E, int WIDTH>
static sv_status launch_attention8(const Batch &A, const Cache8 &C, const Attn8Args &P, const sv_kv_cache8 &cache, cudaStream_t st) {
    const int rows = (A.k_max + 1) * P.G;
    if (rows <= 16) return launch_rows8<E, 1, WIDTH>(A, C, P, cache, st);
    if (rows <= 32 || Parts<E>::ROWS == 32) return launch_rows8<E, 2, WIDTH>(A, C, P, cache, st);
    return launch_rows8<E, Parts<E>::ROWS / 16, WIDTH>(A, C, P, cache, st);
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
    // (the 16-bit call's workspace serves both: its parts have more rows)
    const Attn8Ws L = attn8_ws(cache.head_dim);
    if (((uintptr_t)workspace & 255) || workspace_bytes < sv_attention_workspace_bytes(cache.head_dim) || workspace_bytes < L.total)
        return SV_ERR_WORKSPACE;
    char *w = static_cast<char *>(workspace);
    Attn8Args P = {};
    P.q = q;
    P.q_stride = q_stride;
    P.out = out;
    P.lse = out_lse;
    P.hdr = reinterpret_cast<int32_t *>(w);
    P.desc = reinterpret_cast<int4 *>(w + L.desc);
    P.part_lse = reinterpret_cast<float *>(w + L.lse);
    P.part_o = reinterpret_cast<float *>(w + L.o);
    P.shift = fabsf(scale) < 0x1p-60f ? 64 : 0;
    P.c = (P.shift ? scale * 0x1p64f : scale) * 1.4426950408889634f;
    P.withhold = sv::withholding();
    P.Hq = num_q_heads;
    P.G = num_q_heads / cache.num_heads;
    // (a window that holds every length is none: differences of positions stay in 32 bits)
    P.window = window < (cache.max_pages << C.page_shift) ? window : 0;
    P.sinks = sinks;
    P.pitch = cache.head_dim <= 64 ? 64 : 128;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = cache.head_dim > 64;
    if (dtype == SV_BF16)
        return wide ? launch_attention8<__nv_bfloat16, 128>(A, C, P, cache, st) : launch_attention8<__nv_bfloat16, 64>(A, C, P, cache, st);
    return wide ? launch_attention8<__half, 128>(A, C, P, cache, st) : launch_attention8<__half, 64>(A, C, P, cache, st);
}
