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
// The B operands are sums of 8-bit parts that lie side by side along N:
//   - a query row, times the power of two that brings its largest element into (224, 448], is q0 + q1 / 16 (+ q2 / 256) with
//     e4m3 q0 = RN(q), q1 = RN(16 (q - q0)): 4 bits each, so 2 parts hold a bf16 and 3 an fp16 without loss, for
//     elements down to 2^-14 of the largest;
//   - a weight in fp16 is a sum of its top byte, the top byte of the rest, and so on: an fp16's top byte is an e5m2
//     number.  2 (3) of them and the rest rounded to e5m2 hold 9 bits for bf16 (11, all, for fp16).  e5m2 spans
//     2^-17 to 2^15.8, and the running maximum is kept between 2^12 and 2^15.5, so what is rounded away is below 2^-29 of
//     a row's largest weight, and unbiased.  (e4m3 parts would end 2^-18 below it: 131 072 small weights
//     would lose a percent of the sum.)
// The score of a key is c ks_j qs_r S (ks: the key's scale, qs: the row's power of two), and the weight that goes to the
// product with v is p vs_j: log2 vs_j is added to the exponent, and m is the maximum of the sums.  l adds p alone.
//
// A CTA: a front warp (segments, queries in parts), a K and a V warp (tensor copies of pages into two rings; with the
// keys, 4-byte copies of both sides' scales), one that issues the matrix instructions, and two groups of 8 softmax warps,
// which take alternate key tiles, each with its own S, P, m, l and O, joined at the end of a segment.  A group's warps
// decide together, at a barrier per tile, whether a maximum lags too far; every decision that a barrier depends on is
// taken that way, so a wait that runs out in one warp ends all of them.
#include "sv_cache8.cuh"
#include "sv_launch.h"
#include "sv_segments.cuh"
#include "sv_tc.cuh"

namespace svc {

constexpr int STAGE8 = TILE * 128;       // bytes of a key tile: 128 bytes a key whatever head_dim
constexpr int NTHREADS8 = 640;           // 2 x 8 softmax warps, then one warp for each of:
constexpr int W_K = 17, W_V = 18, W_MMA = 19;   // 16 is the front warp
constexpr int MAX_STAGES8 = 7, MAX_QBUFS8 = 4;
constexpr int MAX_ROWS8 = 48;            // rows of a row tile, at most
constexpr int READERS8 = 19;             // warps that take each segment

template <typename E>
struct Parts;
template <>
struct Parts<__nv_bfloat16> {
    static constexpr int Q = 2, P = 3, ROWS = 48;   // 2 (Q + P) ROWS columns of tensor memory
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
    int4 *desc;        // as in AttnArgs
    float *part_lse;   // [2 * MAX_CTAS][PART]
    float *part_o;     // [2 * MAX_CTAS][PART][pitch]
    float c;           // scale log2(e)
    int withhold;
    int Hq, G, window, sinks;
    int k_stages, v_stages, q_bufs;
    int overhead;      // cost of a row tile beside its key tiles, in key tiles
    int tile_rows;     // rows of a row tile at most
    int pitch;         // of part_o: 64 or 128

    // Row tiles of M rows: as few as it takes, of one height, a multiple of 8.
    static constexpr int PART = MAX_ROWS8;
    __device__ __forceinline__ int tiles_of(int M) const { return (M + tile_rows - 1) / tile_rows; }
    __device__ __forceinline__ int height(int M) const {
        const int mt = tiles_of(M);
        return mt <= 1 ? M : ((M + mt - 1) / mt + 7) & ~7;
    }
    __device__ __forceinline__ int first_row(int M, int m) const { return m * height(M); }
    __device__ __forceinline__ int rows_of(int M, int m) const { return min(M - m * height(M), height(M)); }
};

// Offsets in shared memory of what stands before the rings.
struct Small8 {
    uint64_t k_full[MAX_STAGES8], k_empty[MAX_STAGES8], v_full[MAX_STAGES8], v_empty[MAX_STAGES8];
    uint64_t s_full[2], s_free[2], p_full[2], o_done[2], both[2], drained, q_full[MAX_QBUFS8], q_empty[MAX_QBUFS8];
    uint64_t seg_full[SEGS], seg_empty[SEGS];
    int dead, tmem, patched[2][4], bad[16];
    long long scan[24];
    Seg segs[SEGS];
    float scale[MAX_STAGES8][32];                 // a K stage's scales of keys (16) and of values
    __align__(16) float q_scale[MAX_QBUFS8][MAX_ROWS8];
    int q_place[MAX_QBUFS8][MAX_ROWS8];           // a row's token of the request << 16 | head of the group
    __align__(16) float neg_m[2][MAX_ROWS8];      // BIAS - m, or UNSET
    __align__(16) float lift[2][MAX_ROWS8];
    int top[2][4][MAX_ROWS8];
    float sum[2][4][MAX_ROWS8];
    float total[2][MAX_ROWS8];
    float factor[2][2][MAX_ROWS8];                // [group that reads][group whose O]
};
constexpr int SMALL8 = (sizeof(Small8) + 1023) / 1024 * 1024;

constexpr float BIAS8 = 12.f;      // log2 of the largest weight, for a maximum that does not lag
constexpr float MOST8 = 15.5f;     // and the largest that may be: 57344 is e5m2's last number
constexpr float UNSET8 = 1e30f;    // neg_m of a row that has seen nothing yet

// fp32 numbers as integers of the same order.
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

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

// Four fp16 weights (two pairs of rows) as P parts: part i of them in out[i].
template <int P>
__device__ __forceinline__ void parts_of(uint32_t a, uint32_t b, uint32_t *out) {
#pragma unroll
    for (int i = 0; i < P - 1; i++) {
        out[i] = __byte_perm(a, b, 0x7531);
        a = sub_half2(a, a & 0xff00ff00u);
        b = sub_half2(b, b & 0xff00ff00u);
    }
    out[P - 1] = __byte_perm(e5m2_of(a), e5m2_of(b), 0x5410);
}

// CHUNKS: of 8 rows that a softmax warp may have; a row tile has 16 CHUNKS rows at most.
template <typename E, int CHUNKS>
__global__ void __launch_bounds__(NTHREADS8, 1)
attention8_kernel(const Batch A, const Cache8 C, const Attn8Args P, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
    constexpr int QP = Parts<E>::Q, PP = Parts<E>::P;
    constexpr int S_COLS = QP * 16 * CHUNKS, O_COLS = PP * 16 * CHUNKS;
    static_assert(2 * (S_COLS + O_COLS) <= 512, "tensor memory");
    constexpr int NW = NTHREADS8 / 32;
    extern __shared__ __align__(1024) char smem[];
    Small8 &sm = *reinterpret_cast<Small8 *>(smem);
    // [barriers and small state][ring of K tiles][ring of V tiles][query buffers][weights of each group]
    char *const k_p = smem + SMALL8, *const v_p = k_p + P.k_stages * STAGE8, *const q_p = v_p + P.v_stages * STAGE8;
    const int q_buffer = QP * P.tile_rows * 128, p_buffer = PP * P.tile_rows * 128;
    char *const p_p = q_p + P.q_bufs * q_buffer;
    volatile int *const dead = &sm.dead;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t k_stages = P.k_stages, v_stages = P.v_stages, q_bufs = P.q_bufs;
    auto bar = [&](const uint64_t &b) { return smem_addr(&b); };

    if (tid == 0) {
        for (int i = 0; i < MAX_STAGES8; i++) {
            mbar_init(bar(sm.k_full[i]), 33);    // the copies' bytes, and each lane's scale
            mbar_init(bar(sm.k_empty[i]), 8);    // a group's warps
            mbar_init(bar(sm.v_full[i]), 1);
            mbar_init(bar(sm.v_empty[i]), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(bar(sm.s_full[i]), 1);
            mbar_init(bar(sm.s_free[i]), 8);
            mbar_init(bar(sm.p_full[i]), 8);
            mbar_init(bar(sm.o_done[i]), 1);
            mbar_init(bar(sm.both[i]), 16);
        }
        for (int i = 0; i < MAX_QBUFS8; i++) {
            mbar_init(bar(sm.q_full[i]), 1);
            mbar_init(bar(sm.q_empty[i]), 17);   // the products, and the softmax warps (for scale and place)
        }
        mbar_init(bar(sm.drained), 1);
        sm.dead = 0;
    } else if (tid >= 64 && tid < 64 + 2 * SEGS) {
        const int i = tid - 64;
        mbar_init(i < SEGS ? bar(sm.seg_full[i]) : bar(sm.seg_empty[i - SEGS]), i < SEGS ? 1 : READERS8);
    } else if (tid >= 128 && tid < 136) {
        sm.patched[(tid - 128) >> 2][tid & 3] = -1;
    } else if (tid >= 160 && tid < 176) {
        sm.bad[tid - 160] = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (warp == W_MMA) tmem_alloc(smem_addr(&sm.tmem), 512);
    grid_wait();   // the work before this on the stream may still be writing what follows

    // The batch's units, and where this CTA's range begins, as in attention_kernel.
    long long &start_pre = sm.scan[NW], &start_b = sm.scan[NW + 1];
    long long W = 0, T = 0, lo = 0, hi = 0, before = 0;   // units of one key head, of all, and this CTA's range
    int nc = 0, kvh0 = 0;
    const int cta = blockIdx.x;
    auto units_of = [&](const Req &r) { return r.nt ? (long long)(r.nt + P.overhead) * r.mt : 0ll; };
    auto range = [&]() {   // [T cta / nc, T (cta + 1) / nc), and the head that it begins in
        T = W * C.heads;
        nc = (int)min((long long)gridDim.x, T);
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
        for (int pass = A.B <= NTHREADS8; pass < 2; pass++) {   // pass 0 sums, pass 1 finds
            before = 0;
#pragma unroll 1
            for (int b0 = 0; b0 < A.B; b0 += NTHREADS8) {
                const int b = b0 + tid;
                Req r = {};
                if (b < A.B) r = req_of(A, C, P, b);
                const long long w = units_of(r);
                long long inc = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                if (b0) __syncthreads();
                if (lane == 31) sm.scan[warp] = inc;
                __syncthreads();
                long long pre = before + inc - w, all = 0;
#pragma unroll
                for (int i = 0; i < NW; i++) {
                    const long long x = sm.scan[i];
                    if (i < warp) pre += x;
                    all += x;
                }
                before += all;
                if (pass == 0) continue;
                if (b0 == 0) {
                    if (A.B <= NTHREADS8) W = all;
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
    const uint32_t tmem = *reinterpret_cast<volatile int *>(&sm.tmem);
    grid_launch_dependents();

    // Takes segment k into registers; false at the end of the list, or when a wait ran out (ok).
    bool ok = true;
    auto take = [&](int k, Seg &s, bool release_now) {
        const int slot = k & (SEGS - 1);
        ok = warp_wait(bar(sm.seg_full[slot]), k / SEGS & 1, dead);
        if (!ok) return false;
        int4 *to = reinterpret_cast<int4 *>(&s);
        const int4 *from = reinterpret_cast<const int4 *>(sm.segs + slot);
#pragma unroll
        for (int i = 0; i < 4; i++) to[i] = from[i];
        __syncwarp();
        if (release_now && lane == 0) mbar_arrive(bar(sm.seg_empty[slot]));
        return s.nt > 0;
    };
    auto drain = [&](uint64_t &barrier, bool leader) {   // the matrix instructions in flight, before tensor memory is given back
        if (leader) mma_commit(bar(barrier));
        const uint32_t t0 = now_ns32();
        while (!mbar_try(bar(barrier), 0) && now_ns32() - t0 < WAIT_NS) {}
    };
    const int steps = (C.D + 31) / 32;                    // of 32 elements of a head

    if (warp >= 16) {
        regs_down<64>();   // to the softmax warps: 4 x 104 + 64 = 5 x 96
        if (warp == W_K || warp == W_V) {
            // Keys, or values, of each segment's tiles; with the keys, both sides' scales.
            const bool is_v = warp == W_V;
            const CUtensorMap *const map = is_v ? &map_v : &map_k;
            uint64_t *const fulls = is_v ? sm.v_full : sm.k_full, *const empties = is_v ? sm.v_empty : sm.k_empty;
            const uint32_t ring = smem_addr(is_v ? v_p : k_p), stages = is_v ? v_stages : k_stages;
            Seg s;
            const int P_ = 1 << C.page_shift, box = min(P_, TILE), npg = TILE / box, tpl = 32 / npg;
            const int sub = lane & (npg - 1), lane_tile = lane / npg;
            const int per = min(1 << C.block_shift, TILE), blocks = TILE / per;   // tokens per scale, scales per tile and side
            const int blk = lane & 15, blk_tok = blk * per, blk_page = blk_tok / box;
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
                    // this lane's page of tile t (lanes below npg), or -1, and its block's
                    int id = __shfl_sync(0xffffffffu, ids, (t - t_ids) * npg + sub);
                    const int of_block = __shfl_sync(0xffffffffu, ids, (t - t_ids) * npg + (blk_page & (npg - 1)));
                    if (lane >= npg) id = -1;
                    if (id == C.num_pages) {
                        *reinterpret_cast<volatile int *>(&sm.bad[seg & 15]) = seg + 1;
                        record_error(P.hdr, SV_DEV_BAD_PAGE, s.b);
                        id = -1;
                    }
                    const int base = s.base(t);
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * box * 128;
                    const uint32_t full = bar(fulls[at.stage]);
                    __syncwarp();   // (a bad page noted by any lane, before the arrival that publishes it)
                    ok = warp_wait(bar(empties[at.stage]), at.parity, dead);
                    if (!ok) break;
                    if (P.withhold && !is_v && loads == 0) {   // (its waits then run out, as they are meant to)
                        ok = false;
                        break;
                    }
                    loads++;
                    if (lane == 0) mbar_expect(full, bytes);
                    __syncwarp();
                    if (id >= 0)
                        tma_load_4d(ring + at.stage * STAGE8 + sub * box * 128, map, full, 0, base & (P_ - 1) & ~(box - 1), s.kvh, id);
                    if (!is_v) {
                        if (blk < blocks && of_block >= 0 && of_block < C.num_pages && base + blk_tok < s.len) {
                            const int slot = (base + blk_tok) & (P_ - 1);
                            const float *from = lane < 16 ? C.k_scale : C.v_scale;
                            copy4(smem_addr(&sm.scale[at.stage][lane]),
                                  from + of_block * C.s_page + (slot >> C.block_shift) * C.s_block + s.kvh * C.s_head);
                        }
                        copies_arrive(full);
                    }
                    __syncwarp();
                    at.advance(stages);
                }
            }
            copies_commit();
            copies_wait<0>();
            if (!ok) {   // let the copies in flight land before the CTA may end
                const uint32_t t0 = now_ns32();
                for (uint32_t i = loads > stages ? loads - stages : 0; i < loads; i++)
                    while (!mbar_try(bar(fulls[i % stages]), i / stages & 1) && now_ns32() - t0 < WAIT_NS) {}
            }
        } else if (warp == W_MMA) {
            // Matrix instructions: each tile's scores as soon as its group has the last ones in registers, and its P V as
            // soon as the weights are there, whichever comes first.  The whole warp runs this; one lane issues.
            const bool leader = elect();
            int sseg = 0, oseg = 0;                    // segments opened
            int st = 0, snt = 0, srp = 0, ot = 0, ont = 0, orp = 0;   // tile, tiles and columns of a part of the current ones
            auto open = [&](int &k, int &t, int &nt, int &rp, bool release) {
                Seg s;
                t = nt = 0;
                if (!take(k++, s, release)) return;
                nt = s.t1 - s.t0;
                rp = (P.rows_of(s.M, s.m) + 15) & ~15;
            };
            open(sseg, st, snt, srp, false);
            if (ok) open(oseg, ot, ont, orp, true);
            Place ks{0, 0}, vs{0, 0}, qs{0, 0};
            uint32_t gs = 0, go = 0, nf = 3, np = 0;   // groups whose turn it is; parities of each one's free S and next P
            uint32_t polls = 0, idle_since = 0;
#pragma unroll 1
            while (ok && ont) {
                // all that may be waited for is asked at once; every lane has to have seen it
                uint32_t there = 0;
                if (snt) {
                    there = mbar_test(bar(sm.s_free[gs]), nf >> gs & 1) && mbar_test(bar(sm.k_full[ks.stage]), ks.parity) &&
                            (st || mbar_test(bar(sm.q_full[qs.stage]), qs.parity));
                }
                there |= (uint32_t)(mbar_test(bar(sm.p_full[go]), np >> go & 1) && mbar_test(bar(sm.v_full[vs.stage]), vs.parity)) << 1;
                there = __reduce_and_sync(0xffffffffu, there);
                if (!there) {
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
                if (there & 1) {
                    if (leader) {
                        const uint32_t idesc = mma8_idesc(false, QP * srp, false);
                        const uint64_t qd = smem_desc(smem_addr(q_p) + qs.stage * q_buffer, 16),
                                       kd = smem_desc(smem_addr(k_p) + ks.stage * STAGE8, 16);
                        for (int k = 0; k < steps; k++)
                            mma8_ss(tmem + gs * S_COLS, kd + (uint64_t)(k * 2), qd + (uint64_t)(k * 2), idesc, k > 0);
                        mma_commit(bar(sm.s_full[gs]));
                        if (st == snt - 1) mma_commit(bar(sm.q_empty[qs.stage]));
                    }
                    __syncwarp();
                    nf ^= 1u << gs;
                    gs ^= 1;
                    ks.advance(k_stages);
                    if (++st == snt) {
                        qs.advance(q_bufs);
                        open(sseg, st, snt, srp, false);
                    }
                }
                if ((there & 2) && ok) {
                    if (leader) {
                        const uint32_t idesc = mma8_idesc(true, PP * orp, true);
                        const uint64_t vd = smem_desc(smem_addr(v_p) + vs.stage * STAGE8, STAGE8),
                                       pd = smem_desc_plain(smem_addr(p_p) + go * p_buffer, 128, 2048);
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            mma8_ss(tmem + 2 * S_COLS + go * O_COLS, vd + (uint64_t)(k * (4096 >> 4)), pd + (uint64_t)(k * (512 >> 4)), idesc,
                                    ot >= 2 || k > 0);
                        mma_commit(bar(sm.o_done[go]));
                    }
                    __syncwarp();
                    np ^= 1u << go;
                    go ^= 1;
                    vs.advance(v_stages);
                    if (++ot == ont) open(oseg, ot, ont, orp, true);
                }
            }
            if (!ok) drain(sm.drained, leader);
            __syncwarp();
        } else {
            // Front: the segments of this CTA's range, in order, and their queries in parts.  A lane looks at one of 16
            // requests at a time.
            uint32_t pushed = 0, done = 0;   // segments handed out, and with their queries there
            Req r = {};
            long long first = 0, sum = 0;    // this lane's request's first unit, all 16's units
            bool fresh = true;
            auto look = [&](int b) {         // at requests b .. b + 15: first and sum from this head's start
                r.nt = r.mt = 0;
                if (lane < SMALL_BATCH && b + lane < A.B) r = req_of(A, C, P, b + lane);
                const long long w = units_of(r);
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
            Place at{0, 1};                  // query buffer to fill
            if (lane == 0) P.desc[cta] = make_int4(-1, 0, 0, 0);
            __syncwarp();
            auto push = [&](uint32_t k, const Seg &s) {   // (any subset of lanes, each its own k)
                const uint32_t slot = k & (SEGS - 1);
                const bool free = mbar_wait(bar(sm.seg_empty[slot]), (k / SEGS & 1) ^ 1, dead);
                if (free) {
                    sm.segs[slot] = s;
                    mbar_arrive(bar(sm.seg_full[slot]));
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
                    const int per = r.nt + P.overhead;
                    const long long mine = kvh * W + pre + first + (long long)m * per;
                    Seg s;
                    s.row0 = r.row0, s.n = r.n, s.len = r.len, s.M = r.M, s.lo = r.lo, s.w0 = r.w0, s.ns = r.ns, s.nt = r.nt;
                    s.b = b_base + lane;
                    s.kvh = kvh;
                    s.m = m;
                    s.solo = 0;
                    // (the CTA of the row tile's last unit has its last key tile)
                    s.t0 = max((int)min(max(lo - mine, 0ll), (long long)per) - P.overhead, 0);
                    s.t1 = (int)min(max(hi - mine, 0ll), (long long)per) - P.overhead;
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
                if (!ok || done == pushed) break;   // (nothing is left)
                ok = warp_wait(bar(sm.q_empty[at.stage]), at.parity, dead);
                if (!ok) break;
                const Seg &s = sm.segs[done & (SEGS - 1)];   // (not written again before its queries are there)
                const int row0 = P.first_row(s.M, s.m), rows = P.rows_of(s.M, s.m), rp = (rows + 15) & ~15;
                const int lpr = C.D > 64 ? 16 : 8, rpw = 32 / lpr;   // lanes of a row, rows per warp step
                const int ch = lane & (lpr - 1), team = lane / lpr;
                const E *q = static_cast<const E *>(P.q) + s.row0 * P.q_stride + (int64_t)s.kvh * P.G * C.D + ch * 8;
                char *const to = q_p + at.stage * q_buffer;
                constexpr int U = 2;
#pragma unroll 1
                for (int r0 = 0; r0 < rp; r0 += U * rpw) {
                    uint4 raw[U];
                    int place[U];
#pragma unroll
                    for (int u = 0; u < U; u++) {
                        const int row = r0 + u * rpw + team, rr = row0 + row, tok = rr / P.G, head = rr - tok * P.G;
                        raw[u] = make_uint4(0u, 0u, 0u, 0u);
                        place[u] = tok << 16 | head;
                        if (row < rows && ch * 8 < C.D)
                            raw[u] = *reinterpret_cast<const uint4 *>(q + tok * P.q_stride + (int64_t)head * C.D);
                    }
#pragma unroll
                    for (int u = 0; u < U; u++) {
                        const int row = r0 + u * rpw + team;
                        float x[8], top = 0.f;
                        unpack8<E>(raw[u], x);
#pragma unroll
                        for (int e = 0; e < 8; e++) top = fabsf(x[e]) < INFINITY ? fmaxf(top, fabsf(x[e])) : INFINITY;
                        // (an infinity stays: fmaxf(inf, x), and what is not finite sets it again)
#pragma unroll
                        for (int e = 0; e < 8; e++) top = fabsf(x[e]) < INFINITY ? top : INFINITY;
                        for (int o = lpr / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        // the power of two s with top in (224 s, 448 s]
                        const uint32_t b = __float_as_uint(top);
                        const int k = (int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
                        const float s_ = __uint_as_float((uint32_t)(min(max(k, -118), 118) + 127) << 23), inv = 1.f / s_;
                        if (row < rp) {
                            if (ch == 0) {
                                sm.q_scale[at.stage][row] = top < INFINITY ? s_ : NAN;
                                sm.q_place[at.stage][row] = place[u];
                            }
#pragma unroll
                            for (int e = 0; e < 8; e++) x[e] *= inv;
#pragma unroll
                            for (int part = 0; part < QP; part++) {
                                uint32_t two[4];
#pragma unroll
                                for (int e = 0; e < 4; e++) {
                                    two[e] = pack_e4m3(x[2 * e], x[2 * e + 1]);
                                    const float2 y = unpack_e4m3(two[e]);
                                    x[2 * e] = (x[2 * e] - y.x) * 16.f;
                                    x[2 * e + 1] = (x[2 * e + 1] - y.y) * 16.f;
                                }
                                const int n = part * rp + row;
                                *reinterpret_cast<uint2 *>(to + n * 128 + (((ch >> 1) ^ (n & 7)) << 4) + (ch & 1) * 8) =
                                    make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
                            }
                        }
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sm.q_full[at.stage]));
                done++;
                at.advance(q_bufs);
            }
        }
    } else {
        regs_up<104>();
        // Softmax and epilogue: group g, two threads per key of a tile, which have its rows by turns of 8.
        const int g = warp >> 3, half = warp >> 2 & 1, key = (warp & 3) * 32 + lane, place = tid & 255;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // this warp's 32 lanes of tensor memory
        const uint32_t t_s = tmem + g * S_COLS + lanes, t_o = tmem + 2 * S_COLS + lanes;
        const int block = key >> min(C.block_shift, 7);               // of this thread's key in a tile
        char *const p_at = p_p + g * p_buffer + (key >> 3) * 128 + (key & 7) * 16 + half * 8;
        auto any_of = [&](bool x) { return barrier_any(1 + g, 256, x); };
        float *const neg_m = sm.neg_m[g], *const lift = sm.lift[g];
        uint32_t mine_done = 0, turn = 0, tiles = 0, joint = 0;   // own tiles; all tiles; barriers of both groups
        Place qs{0, 0};
#pragma unroll 1
        for (int seg = 0;; seg++) {
            ok = warp_wait(bar(sm.seg_full[seg & (SEGS - 1)]), seg / SEGS & 1, dead);
            if (any_of(!ok)) break;
            const Seg &s = sm.segs[seg & (SEGS - 1)];   // (its fields are read where they are needed)
            if (s.nt == 0) break;
            const int nt = s.t1 - s.t0, mine = (g ^ turn) & 1;        // this group's first key tile
            const uint32_t tile0 = tiles;
            turn += nt;
            tiles += nt;
            const int rows = P.rows_of(s.M, s.m), rp = (rows + 15) & ~15;
            const float *const q_scale = sm.q_scale[qs.stage];
            const int *const q_place = sm.q_place[qs.stage];
            auto release = [&]() {   // the segment's and its queries' buffers
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(sm.q_empty[qs.stage]));
                    mbar_arrive(bar(sm.seg_empty[seg & (SEGS - 1)]));
                }
                qs.advance(q_bufs);
            };
            if (mine >= nt) {   // the other group's alone
                release();
                continue;
            }
            const bool pair = nt > 1;   // both groups hold a part of every row
            float l[CHUNKS][8];
#pragma unroll
            for (int c = 0; c < CHUNKS; c++)
#pragma unroll
                for (int i = 0; i < 8; i++) l[c][i] = 0.f;
            bool any_tile = false;
            if (place < MAX_ROWS8) neg_m[place] = UNSET8;
            ok = warp_wait(bar(sm.q_full[qs.stage]), qs.parity, dead);   // (for the queries' scales and places)
            any_of(false);
#pragma unroll 1
            for (int t = mine; t < nt; t += 2) {
                const int base = s.base(s.t0 + t), j = base + key;
                const bool whole = whole_tile(P, s, base);
                const uint32_t tile = tile0 + t, k_round = tile / k_stages, k_stage = tile - k_round * k_stages,
                               v_round = tile / v_stages, v_stage = tile - v_round * v_stages;
                if (!whole && !seen_by_all(P, s, j)) {   // a value that must not reach the product as it is
                    ok = ok && mbar_wait(bar(sm.v_full[v_stage]), v_round & 1, dead);
                    uint4 *const row = reinterpret_cast<uint4 *>(v_p + v_stage * STAGE8 + key * 128);
                    // (each half 64 of its bytes, a different bank per lane)
                    if (!seen_by_any(P, s, j)) {         // (a slot never written may hold NaN, and 0 * NaN is NaN)
#pragma unroll
                        for (int i = 0; i < 4; i++) row[(4 * half + i) ^ (key & 7)] = make_uint4(0u, 0u, 0u, 0u);
                    } else {                             // (the epilogue gives its NaN to the rows that see it)
                        bool took = false;
#pragma unroll 1
                        for (int i = 4 * half; i < 4 * half + 4; i++) {
                            uint4 w = row[i ^ (key & 7)];
                            uint32_t *p = &w.x;
                            bool hit = false;
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const uint32_t nan = __vcmpeq4(p[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                p[e] &= ~nan;
                                hit |= nan != 0;
                            }
                            if (hit) row[i ^ (key & 7)] = w, took = true;
                        }
                        if (took) *reinterpret_cast<volatile int *>(&sm.patched[g][seg & 3]) = seg;
                    }
                }
                __syncwarp();
                ok = warp_wait(bar(sm.s_full[g]), mine_done & 1, dead) && ok;
                ok = warp_wait(bar(sm.k_full[k_stage]), k_round & 1, dead) && ok;   // (complete: for the scales)
                tc_fence_after();
                const float ck = P.c * clean_scale(sm.scale[k_stage][block]);
                const float lvs = lg2(clean_scale(sm.scale[k_stage][16 + block])), rvs = ex2(-lvs);
                // the scores in powers of two, with the value's scale.  Rows lie in order of their tokens, so those that see
                // this key are neighbours: tokens from the key's own on, up to the last whose window has it.
                int from = 0, to = 0x7fffffff;
                if (!whole) {
                    const int first = j - (s.len - s.n), row0 = P.first_row(s.M, s.m);
                    from = min(max(first, 0), s.n) * P.G - row0;
                    if (P.window && j >= P.sinks) to = min(max(first + P.window, 0), s.n) * P.G - row0;
                }
                float u[CHUNKS][8];
                float most = -INFINITY;
#pragma unroll
                for (int c = 0; c < CHUNKS; c++) {
                    const int r0 = 16 * c + 8 * half;
                    if (r0 >= rows) break;
                    uint32_t x[QP][8];
#pragma unroll
                    for (int part = 0; part < QP; part++) tmem_ld8(t_s + part * rp + r0, x[part]);
                    tmem_wait_ld();
#pragma unroll
                    for (int part = 0; part < QP; part++) after_wait<8>(x[part]);
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 qsc = *reinterpret_cast<const float4 *>(q_scale + r0 + i);
#pragma unroll
                        for (int h = 0; h < 4; h += 2) {
                            auto pair_at = [&](int part) {
                                return pair_of(__uint_as_float(x[part][i + h]), __uint_as_float(x[part][i + h + 1]));
                            };
                            uint64_t v = pair_at(QP - 1);
#pragma unroll
                            for (int part = QP - 2; part >= 0; part--) v = fma2(v, pair_of(0.0625f, 0.0625f), pair_at(part));
                            const uint64_t f = mul2(pair_of(ck, ck), h ? pair_of(qsc.z, qsc.w) : pair_of(qsc.x, qsc.y));
                            split(fma2(v, f, pair_of(lvs, lvs)), u[c][i + h], u[c][i + h + 1]);
                        }
                    }
                    if (!whole) {   // (rows from `from` up to `to` see this key)
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            if (r0 + i < from || r0 + i >= to) u[c][i] = -INFINITY;
                    }
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 nm = *reinterpret_cast<const float4 *>(neg_m + r0 + i);
                        float d[4];
                        split(add2(pair_of(u[c][i], u[c][i + 1]), pair_of(nm.x, nm.y)), d[0], d[1]);
                        split(add2(pair_of(u[c][i + 2], u[c][i + 3]), pair_of(nm.z, nm.w)), d[2], d[3]);
                        most = max3(most, max3(d[0], d[1], d[2]), d[3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(sm.s_free[g]));
                    mbar_arrive(bar(sm.k_empty[k_stage]));
                }
                bool waited = !any_tile;
                auto last_product = [&]() {   // the group's last product is through with its weights, its V tile and O
                    if (waited) return;
                    ok = warp_wait(bar(sm.o_done[g]), (mine_done - 1) & 1, dead) && ok;
                    tc_fence_after();
                    if ((warp & 7) == 0 && lane == 0) mbar_arrive(bar(sm.v_empty[(tile - 2) % v_stages]));
                    waited = true;
                };
                if (any_of(most > MOST8 || !ok)) {
                    if (any_of(!ok)) {
                        ok = false;
                        break;
                    }
                    // lift the maxima: of the tile's keys over the warps, then of each row by a thread
#pragma unroll
                    for (int c = 0; c < CHUNKS; c++) {
                        if (16 * c + 8 * half >= rows) break;
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const int top = __reduce_max_sync(0xffffffffu, ordered(u[c][i]));
                            if (lane == 0) sm.top[g][warp & 3][16 * c + 8 * half + i] = top;
                        }
                    }
                    any_of(false);
                    if (place < (rows + 7) / 8 * 8) {
                        int top = sm.top[g][0][place];
#pragma unroll
                        for (int w = 1; w < 4; w++) top = max(top, sm.top[g][w][place]);
                        const float m = unordered(top), was = neg_m[place];
                        float f = 1.f;
                        if (!(m <= INFINITY)) {   // a NaN that the row sees: it has no maximum any more
                            neg_m[place] = NAN;
                        } else if (m + was > BIAS8) {
                            neg_m[place] = BIAS8 - m;
                            if (was != UNSET8) f = ex2((BIAS8 - was) - m);
                        }
                        lift[place] = f;
                    }
                    any_of(false);
                    last_product();
#pragma unroll
                    for (int c = 0; c < CHUNKS; c++) {
                        const int r0 = 16 * c + 8 * half;
                        if (r0 >= rows) break;
                        float f[8];
#pragma unroll
                        for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4 *>(f + i) = *reinterpret_cast<const float4 *>(lift + r0 + i);
#pragma unroll
                        for (int i = 0; i < 8; i++) l[c][i] *= f[i];
                        if (!any_tile) continue;
#pragma unroll
                        for (int part = 0; part < PP; part++) {
                            uint32_t o[8];
                            tmem_ld8(t_o + g * O_COLS + part * rp + r0, o);
                            tmem_wait_ld();
                            after_wait<8>(o);
#pragma unroll
                            for (int i = 0; i < 8; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f[i]);
                            tmem_st8(t_o + g * O_COLS + part * rp + r0, o);
                        }
                    }
                    tmem_wait_st();
                }
                last_product();
                // the weights: their sum, and their parts
#pragma unroll
                for (int c = 0; c < CHUNKS; c++) {
                    const int r0 = 16 * c + 8 * half;
                    if (r0 >= rows) break;
                    uint32_t w[PP][2];
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 nm = *reinterpret_cast<const float4 *>(neg_m + r0 + i);
                        float d[4];
                        split(add2(pair_of(u[c][i], u[c][i + 1]), pair_of(nm.x, nm.y)), d[0], d[1]);
                        split(add2(pair_of(u[c][i + 2], u[c][i + 3]), pair_of(nm.z, nm.w)), d[2], d[3]);
#pragma unroll
                        for (int e = 0; e < 4; e++) d[e] = ex2(d[e]);
#pragma unroll
                        for (int e = 0; e < 4; e += 2)
                            split(fma2(pair_of(d[e], d[e + 1]), pair_of(rvs, rvs), pair_of(l[c][i + e], l[c][i + e + 1])), l[c][i + e],
                                  l[c][i + e + 1]);
                        uint32_t parts[PP];
                        parts_of<PP>(half2_of(d[0], d[1]), half2_of(d[2], d[3]), parts);
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
                mine_done++;
                any_tile = true;
            }
            // each row's sum over this warp's keys, while the last product runs
#pragma unroll
            for (int c = 0; c < CHUNKS; c++) {
                if (16 * c + 8 * half >= rows) break;
                float *x = l[c];
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
            if (ok) ok = warp_wait(bar(sm.o_done[g]), (mine_done - 1) & 1, dead);
            if (ok && (warp & 7) == 0 && lane == 0)
                mbar_arrive(bar(sm.v_empty[(tile0 + nt - 1 - ((nt - 1 - mine) & 1)) % v_stages]));
            if (any_of(!ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (place < rows)
                sm.total[g][place] = sm.sum[g][0][place] + sm.sum[g][1][place] + sm.sum[g][2][place] + sm.sum[g][3][place];
            if (pair) {   // the other group's maxima, sums and O
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sm.both[0]));
                ok = warp_wait(bar(sm.both[0]), joint & 1, dead);
                tc_fence_after();
            }
            if (any_of(!ok)) {
                ok = false;
                break;
            }
            const bool direct = s.t0 == 0 && s.t1 == s.nt;
            const int slot = 2 * cta + (s.t0 > 0 ? 0 : 1);
            const int64_t orow0 = (int64_t)s.row0 * P.Hq + s.kvh * P.G;
            const bool broken = *reinterpret_cast<volatile int *>(&sm.bad[seg & 15]) == seg + 1;
            auto patched_by = [&](int i) { return *reinterpret_cast<volatile int *>(&sm.patched[i][seg & 3]) == seg; };
            const bool patch = patched_by(g) || (pair && patched_by(g ^ 1));
            if (place < rows) {   // the row's maximum and sum, and the factors of the (up to) two sums O
                const float m0 = BIAS8 - neg_m[place], m1 = pair ? BIAS8 - sm.neg_m[g ^ 1][place] : -UNSET8;
                const float top = fmaxf(m0, m1), f0 = ex2(m0 - top), f1 = pair ? ex2(m1 - top) : 0.f;
                float sum = sm.total[g][place] * f0 + (pair ? sm.total[g ^ 1][place] * f1 : 0.f);
                if (broken) sum = NAN;
                const float inv = sum == 0.f ? 0.f : rcp(sum);
                sm.factor[g][g][place] = f0 * inv;
                sm.factor[g][g ^ 1][place] = f1 * inv;
                if (!pair || g == 0) {
                    const float lse2 = sum == 0.f ? -INFINITY : top + lg2(sum) - BIAS8;
                    const int at = q_place[place];
                    if (!direct) P.part_lse[slot * MAX_ROWS8 + place] = lse2;
                    else if (P.lse) P.lse[orow0 + (int64_t)(at >> 16) * P.Hq + (at & 0xffff)] = lse2 * 0.6931471805599453f;
                }
            }
            any_of(false);
#pragma unroll 1
            for (int c = pair ? 16 * g + 8 * half : 8 * half; c < rows; c += pair ? 32 : 16) {
                uint32_t x[PP][8], y[PP][8];
#pragma unroll
                for (int part = 0; part < PP; part++) {
                    tmem_ld8(t_o + g * O_COLS + part * rp + c, x[part]);
                    if (pair) tmem_ld8(t_o + (g ^ 1) * O_COLS + part * rp + c, y[part]);
                }
                tmem_wait_ld();
#pragma unroll
                for (int part = 0; part < PP; part++) after_wait<8>(x[part]), after_wait<8>(y[part]);
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    float a = 0.f, b = 0.f;
#pragma unroll
                    for (int part = PP - 1; part >= 0; part--) a += __uint_as_float(x[part][i]);
                    o[i] = a * sm.factor[g][g][c + i];
                    if (pair) {
#pragma unroll
                        for (int part = PP - 1; part >= 0; part--) b += __uint_as_float(y[part][i]);
                        o[i] = fmaf(b, sm.factor[g][g ^ 1][c + i], o[i]);
                    }
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
            if (pair) {   // neither group's next product may overwrite an O that the other still reads
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sm.both[1]));
                ok = warp_wait(bar(sm.both[1]), joint++ & 1, dead);
            }
            release();
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

// Tensor map of a cache in 8 bits: (byte, slot, head, page), boxes of 128 bytes x the slots of one page that fit a
// key tile.  Bytes past head_dim read as zero.
static bool encode8(CUtensorMap *map, const sv_kv_cache8 &c, void *ptr) {
    EncodeFn f = encode_fn();
    if (!f) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_heads,
                                (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride, (cuuint64_t)c.head_stride, (cuuint64_t)c.page_stride};
    const cuuint32_t box[4] = {128, (cuuint32_t)(c.page_size < TILE ? c.page_size : TILE), 1, 1}, one[4] = {1, 1, 1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, ptr, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B,
             c.head_dim % 128 ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Attn8Ws {
    size_t desc, lse, o, total;
};
static Attn8Ws attn8_ws(int D) {
    Attn8Ws L;
    L.desc = HEADER;
    L.lse = L.desc + MAX_CTAS * sizeof(int4);
    L.o = L.lse + (size_t)2 * MAX_CTAS * MAX_ROWS8 * 4;
    L.total = L.o + (size_t)2 * MAX_CTAS * MAX_ROWS8 * (D <= 64 ? 64 : 128) * 4;
    return L;
}

constexpr int SMEM_MAX8 = 232448;

template <typename E, int CHUNKS>
static sv_status launch_rows8(const Batch &A, const Cache8 &C, Attn8Args P, const sv_kv_cache8 &cache, cudaStream_t st) {
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return SV_ERR_CUDA;
    const int most_rows = (A.k_max + 1) * P.G;
    P.tile_rows = 16 * CHUNKS;
    P.q_bufs = P.tile_rows <= 16 ? MAX_QBUFS8 : 2;
    const int other = P.q_bufs * Parts<E>::Q * P.tile_rows * 128 + 2 * Parts<E>::P * P.tile_rows * 128;
    const int stages = (SMEM_MAX8 - SMALL8 - other) / STAGE8;
    P.overhead = 2;
    P.k_stages = stages / 2 < MAX_STAGES8 ? stages / 2 : MAX_STAGES8;
    P.v_stages = stages - P.k_stages < MAX_STAGES8 ? stages - P.k_stages : MAX_STAGES8;
    const int smem = SMALL8 + other + (P.k_stages + P.v_stages) * STAGE8;
    // no more CTAs than the batch can have units
    const long long most = (long long)A.B * C.heads * (((long long)most_rows + P.tile_rows - 1) / P.tile_rows) *
                           ((((long long)C.max_pages << C.page_shift) + TILE - 1) / TILE + P.overhead);
    int ctas = nsm < MAX_CTAS ? nsm : MAX_CTAS;
    // heads that share lines keep step only if each has a whole number of CTAs: worth up to 5 % of them
    if (C.D % 128 && cache.head_stride % 128 && C.heads <= 16 && ctas % C.heads * 20 <= ctas) ctas -= ctas % C.heads;
    if (most < ctas) ctas = (int)most;
    // (one limit for every call: another thread's call may come between this and the launch)
    if (cudaFuncSetAttribute(attention8_kernel<E, CHUNKS>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX8) != cudaSuccess)
        return SV_ERR_CUDA;
    // (after a runtime call that brings this host thread to the device)
    CUtensorMap mk, mv;
    if (!encode8(&mk, cache, cache.k) || !encode8(&mv, cache, cache.v)) return SV_ERR_CUDA;
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
    if (cudaLaunchKernelEx(&cfg, attention8_kernel<E, CHUNKS>, A, C, P, mk, mv) != cudaSuccess) return SV_ERR_CUDA;
    cfg.gridDim = dim3(ctas, (most_rows < 8 ? most_rows : 8) + 1);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return (P.pitch == 128 ? cudaLaunchKernelEx(&cfg, join_kernel<E, 128, Cache8, Attn8Args>, A, C, P)
                           : cudaLaunchKernelEx(&cfg, join_kernel<E, 64, Cache8, Attn8Args>, A, C, P)) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

template <typename E>
static sv_status launch_attention8(const Batch &A, const Cache8 &C, const Attn8Args &P, const sv_kv_cache8 &cache, cudaStream_t st) {
    const int rows = (A.k_max + 1) * P.G;
    if (rows <= 16) return launch_rows8<E, 1>(A, C, P, cache, st);
    if (rows <= 32 || Parts<E>::ROWS == 32) return launch_rows8<E, 2>(A, C, P, cache, st);
    return launch_rows8<E, Parts<E>::ROWS / 16>(A, C, P, cache, st);
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
    P.c = scale * 1.4426950408889634f;
    P.withhold = sv::withholding();
    P.Hq = num_q_heads;
    P.G = num_q_heads / cache.num_heads;
    // (a window that holds every length is none: differences of positions stay in 32 bits)
    P.window = window < (cache.max_pages << C.page_shift) ? window : 0;
    P.sinks = sinks;
    P.pitch = cache.head_dim <= 64 ? 64 : 128;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == SV_BF16 ? launch_attention8<__nv_bfloat16>(A, C, P, cache, st)
                            : launch_attention8<__half>(A, C, P, cache, st);
}
