// sv_segments.cuh -- what the attention kernels share: the batch's work as tiles of keys cut into equal
// ranges, which tokens a row sees, and the kernel that joins the parts of rows whose keys lie in several ranges.
#pragma once

#include <cuda.h>
#include <math.h>

#include <atomic>

#include "sv_cache.cuh"
#include "sv_tc.cuh"

namespace svc {

constexpr int TILE = 128;                // tokens per key tile, rows per row tile
constexpr int MAX_CTAS = 160;

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

template <typename C, typename A>
__device__ __forceinline__ Req req_of(const Batch &batch, const C &cache, const A &P, int b) {
    const Span s = span_of(batch, cache.max_pages << cache.page_shift, b);
    Req r;
    r.row0 = s.row0;
    r.n = s.n;
    r.len = s.len;
    r.M = s.n * P.G;
    r.mt = P.tiles_of(r.M);
    r.lo = P.window ? max(0, s.len - s.n - P.window + 1) : 0;
    r.w0 = r.lo / TILE;
    r.ns = P.window ? min((min(P.sinks, s.len) + TILE - 1) / TILE, r.w0) : 0;
    r.nt = s.n ? r.ns + (s.len + TILE - 1) / TILE - r.w0 : 0;
    return r;
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
template <typename A>
__device__ __forceinline__ bool sees(const A &P, int pos, int j) {
    return j <= pos && (!P.window || j > pos - P.window || j < P.sinks);
}
// The same for tokens j .. j + 31, a bit each.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
template <typename A>
__device__ __forceinline__ uint32_t seen_mask(const A &P, int pos, int j) {
    uint32_t m = low_bits(pos + 1 - j);
    if (P.window) m &= ~low_bits(pos - P.window + 1 - j) | low_bits(P.sinks - j);
    return m;
}
template <typename A>
__device__ __forceinline__ bool seen_by_all(const A &P, const Seg &s, int j) {
    return j <= s.len - s.n && (!P.window || j > s.len - 1 - P.window || j < P.sinks);
}
template <typename A>
__device__ __forceinline__ bool seen_by_any(const A &P, const Seg &s, int j) {
    return j < s.len && (j >= s.lo || j < P.sinks);
}
// Whether every row sees all 128 tokens from base on.
template <typename A>
__device__ __forceinline__ bool whole_tile(const A &P, const Seg &s, int base) {
    return base + TILE - 1 <= s.len - s.n && (!P.window || base > s.len - 1 - P.window || base + TILE - 1 < P.sinks);
}

// A position in a ring of tiles: the stage, and the parity of its turn.
struct Place {
    uint32_t stage, parity;
    __device__ __forceinline__ void advance(uint32_t stages) {
        if (++stage == stages) stage = 0, parity ^= 1;
    }
};

// Four columns (from 4 sub on) of a joined row, and its lse.
template <typename E, typename CacheT, typename ArgsT>
__device__ __forceinline__ void store_joined(const ArgsT &P, const CacheT &C, int4 d, int rt, int sub, float4 o, float sum,
                                             float top) {
    if (sub * 4 >= C.D) return;
    const float inv = 1.f / sum;
    const int rr = P.first_row(d.w >> ArgsT::RANGE_BITS, d.z) + rt, tok = rr / P.G;
    const int64_t orow = (int64_t)(d.x + tok) * P.Hq + d.y * P.G + rr - tok * P.G;
    *reinterpret_cast<uint2 *>(static_cast<E *>(P.out) + orow * C.D + sub * 4) =
        make_uint2(Num<E>::down(o.x * inv, o.y * inv), Num<E>::down(o.z * inv, o.w * inv));
    if (P.lse && sub == 0) P.lse[orow] = (top + log2f(sum)) * 0.6931471805599453f;
}

// Joins the parts of the row tiles that several CTAs hold, in order of the CTAs, and sets the rows
// that no request uses.  Blocks (c, y): rows y, y + ny, ... of the row tile that begins in range c; the last y
// has the rows that no request uses.
// Many rows of few parts (long draft chains): a row per DP / 4 lanes.  Else a row's parts are spread over
// the block, 16 bytes of a part per thread, and the thread groups' sums are added in shared memory: one
// long request's parts (19 for 131 072 keys) then come in one round trip.
template <typename E, int DP, typename CacheT, typename ArgsT>
__global__ void __launch_bounds__(256) join_kernel(const Batch A, const CacheT C, const ArgsT P) {
    constexpr int PART_ROWS = ArgsT::PART, MAX_PARTS = ArgsT::MAX_RANGES, OWN = (MAX_PARTS + 255) / 256;   // parts of a thread
    constexpr int TPP = DP / 4, LANES = 256 / TPP;   // threads per part, parts at a time
    __shared__ float weight[MAX_PARTS];
    __shared__ float4 sums[LANES][TPP];
    __shared__ float red[2][8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ny = gridDim.y - 1;
    grid_wait();
    if ((int)blockIdx.y < ny) {
        const int4 d = P.desc[blockIdx.x];
        if (d.x < 0) return;
        const int rows = P.rows_of(d.w >> ArgsT::RANGE_BITS, d.z), first = blockIdx.x,
                  parts = (d.w & ((1 << ArgsT::RANGE_BITS) - 1)) - first + 1;
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
            float v[OWN], top = -INFINITY;
#pragma unroll
            for (int i = 0; i < OWN; i++) {
                v[i] = tid + 256 * i < parts ? lse[slot(tid + 256 * i) * PART_ROWS] : -INFINITY;
                top = i ? fmaxf(top, v[i]) : v[i];
            }
            const float *from = P.part_o + (int64_t)rt * DP + (tid % TPP) * 4;
            float4 x[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {   // the first parts' values, under way while the weights come together
                const int p = tid / TPP + i * LANES;
                x[i] = p < parts ? *reinterpret_cast<const float4 *>(from + (int64_t)slot(p) * PART_ROWS * DP)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (lane == 0) red[0][warp] = top;
            __syncthreads();
            top = red[0][0];
            for (int i = 1; i < 8; i++) top = fmaxf(top, red[0][i]);
            float f = 0.f;
#pragma unroll
            for (int i = 0; i < OWN; i++) {
                const float w = v[i] == -INFINITY ? 0.f : ex2(v[i] - top);   // (NaN where a part is)
                if (tid + 256 * i < parts) weight[tid + 256 * i] = w;
                f = i ? f + w : w;
            }
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

}  // namespace svc
