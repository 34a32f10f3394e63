// Attention with a sliding window and sinks over a (paged) cache
// (dbs_window_attention, sm_103a): softmax over the entries a token sees, with the
// running maximum and sum held in fp32.
#include "cache_dev.h"
#include "places.h"
#include "tc_dev.h"

using namespace dbs::ops;

namespace {

struct Win {
    dbs_window_args a;
    float scale_log2;          // scale * log2(e): probabilities are powers of two
    int window, sinks;         // (at most 2^31 - 1024)
    int group;                 // query heads of a kv head
    bool wide_out;             // heads of out start on 16-byte boundaries
    Waits waits;
};

// What sequence b holds, with every length clamped to its range.
struct Seq {
    int kv, first;             // entries; the position of token 0 (may be < 0)
    int tokens;                // of this call
};

__device__ __forceinline__ Seq sequence(const Win &A, int64_t b)
{
    const dbs_window_args &a = A.a;
    Seq s;
    const int64_t room = a.max_pages * a.page_size;
    const int64_t kv = a.kv_lens[b], t = a.q_lens ? a.q_lens[b] : a.tokens;
    s.kv = (int)(kv < 0 ? 0 : kv > room ? room : kv);
    s.tokens = (int)(t < 0 ? 0 : t > a.tokens ? a.tokens : t);
    s.first = s.kv - s.tokens;
    return s;
}

// The first entry of the window of a token at position p (p >= 0).
__device__ __forceinline__ int window_start(const Win &A, int p) { return p >= A.window ? p - A.window + 1 : 0; }

// One query row by one warp, entry by entry (every step-th of those it sees, from the
// part-th on), touching only what the row sees.  OUT_ONLY: it ends once all of the output is NaN, so that l may
// lack entries then.
template <class T, bool OUT_ONLY = false>
__device__ __forceinline__ void row_by_warp(const Win &A, const Seq &s, int64_t b, int t, int h, int part, int step, float &m, float &l,
                                            float (&o)[8])
{
    const dbs_window_args &a = A.a;
    const int lane = threadIdx.x & 31;
    float qr[8];
    begin_row<T>(a, b, t, h, qr, m, l, o);
    const int p = s.first + t;
    if (t >= s.tokens || p < 0) return;
    const int lo = window_start(A, p), sinks = A.sinks < lo ? A.sinks : lo, n = sinks + p + 1 - lo;
    for (int i = part; i < n; i += step) {
        take_entry<T>(a, place_of(a, b, i < sinks ? i : lo + i - sinks), h / A.group, A.scale_log2, qr, m, l, o);
        if (OUT_ONLY) {
            bool rest = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) rest |= lane + 32 * e < a.head_dim && o[e] == o[e];
            if (!__any_sync(~0u, rest)) break;
        }
    }
}

constexpr int ROW_NT = 128;

// Any head size and alignment: one block per query row, its warps take every fourth
// entry, a lane every 32nd value.  Bound by the latency of each entry's sum: one token, window 1024, 176 us; a prompt
// of 8192 tokens, window 4096, 150 ms.
template <class T>
__global__ void __launch_bounds__(ROW_NT) k_window_rows(Win A)
{
    const dbs_window_args &a = A.a;
    constexpr int W = ROW_NT / 32;
    __shared__ float s_m[W], s_l[W], s_o[W][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t r = blockIdx.x, heads = (uint32_t)a.q_heads, h = r % heads, bt = r / heads;
    const int64_t b = bt / (uint32_t)a.tokens;
    const int t = (int)(bt % (uint32_t)a.tokens);
    float o[8], m, l;
    row_by_warp<T>(A, sequence(A, b), b, t, (int)h, warp, W, m, l, o);
#pragma unroll
    for (int e = 0; e < 8; ++e) s_o[warp][lane + 32 * e] = o[e];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    if (warp == 0) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
        for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w]);
        for (int w = 0; w < W; ++w) {
            const float f = weight_of(s_m[w], s_l[w], top);
            sum += f * s_l[w];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] += f * s_o[w][lane + 32 * e];
        }
        store_row<T>(a, b, t, (int)h, top, sum, o);
    }
}

// ---- the entries of a unit ----
//
// A unit is one kv head of one sequence and some tokens' rows of it.  Its entries lie
// in one line without a gap: the sinks, then those from the first token's window on.  Where
// copies take boxes of `grain` entries both parts begin on a box, so that a few entries that no
// row sees are among them; where the parts meet the line is simply the cache's.
struct Range {
    int sinks, lo, n;          // entries of the first part, first entry of the second, length of the line
    int hi;                    // behind the last entry that a row sees
    int first, last;           // positions of the unit's first and last token
    __device__ __forceinline__ int real(int v) const { return v < sinks ? v : v - sinks + lo; }
};

__device__ __forceinline__ Range range_of(const Win &A, const Seq &s, int t0, int t1, int grain)
{
    Range r;
    t1 = t1 < s.tokens ? t1 : s.tokens - 1;
    r.last = s.first + t1;
    r.first = s.first + t0 < 0 ? 0 : s.first + t0;
    r.hi = r.last + 1;
    r.sinks = r.lo = r.n = 0;
    if (t0 > t1 || r.last < 0) {
        r.hi = 0;
        return r;
    }
    r.lo = window_start(A, r.first) & -grain;                              // (a power of two)
    if (A.sinks < r.lo) r.sinks = (A.sinks + grain - 1) & -grain;
    if (A.sinks >= r.lo || r.sinks >= r.lo) r.sinks = r.lo = 0;
    r.n = r.sinks + r.hi - r.lo;
    return r;
}

// bar_wait, whose first look is all there is most of the time.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int *stop, uint32_t limit)
{
    return __builtin_expect(bar_test(bar, parity), 1) || bar_wait(bar, parity, stop, limit);
}

// Whether all rows see the entries v .. v + size - 1 of the line, all of which it has.
__device__ __forceinline__ bool seen_by_all(const Win &A, const Range &r, int v, int size)
{
    if (v + size <= r.sinks) return v + size <= A.sinks;
    if (v < r.sinks) return false;
    const int j = r.real(v);
    return j + size - 1 <= r.first && (j > r.last - A.window || j + size <= A.sinks);
}
// Whether some row sees entry j, and whether the token at position p does (p >= -1).
__device__ __forceinline__ bool seen_by_any(const Win &A, const Range &r, int j)
{
    return j < r.hi && (j < A.sinks || j > r.first - A.window);
}
__device__ __forceinline__ bool sees(const Win &A, int p, int j) { return j <= p && (j > p - A.window || j < A.sinks); }

// Row `r` of a kv head's rows: r = token * G + head within the group.
struct Row {
    int t, h, p;               // p: its position, -1 if it sees nothing
    bool inside;               // a row of the call
};

__device__ __forceinline__ Row row_of(const Win &A, const Seq &s, int hk, int64_t R)
{
    const uint32_t G = (uint32_t)A.group, t = (uint32_t)R / G;
    Row r;
    r.t = (int)t;
    r.h = hk * (int)G + (int)((uint32_t)R - t * G);
    r.inside = R < A.a.tokens * G;
    r.p = r.inside && r.t < s.tokens && s.first + r.t >= 0 ? s.first + r.t : -1;
    return r;
}

// The matrix products give every row every entry of a tile, with probability 0 where it
// is not seen, and 0 * NaN is NaN.  What no row of a unit sees is replaced by 0 on its way
// through shared memory; a row whose result is not finite, and of whose unit V has such a value at an entry that
// others see and it does not, is made anew by a warp from what it sees alone.  (Those are the rows near such an
// entry: what they all see costs them nothing more.)

// Whether there is such a value for the row at position p (p >= 0), by a warp; heads in pieces of 16 bytes.
template <class T> __device__ __forceinline__ bool spoiled(const Win &A, const Range &r, int64_t b, int hk, int p)
{
    const dbs_window_args &a = A.a;
    const int lane = threadIdx.x & 31, chunks = a.head_dim / 8, begins = window_start(A, r.first), mine = window_start(A, p);
    // entries lo .. mine - 1, which the row's window has passed, and p + 1 .. hi - 1, which come after it
    const int lo = begins < A.sinks ? A.sinks : begins, past = mine > lo ? mine - lo : 0, n = past + r.hi - 1 - p;
    constexpr uint32_t TOP = __is_same(T, __half) ? 0x7c00u : 0x7f80u;     // the exponent of infinity and NaN
    bool bad = false;
    for (int i = lane; i < n * chunks; i += 32) {
        const int e = i / chunks;
        const Place at = place_of(a, b, e < past ? lo + e : p + 1 + e - past);
        const uint4 v = *((const uint4 *)((const T *)a.v + at.page * a.v_page + at.in * a.v_entry + hk * a.v_head) + (i - e * chunks));
        for (uint32_t w : {v.x, v.y, v.z, v.w}) bad |= (w & TOP) == TOP || (w >> 16 & TOP) == TOP;
    }
    return __any_sync(~0u, bad);
}

// ---- few rows: every warp streams its own entries ----

// Fetches a map before its first copy asks for it.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) { asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory"); }

template <int DP> struct Few {
    static constexpr int STAGES = DP == 64 ? 6 : 3;
    static constexpr int SUB = FEW_STEP * 128, HALF = DP / 64 * SUB;       // 64 columns of a stage's K; all of it
    static constexpr int RING = STAGES * 2 * HALF;
    static constexpr int SMEM = FEW_W * RING + 1024;
    static_assert((FEW_ROWS + FEW_ROWS / FEW_W) * DP * 4 <= RING, "room for a warp's sums, and behind them for its joined rows");
};

// 16 query rows against the line of their entries, which the blocks of a cluster share in
// equal parts.  The four warps of a block take turns of 16 entries, each with its own ring of K
// and V stages (in the 128-byte swizzle: 64 columns a row), running maximum, sum and output, so
// no block-wide wait runs in the loop; they are joined in the end, first in the block, then in
// the cluster through shared memory.  A maximum is replaced only when it grew by more than 2^8, so the output is
// hardly ever rescaled (probabilities stay below 2^8, exact in proportion).
//
// BOXES: K and V come by tiled copies (TMA) of boxes of 16 entries, or of 8 where pages split
// into eights only; else by 16-byte asynchronous copies.  Bound by HBM where many tokens'
// windows are read (64 sequences of one token, 32/8 heads of 128, window 4096: 170 us, 93% of the memory's rate), by latency for
// one (window 1024: 7.5 us on the device, 10.3 as a call).
template <class T, int DP, bool BOXES>
__global__ void __launch_bounds__(FEW_NT) k_window_few(Win A, int groups, int split, const __grid_constant__ Maps maps)
{
    using F = Few<DP>;
    const dbs_window_args &a = A.a;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bars[FEW_W][F::STAGES];
    __shared__ float s_m[FEW_W][FEW_ROWS], s_l[FEW_W][FEW_ROWS];
    __shared__ float j_m[FEW_ROWS], j_l[FEW_ROWS];                         // of the block's rows, for the cluster
    __shared__ int stop;
    constexpr int KK = DP / 16, NN = DP / 8, ST = F::STAGES, CH = DP / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q4 = lane & 3;
    unsigned char *const ring = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    unsigned char *const mine = ring + warp * F::RING;
    const uint32_t base = smem_addr(mine), full = smem_addr(bars[warp]);
    // a row's joined sums, in the ring of the warp that joins it, behind that warp's own
    auto joined = [&](int r) { return (float *)(ring + r % FEW_W * F::RING) + (FEW_ROWS + r / FEW_W) * DP; };

    const uint32_t rank = blockIdx.x % (uint32_t)split, unit = blockIdx.x / (uint32_t)split;
    const uint32_t group = unit % (uint32_t)groups, bh = unit / (uint32_t)groups;
    const int hk = (int)(bh % (uint32_t)a.kv_heads);
    const int64_t b = bh / (uint32_t)a.kv_heads, R0 = (int64_t)group * FEW_ROWS;
    if (threadIdx.x == 0) stop = 0;
    if (BOXES && threadIdx.x == 0) {
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
    }
    if (BOXES && lane == 0) {
        for (int i = 0; i < ST; ++i) bar_init(full + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const Seq s = sequence(A, b);
    const Row ra = row_of(A, s, hk, R0 + g), rb = row_of(A, s, hk, R0 + g + 8);
    const int box = BOXES ? maps.box : 1;
    const Range range = range_of(A, s, (int)((uint32_t)R0 / (uint32_t)A.group), (int)((uint32_t)(R0 + FEW_ROWS - 1) / (uint32_t)A.group), box);
    const int turns = (range.n + FEW_KEYS - 1) / FEW_KEYS;
    const int v0 = (int)((int64_t)turns * rank / split) * FEW_KEYS, v1 = (int)((int64_t)turns * (rank + 1) / split) * FEW_KEYS;
    const int end = v1 < range.n ? v1 : range.n;
    const int steps = end > v0 + warp * FEW_STEP ? (end - v0 - warp * FEW_STEP + FEW_KEYS - 1) / FEW_KEYS : 0;
    auto line_at = [&](int i) { return v0 + i * FEW_KEYS + warp * FEW_STEP; };
    __syncthreads();

    // Places of the next copies: lane l has those of box l % 2 of step `ahead` + l / 2 (BOXES), or
    // finds entry l of the step at hand.
    Place near{0, 0};
    int ahead = -16;
    auto fetch = [&](int i) {
        const uint32_t st = base + i % ST * (2 * F::HALF);
        if constexpr (BOXES) {
            if (i >= steps) return;
            if (i >= ahead + 16) {
                ahead = i;
                const int v = line_at(i + (lane >> 1)) + (lane & 1) * 8;
                if (i + (lane >> 1) < steps && v < end) near = place_of(a, b, range.real(v));
            }
            const int v = line_at(i), from = 2 * (i - ahead);
            const int p0 = __shfl_sync(~0u, (int)near.page, from), e0 = __shfl_sync(~0u, (int)near.in, from);
            const int p1 = __shfl_sync(~0u, (int)near.page, from + 1), e1 = __shfl_sync(~0u, (int)near.in, from + 1);
            const int boxes = box == 16 || v + 8 >= end ? 1 : 2;
            if (elected()) {
                const uint32_t bar = full + 8 * (i % ST);
                bar_expect(bar, (uint32_t)(boxes * box * 2 * DP * 2) + vain_bytes(A.waits));
#pragma unroll
                for (int c = 0; c < DP / 64; ++c) {
                    box_load(st + c * F::SUB, &maps.k, 64 * c, hk, e0, p0, bar);
                    box_load(st + F::HALF + c * F::SUB, &maps.v, 64 * c, hk, e0, p0, bar);
                    if (boxes == 2) {
                        box_load(st + c * F::SUB + 1024, &maps.k, 64 * c, hk, e1, p1, bar);
                        box_load(st + F::HALF + c * F::SUB + 1024, &maps.v, 64 * c, hk, e1, p1, bar);
                    }
                }
            }
            __syncwarp();
        } else {
            if (i < steps) {
                // lane l < 16 finds entry l, all lanes copy
                const int v = line_at(i) + (lane & 15);
                const bool in = v < end;
                const Place at = place_of(a, b, range.real(in ? v : end - 1));
                const int64_t ok = at.page * a.k_page + at.in * a.k_entry, ov = at.page * a.v_page + at.in * a.v_entry;
                const unsigned ins = __ballot_sync(~0u, in);
                const T *k = (const T *)a.k + hk * a.k_head, *w = (const T *)a.v + hk * a.v_head;
                const int chunks = a.head_dim / 8;
#pragma unroll
                for (int c0 = 0; c0 < FEW_STEP * CH; c0 += 32) {
                    const int row = (c0 + lane) / CH, c = (c0 + lane) % CH;
                    const int64_t rk = __shfl_sync(~0u, ok, row), rv = __shfl_sync(~0u, ov, row);
                    const bool take = (ins >> row & 1u) && c < chunks;
                    const uint32_t to = st + (c >> 3) * F::SUB + row * 128 + (((c & 7) ^ (row & 7)) << 4);
                    cp16(to, take ? (const void *)(k + rk + c * 8) : (const void *)a.k, take);
                    cp16(to + F::HALF, take ? (const void *)(w + rv + c * 8) : (const void *)a.v, take);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    for (int i = 0; i < ST - 1; ++i) fetch(i);

    // query rows g and g + 8 as matrix fragments
    uint32_t qf[KK][4];
    {
        const T *qa = (const T *)a.q + b * a.q_batch + ra.t * a.q_token + ra.h * a.q_head;
        const T *qb = (const T *)a.q + b * a.q_batch + rb.t * a.q_token + rb.h * a.q_head;
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            const int c = 16 * k + 2 * q4;
            qf[k][0] = ra.inside && c < a.head_dim ? *(const uint32_t *)(qa + c) : 0u;
            qf[k][1] = rb.inside && c < a.head_dim ? *(const uint32_t *)(qb + c) : 0u;
            qf[k][2] = ra.inside && c + 8 < a.head_dim ? *(const uint32_t *)(qa + c + 8) : 0u;
            qf[k][3] = rb.inside && c + 8 < a.head_dim ? *(const uint32_t *)(qb + c + 8) : 0u;
        }
    }
    float o[NN][4], ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
#pragma unroll
    for (int i = 0; i < NN; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

    bool ok = true;
    int i = 0;
    for (; i < steps; ++i) {
        fetch(i + ST - 1);
        if constexpr (BOXES) {
            ok = __all_sync(~0u, bar_wait(full + 8 * (i % ST), i / ST & 1, &stop, A.waits.limit));
            if (!ok) break;
        } else {
            asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
            __syncwarp();
        }
        const uint32_t st = base + i % ST * (2 * F::HALF);
        float sc[2][4] = {};
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            // matrices: entries 0-7 and 8-15, halves of 16 columns
            uint32_t r[4];
            const int row = (lane & 7) + ((lane >> 4) << 3), c = 2 * k + ((lane >> 3) & 1);
            ldsm4(r, st + (c >> 3) * F::SUB + row * 128 + (((c & 7) ^ (row & 7)) << 4));
            mma16816<T>(sc[0], qf[k], r[0], r[1]);
            mma16816<T>(sc[1], qf[k], r[2], r[3]);
        }
        const int v = line_at(i);
        const bool whole = v + FEW_STEP <= end && seen_by_all(A, range, v, FEW_STEP);
        float ta = -INFINITY, tb = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sc[h][e] *= A.scale_log2;
                sc[h][e + 2] *= A.scale_log2;
                if (!whole) {
                    const int at = v + 8 * h + 2 * q4 + e, j = range.real(at);
                    if (at >= end || !sees(A, ra.p, j)) sc[h][e] = -INFINITY;
                    if (at >= end || !sees(A, rb.p, j)) sc[h][e + 2] = -INFINITY;
                }
                ta = fmaxf(ta, sc[h][e]);
                tb = fmaxf(tb, sc[h][e + 2]);
            }
        if (BOXES && !whole) {
            // (what the copies brought that no row sees)
            unsigned clear = __ballot_sync(~0u, lane < FEW_STEP && (v + lane >= end || !seen_by_any(A, range, range.real(v + lane))));
            for (; clear; clear &= clear - 1) {
                const uint32_t row = st + F::HALF + (__ffs(clear) - 1) * 128;
                if (lane < DP / 8)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(row + (lane >> 3) * F::SUB + ((lane & 7) << 4)), "r"(0) : "memory");
            }
            async_fence();
            __syncwarp();
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            ta = fmaxf(ta, __shfl_xor_sync(~0u, ta, d));
            tb = fmaxf(tb, __shfl_xor_sync(~0u, tb, d));
        }
        const bool ga = ta > ma + 8.f || (ma == -INFINITY && ta > ma), gb = tb > mb + 8.f || (mb == -INFINITY && tb > mb);
        if (__any_sync(~0u, ga || gb)) {
            const float fa = ga ? (ma == -INFINITY ? 0.f : exp2f(ma - ta)) : 1.f;
            const float fb = gb ? (mb == -INFINITY ? 0.f : exp2f(mb - tb)) : 1.f;
            if (ga) ma = ta;
            if (gb) mb = tb;
            la *= fa;
            lb *= fb;
#pragma unroll
            for (int k = 0; k < NN; ++k) {
                o[k][0] *= fa;
                o[k][1] *= fa;
                o[k][2] *= fb;
                o[k][3] *= fb;
            }
        }
        const float sa = ma == -INFINITY ? 0.f : ma, sb = mb == -INFINITY ? 0.f : mb;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sc[h][e] = exp2f(sc[h][e] - sa);
                sc[h][e + 2] = exp2f(sc[h][e + 2] - sb);
                la += sc[h][e];
                lb += sc[h][e + 2];
            }
        // probabilities rounded once to the caches' type, the type of V in the matrix instruction (the
        // sums take them as they are)
        const uint32_t pf[4] = {pack2<T>(sc[0][0], sc[0][1]), pack2<T>(sc[0][2], sc[0][3]), pack2<T>(sc[1][0], sc[1][1]),
                                pack2<T>(sc[1][2], sc[1][3])};
#pragma unroll
        for (int k = 0; k < NN; k += 2) {
            // matrices: entries 0-7 and 8-15 of two groups of 8 columns
            uint32_t r[4];
            const int row = (lane & 7) + (((lane >> 3) & 1) << 3), c = k + (lane >> 4);
            ldsm4t(r, st + F::HALF + (c >> 3) * F::SUB + row * 128 + (((c & 7) ^ (row & 7)) << 4));
            mma16816<T>(o[k], pf, r[0], r[1]);
            mma16816<T>(o[k + 1], pf, r[2], r[3]);
        }
        __syncwarp();
    }
    if constexpr (BOXES) {
        // after a wait ran out: copies under way end before their memory is used again
        for (const int behind = i + ST < steps ? i + ST : steps; i < behind; ++i) {
            int last = 0;
            bar_wait(full + 8 * (i % ST), i / ST & 1, &last, A.waits.limit);
        }
    } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        la += __shfl_xor_sync(~0u, la, d);
        lb += __shfl_xor_sync(~0u, lb, d);
    }
    __syncwarp();
    // the warp's output into its own ring, rows of DP floats
    float *so = (float *)mine;
#pragma unroll
    for (int k = 0; k < NN; ++k) {
        *(float2 *)(so + g * DP + 8 * k + 2 * q4) = make_float2(o[k][0], o[k][1]);
        *(float2 *)(so + (g + 8) * DP + 8 * k + 2 * q4) = make_float2(o[k][2], o[k][3]);
    }
    if (q4 == 0) {
        s_m[warp][g] = ma;
        s_l[warp][g] = ok ? la : nanf("");
        s_m[warp][g + 8] = mb;
        s_l[warp][g + 8] = ok ? lb : nanf("");
    }
    __syncthreads();
    for (int r = warp; r < FEW_ROWS; r += FEW_W) {
        float top = -INFINITY, sum = 0.f, oo[DP / 32] = {};
#pragma unroll
        for (int w = 0; w < FEW_W; ++w) top = fmaxf(top, s_m[w][r]);
#pragma unroll
        for (int w = 0; w < FEW_W; ++w) {
            const float f = weight_of(s_m[w][r], s_l[w][r], top);
            const float *po = (const float *)(ring + w * F::RING) + r * DP;
            sum += f * s_l[w][r];
#pragma unroll
            for (int e = 0; e < DP / 32; ++e) oo[e] += f * po[lane + 32 * e];
        }
#pragma unroll
        for (int e = 0; e < DP / 32; ++e) joined(r)[lane + 32 * e] = oo[e];
        if (lane == 0) {
            j_m[r] = top;
            j_l[r] = sum;
        }
    }
    if (split > 1) cluster_sync();
    else __syncthreads();
    // 32 columns of a row for each of the cluster's warps in turn
    const int64_t left = a.tokens * A.group - R0;
    const int rows = (int)(left < FEW_ROWS ? left : FEW_ROWS);
    for (int i = (int)rank * FEW_W + warp; i < rows * (DP / 32); i += split * FEW_W) {
        const int r = i / (DP / 32), e0 = i % (DP / 32), col = lane + 32 * e0;
        const Row row = row_of(A, s, hk, R0 + r);
        const bool in = lane < split;
        const float m = in ? remote(j_m + r, lane) : -INFINITY;
        float l = in ? remote(j_l + r, lane) : 0.f;
        float v[FEW_SPLIT], out = 0.f, top = m;
#pragma unroll
        for (int k = 0; k < FEW_SPLIT; ++k) v[k] = k < split ? remote(joined(r) + col, k) : 0.f;
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        const float f = weight_of(m, l, top);
        l = weighed(f, l);
#pragma unroll
        for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
#pragma unroll
        for (int k = 0; k < FEW_SPLIT; ++k) {
            const float fk = __shfl_sync(~0u, f, k);
            out += fk * v[k];
        }
        if (row.p < 0) l = out = 0.f;
        float lo = l;                                                      // the output's divisor
        if (l == l && __any_sync(~0u, col < a.head_dim && !isfinite(out)) && spoiled<T>(A, range, b, hk, row.p)) {
            float ol[8], m1;
            row_by_warp<T, true>(A, s, b, row.t, row.h, 0, 1, m1, lo, ol);
#pragma unroll
            for (int e = 0; e < 8; ++e) out = e == e0 ? ol[e] : out;
        }
        if (col < a.head_dim) ((T *)a.out + b * a.o_batch + row.t * a.o_token + row.h * a.o_head)[col] = from_f32<T>(lo == 0.f ? 0.f : out / lo);
        if (a.lse && e0 == 0 && lane == 0) store_lse(a, b, row.t, row.h, top, l);
    }
    // (no block ends while another one reads its shared memory)
    if (split > 1) cluster_sync();
    if (threadIdx.x == 0 && stop) ran_out = 1;
}

// ---- many rows: tcgen05 ----
//
// A unit is TILES tiles of rows of one kv head, each of as many tokens as fill 128 rows
// with their heads; its entries come in tiles of KEYS, once for all its row tiles.  S = Q K^T and
// O += P V have both accumulators in tensor memory (a row per lane), Q, K and V lie in
// shared memory in the 128-byte swizzle (V as it lies, its entries as the contraction's dimension), and
// P, rounded to the caches' type, goes to tensor memory too, so that the second product reads only V from
// shared memory.  It has columns of its own: the next tile's scores are made as soon as this one's have been read, and
// wait for no product (with P over S and tiles of 128, or of 64 with two buffers: 463 and 376 us for the prompt
// below, here 328).  That leaves room for tiles of 80 at head_dim 128.  Warps have roles: four for each row tile do
// the softmax, a thread a row; one fetches Q and K, one V, one for each row tile issues its products (one for
// both: 671), one clears what no row of the unit sees in V.
//
// A row tile skips the tiles that none of its rows sees.  Blocks walk over the units, long ones
// first; of few units `split` blocks take a part each, and k_window_join joins their outputs.
//
// A prompt of 8192 tokens, window 4096, 32/8 heads of 128: 328 us, 66% of the tensor cores' rate, of whose cycles 56%
// are busy.  A step of a pair of row tiles takes 2100 cycles of a softmax thread for 80 entries, most of them
// latencies of its own chain (reading 200, maximum 400, powers of two 800, waits 400), with two such warps a
// scheduler.  Without its arithmetic 265 us are left: reading scores, storing P, and the products, whose Q comes anew from
// shared memory for each tile.  Two threads a row, which halve the chain, have to exchange maxima: 371 us; powers taken
// beside the maximum, with the one so far, and again where it grew: 330; waits that sleep: 330.  8 sequences of 8 tokens,
// 32/4 heads, window 2047 and 64 sinks: 18.5 us in two launches, six tiles a block.
//
// Every wait on a barrier has a limit; a block whose wait runs out stops, leaves NaN in
// the rows of all units that it had not finished, and says so.

template <int DP, int TILES> struct Many {
    static constexpr int KEYS = DP == 64 ? 96 : DP == 128 ? 80 : 64;      // entries of a tile
    static constexpr int STAGES = DP == 256 ? 2 : 4;       // of K, and of V
    static constexpr int SUBQ = 128 * 128, SUBK = KEYS * 128;             // 64 columns of a tile, in bytes
    static constexpr int Q = DP / 64 * SUBQ, KV = DP / 64 * SUBK;
    // first warps of the roles: fetch Q and K, fetch V, clear, issue (a warp for each row tile)
    static constexpr int HELP = 4 * TILES, CLEAR = HELP + 2, ISSUE = HELP + 3, NT = 32 * (TILES == 2 ? 16 : 8);
    // registers of a thread at launch (TILES = 2), and once the helping warps have left some to the softmax's
    static constexpr int REGS = 128, FEW = 80, MANY = 2 * REGS - FEW;
    // columns of tensor memory: scores, P (two to a column) and outputs of each row tile
    static constexpr int S_COL = 0, P_COL = TILES * KEYS, O_COL = (P_COL + TILES * KEYS / 2 + 63) / 64 * 64;
    static constexpr int SMEM = TILES * Q + STAGES * 2 * KV + 1024;
    static_assert(O_COL + TILES * DP <= 512, "tensor memory");
    static_assert(SMEM <= 227 * 1024 && KEYS % 16 == 0, "shared memory");
};

struct ManyMaps {
    Maps kv;
    CUtensorMap q;             // [batch, tokens, heads, head_dim], boxes of 64 columns of a row tile
};

// How the rows are cut: tokens of a row tile (its rows: tokens * G <= 128), units of a kv head and of all.
struct Cut {
    int tokens, groups, units, split;
    float *scratch;            // of split > 1
};

struct Unit {
    Seq s;
    Range r;
    int64_t b;
    int hk, t0;                // kv head, first token
    int begin, end;            // tiles of the line that this block takes
};

template <int KEYS, int TILES>
__device__ __forceinline__ Unit unit_of(const Win &A, const Cut &C, int u, int rank, int box)
{
    Unit U;
    const uint32_t heads = (uint32_t)A.a.kv_heads, per = (uint32_t)A.a.batch * heads;
    // (the last tokens first: their lines are the longest)
    const uint32_t g = (uint32_t)u / per, bh = (uint32_t)u - g * per;
    U.b = bh / heads;
    U.hk = (int)(bh - (uint32_t)U.b * heads);
    U.t0 = (C.groups - 1 - (int)g) * TILES * C.tokens;
    U.s = sequence(A, U.b);
    U.r = range_of(A, U.s, U.t0, U.t0 + TILES * C.tokens - 1, box);
    const int n = (U.r.n + KEYS - 1) / KEYS;
    U.begin = 0;
    U.end = n;
    if (C.split > 1) {                                                     // (n < 2^26, split at most 16)
        U.begin = n * rank / C.split;
        U.end = n * (rank + 1) / C.split;
    }
    return U;
}

// Positions of a row tile's tokens that see anything; none: last < 0.
struct Span {
    int first, last;
};
__device__ __forceinline__ Span span_of(const Unit &U, const Cut &C, int r)
{
    const int ta = U.t0 + r * C.tokens, tb = ta + C.tokens < U.s.tokens ? ta + C.tokens - 1 : U.s.tokens - 1;
    Span p{U.s.first + ta, U.s.first + tb};
    if (p.first < 0) p.first = 0;
    if (ta > tb || p.last < 0) p.last = -1;
    return p;
}
// Which tiles of the line a row tile's tokens reach, those before `sinks` and from `from` to `to`,
// and which all of them see whole, those before `all_sinks` and from `all_from` to `all_to`.
struct Reach {
    int sinks, from, to, all_sinks, all_from, all_to;
    __device__ __forceinline__ bool some(int i) const { return i < sinks || (i >= from && i <= to); }
    __device__ __forceinline__ bool all(int i) const { return i < all_sinks || (i >= all_from && i <= all_to); }
};
template <int KEYS> __device__ __forceinline__ Reach reach_of(const Win &A, const Range &r, const Span &p)
{
    if (p.last < 0) return {0, 1, 0, 0, 1, 0};
    const int shift = r.sinks - r.lo;                                      // from an entry behind the sinks to its place in the line
    const int begins = window_start(A, p.first) + shift, whole = window_start(A, p.last) + shift;
    const int sinks = r.sinks ? r.sinks : A.sinks < p.last + 1 ? A.sinks : p.last + 1;
    const int all = r.sinks || A.sinks < p.first + 1 ? A.sinks : p.first + 1;
    return {(sinks + KEYS - 1) / KEYS, (begins > 0 ? begins : 0) / KEYS, (p.last + shift) / KEYS,
            all / KEYS, (whole + KEYS - 1) / KEYS, (p.first + shift + 1) / KEYS - 1};
}
// Tiles with entries that no row of the unit sees: rounded to boxes between the sinks and the window,
// and behind the line.
struct Idle {
    int from, to, last;
    __device__ __forceinline__ bool any(int i) const { return (i >= from && i <= to) || i == last; }
};
template <int KEYS> __device__ __forceinline__ Idle idle_of(const Win &A, const Range &r)
{
    const int end = r.sinks + window_start(A, r.first) - r.lo;
    return {A.sinks < end ? A.sinks / KEYS : 1, A.sinks < end ? (end - 1) / KEYS : 0, r.n % KEYS ? r.n / KEYS : -1};
}

__device__ __forceinline__ float max_of(float a, float b, float c)
{
    float v;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(v) : "f"(a), "f"(b), "f"(c));
    return v;
}
// 16 columns of tensor memory: with more, a tile's scores would not stay in registers beside them.
__device__ __forceinline__ void ld16(uint32_t (&r)[16], uint32_t a)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\ntcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]) : "r"(a) : "memory");
}
__device__ __forceinline__ void st16(uint32_t a, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
__device__ __forceinline__ void st8(uint32_t a, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
// The lowest n bits, for any n.
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }
// A part's place in scratch: the rows' outputs, maxima and sums.
template <int DP, int TILES> __host__ __device__ constexpr int64_t part_floats() { return TILES * 128 * (int64_t)(DP + 2); }
template <int DP, int TILES> __device__ __forceinline__ float *part_of(const Cut &C, int u, int rank)
{
    return C.scratch + ((int64_t)u * C.split + rank) * part_floats<DP, TILES>();
}

template <class T, int DP, int TILES>
__global__ void __launch_bounds__(Many<DP, TILES>::NT, 1) k_window_many(Win A, Cut C, const __grid_constant__ ManyMaps maps)
{
    using M = Many<DP, TILES>;
    constexpr int KEYS = M::KEYS, ST = M::STAGES;
    const dbs_window_args &a = A.a;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bars[5 * ST + 6 * TILES + 1];
    __shared__ uint32_t tmem_at;
    __shared__ int stop;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t sq = base, sk = base + TILES * M::Q, sv = sk + ST * M::KV;
    const uint32_t k_full = smem_addr(bars), k_empty = k_full + 8 * ST, v_full = k_empty + 8 * ST, v_empty = v_full + 8 * ST, v_fixed = v_empty + 8 * ST;
    const uint32_t q_full = v_fixed + 8 * ST, q_empty = q_full + 8 * TILES, s_full = q_empty + 8 * TILES, s_free = s_full + 8 * TILES;
    const uint32_t p_full = s_free + 8 * TILES, o_done = p_full + 8 * TILES, last_bar = o_done + 8 * TILES;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");       // (a join waits for this grid's end)
    if (tid == 32) {
        prefetch_map(&maps.q);
        prefetch_map(&maps.kv.k);
        prefetch_map(&maps.kv.v);
    }
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            bar_init(k_full + 8 * i, 1);
            bar_init(k_empty + 8 * i, TILES);
            bar_init(v_full + 8 * i, 1);
            bar_init(v_empty + 8 * i, TILES + 1);
            bar_init(v_fixed + 8 * i, 1);
        }
        for (int i = 0; i < TILES; ++i) {
            bar_init(q_full + 8 * i, 1);
            bar_init(q_empty + 8 * i, 1);
            bar_init(s_full + 8 * i, 1);
            bar_init(s_free + 8 * i, 4);
            bar_init(p_full + 8 * i, 4);
            bar_init(o_done + 8 * i, 1);
        }
        bar_init(last_bar, TILES);
        stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == M::ISSUE) tc_alloc(smem_addr(&tmem_at));
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tmem_at;
    const int rank = C.split > 1 ? (int)(blockIdx.x % (uint32_t)C.split) : 0;
    const int u0 = (int)(blockIdx.x / (uint32_t)C.split), step = (int)(gridDim.x / (uint32_t)C.split), box = maps.kv.box;
    // Rounds of a unit for each block, every second backwards: units get shorter, and the block that
    // had the longest of one round has the shortest of the next.
    auto unit_at = [&](int k) { return k * step + (k & 1 ? step - 1 - u0 : u0); };
    const uint32_t limit = A.waits.limit;

    if (warp < M::HELP) {
        // ---- softmax: a thread has a row ----
        more_registers<TILES == 2 ? M::MANY : 0>();
        const int r = warp >> 2, row = (warp & 3) * 32 + lane, tile_row = r * 128 + row;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
        const uint32_t s_at = tmem + lanes + M::S_COL + r * KEYS, p_at = tmem + lanes + M::P_COL + r * KEYS / 2, o_at = tmem + lanes + M::O_COL + r * DP;
        const int dt = row / A.group, dh = row - dt * A.group;             // its token in the row tile, its head
        const uint64_t scale2 = two(A.scale_log2, A.scale_log2);
        int count = 0;                                                     // tiles done
        bool ok = true;
        for (int k = 0, u; (u = unit_at(k)) < C.units; ++k) {
            const Unit U = unit_of<KEYS, TILES>(A, C, u, rank, box);
            const Reach reach = reach_of<KEYS>(A, U.r, span_of(U, C, r));
            const int t = U.t0 + r * C.tokens + dt, h = U.hk * A.group + dh;
            const bool inside = dt < C.tokens && t < a.tokens;
            const int p = inside && t < U.s.tokens && U.s.first + t >= 0 ? U.s.first + t : -1;
            const bool busy = __any_sync(~0u, inside);
            float m = -INFINITY;
            uint64_t l2[2] = {0, 0};
            bool some = false;
            for (int i = U.begin; ok && i < U.end; ++i) {
                if (!reach.some(i)) continue;
                ok = __all_sync(~0u, wait_for(s_full + 8 * r, count & 1, &stop, limit));
                if (!ok) break;
                tc_after();
                // the scores have been read: the next tile's may come
                auto read = [&] {
                    tc_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(s_free + 8 * r);
                };
                // the product before this one is done: O is at rest, and P's place is free (every phase of
                // o_done is waited for, while the next cannot end)
                bool settled = !some;
                auto settle = [&] {
                    if (!settled) ok = __all_sync(~0u, wait_for(o_done + 8 * r, (count - 1) & 1, &stop, limit));
                    settled = true;
                    tc_after();
                };
                if (!busy) {
                    read();
                    settle();
                } else {
                    constexpr int C = KEYS / 32, REST = KEYS % 32;         // whole chunks of 32 columns, and 16 more
                    static_assert(REST == 0 || REST == 16, "a half chunk");
                    uint32_t x[C][32], z[16];
#pragma unroll
                    for (int c = 0; c < C; ++c) tc_ld_begin(x[c], s_at + 32 * c);
                    if (REST) ld16(z, s_at + 32 * C);
#pragma unroll
                    for (int c = 0; c < C; ++c) tc_ld_end(x[c]);
                    read();
                    auto at = [&](int e) -> uint32_t & { return e < 32 * C ? x[e / 32][e % 32] : z[e % 32]; };
                    if (!reach.all(i)) {
                        // columns that the row sees: up to `to`, and from behind `from` on or before `sinks`
                        const int v0 = i * KEYS, to = p - (v0 - U.r.sinks + U.r.lo), from = to - A.window, sinks = A.sinks - v0;
#pragma unroll
                        for (int c = 0; c < KEYS; c += 32) {
                            const uint32_t see = below(to + 1 - c) & (~below(from + 1 - c) | below(sinks - c));
#pragma unroll
                            for (int e = c; e < c + 32 && e < KEYS; ++e) at(e) = see >> (e - c) & 1u ? at(e) : 0xff800000u;
                        }
                    }
                    float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < KEYS; e += 2) t4[e / 2 & 3] = max_of(t4[e / 2 & 3], __uint_as_float(at(e)), __uint_as_float(at(e + 1)));
                    const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * A.scale_log2;      // (scale > 0 here)
                    // replace the maximum only when it grew by more than 2^8
                    const bool grew = top > m + 8.f || (m == -INFINITY && top > m);
                    if (__any_sync(~0u, grew)) {
                        const float f = grew ? (m == -INFINITY ? 0.f : exp2f(m - top)) : 1.f;
                        if (grew) m = top;
#pragma unroll
                        for (int e = 0; e < 2; ++e) l2[e] = fma_two(l2[e], two(f, f), 0);
                        if (some) {
                            settle();
                            if (!ok) break;
#pragma unroll 1
                            for (int c = 0; c < DP; c += 16) {
                                uint32_t o[16];
                                ld16(o, o_at + c);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                st16(o_at + c, o);
                            }
                        }
                    }
                    settle();
                    if (!ok) break;
                    const float shift = m == -INFINITY ? 0.f : -m;
                    const uint64_t shift2 = two(shift, shift);
#pragma unroll
                    for (int c = 0; c < KEYS; c += 32) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = c; e < c + 32 && e < KEYS; e += 2) {
                            float2 f = apart(fma_two(two(__uint_as_float(at(e)), __uint_as_float(at(e + 1))), scale2, shift2));
                            f.x = pow2(f.x);
                            f.y = pow2(f.y);
                            l2[e / 2 & 1] = add_two(l2[e / 2 & 1], two(f.x, f.y));
                            w[(e - c) / 2] = pack2<T>(f.x, f.y);
                        }
                        if (KEYS - c >= 32) st16(p_at + c / 2, w);
                        else st8(p_at + c / 2, w);
                    }
                    tc_wait_st();
                }
                if (!ok) break;
                tc_before();
                __syncwarp();
                if (lane == 0) bar_arrive(p_full + 8 * r);
                ++count;
                some = true;
            }
            const float2 lsum = apart(add_two(l2[0], l2[1]));
            const float l = lsum.x + lsum.y;
            // the unit's (or the part's) output
            if (ok && some) ok = __all_sync(~0u, wait_for(o_done + 8 * r, (count - 1) & 1, &stop, limit));
            tc_after();
            const float nan = nanf("");
            const bool none = p < 0 || l == 0.f, whole = C.split == 1;
            const float by = !ok ? nan : !whole ? 1.f : none ? 0.f : 1.f / l;
            float *const part = whole ? nullptr : part_of<DP, TILES>(C, u, rank);
            T *out = (T *)a.out + U.b * a.o_batch + t * a.o_token + h * a.o_head;
            float odd = 0.f;                                               // NaN once a value was not finite
            if (busy)
#pragma unroll 1
                for (int c = 0; c < DP / 32; ++c) {
                    float v[32];
                    if (some && ok) tc_ld(v, o_at + 32 * c);
                    if (!inside) continue;
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = !ok ? nan : none ? 0.f : v[e] * by;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        const int d = 32 * c + e;
                        if (d >= a.head_dim) break;
                        if (!whole) {
                            store32(part + tile_row * DP + d, v[e], v[e + 1], v[e + 2], v[e + 3], v[e + 4], v[e + 5], v[e + 6], v[e + 7]);
                            continue;
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) odd = fmaf(v[e + k], 0.f, odd);
                        if (A.wide_out) {
                            *(uint4 *)(out + d) = make_uint4(pack2<T>(v[e], v[e + 1]), pack2<T>(v[e + 2], v[e + 3]), pack2<T>(v[e + 4], v[e + 5]),
                                                             pack2<T>(v[e + 6], v[e + 7]));
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k) out[d + k] = from_f32<T>(v[e + k]);
                        }
                    }
                }
            tc_before();
            if (inside && !whole) {
                part[TILES * 128 * DP + tile_row] = m;
                part[TILES * 128 * (DP + 1) + tile_row] = ok ? l : nan;
            } else if (inside && a.lse) {
                a.lse[(U.b * a.tokens + t) * a.q_heads + h] = !ok ? nan : none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            }
            __syncwarp();                                                  // (what follows is written over it)
            for (unsigned again = __ballot_sync(~0u, odd != odd && ok && l == l); again; again &= again - 1) {
                const int k = __ffs(again) - 1, tk = __shfl_sync(~0u, t, k), hh = __shfl_sync(~0u, h, k), pk = __shfl_sync(~0u, p, k);
                if (!spoiled<T>(A, U.r, U.b, U.hk, pk)) continue;
                float ol[8], m1, l1;
                row_by_warp<T, true>(A, U.s, U.b, tk, hh, 0, 1, m1, l1, ol);
                store_out<T>(a, U.b, tk, hh, l1, ol);
            }
        }
    } else {
        fewer_registers<TILES == 2 ? M::FEW : 0>();
        if (warp <= M::HELP + 1) {
            // ---- fetch: one warp Q and K, one V, a lane a box ----
            const bool is_v = warp > M::HELP;
            const uint32_t store = is_v ? sv : sk, full = is_v ? v_full : k_full, empty = is_v ? v_empty : k_empty;
            const CUtensorMap *const map = is_v ? &maps.kv.v : &maps.kv.k;
            const int boxes = KEYS / box;                                  // (boxes of 8 to 64 entries; 1 to 12 of them)
            const uint32_t vain = vain_bytes(A.waits);
            int n = 0, nq[TILES] = {};
            bool ok = true;
            for (int k = 0, u; ok && (u = unit_at(k)) < C.units; ++k) {
                const Unit U = unit_of<KEYS, TILES>(A, C, u, rank, box);
                if (!is_v)
#pragma unroll
                    for (int r = 0; r < TILES; ++r) {
                        if (!ok || span_of(U, C, r).last < 0) continue;
                        ok = __all_sync(~0u, bar_wait(q_empty + 8 * r, (nq[r] + 1) & 1, &stop, limit));   // the first round finds it free
                        if (!ok) continue;
                        if (elected()) {
                            bar_expect(q_full + 8 * r, (uint32_t)(C.tokens * A.group * 128 * (DP / 64)));
#pragma unroll
                            for (int c = 0; c < DP / 64; ++c)
                                box_load(sq + r * M::Q + c * M::SUBQ, &maps.q, 64 * c, U.hk * A.group, U.t0 + r * C.tokens, (int)U.b, q_full + 8 * r);
                        }
                        __syncwarp();
                        ++nq[r];
                    }
                Place at = {0, 0};
                auto find = [&](int i) {
                    const int v = i * KEYS + lane * box;
                    if (lane < boxes && v < U.r.n) at = place_of(a, U.b, U.r.real(v));
                };
                if (U.begin < U.end) find(U.begin);
                for (int i = U.begin; i < U.end && ok; ++i, ++n) {
                    const int st = n % ST;
                    ok = __all_sync(~0u, bar_wait(empty + 8 * st, (n / ST + 1) & 1, &stop, limit));
                    if (!ok) break;
                    const bool mine = lane < boxes && i * KEYS + lane * box < U.r.n;
                    const int count = __popc(__ballot_sync(~0u, mine));
                    if (lane == 0) bar_expect(full + 8 * st, (uint32_t)(count * box * 128 * (DP / 64)) + vain);
                    __syncwarp();
                    if (mine)
#pragma unroll
                        for (int c = 0; c < DP / 64; ++c)
                            box_load(store + st * M::KV + c * M::SUBK + lane * box * 128, map, 64 * c, U.hk, (int)at.in, (int)at.page, full + 8 * st);
                    __syncwarp();
                    if (i + 1 < U.end) find(i + 1);
                }
            }
            // copies under way end before their memory is given back
            for (int i = n > ST ? n - ST : 0; i < n; ++i) {
                int last = 0;
                bar_wait(full + 8 * (i % ST), i / ST & 1, &last, limit);
            }
#pragma unroll
            for (int r = 0; r < TILES; ++r)
                if (nq[r] > 0) {
                    int last = 0;
                    bar_wait(q_full + 8 * r, (nq[r] - 1) & 1, &last, limit);
                }
        } else if (warp >= M::ISSUE && warp < M::ISSUE + TILES) {
            // ---- issue the products of a row tile ----
            const int r = warp - M::ISSUE;
            constexpr uint32_t FMT = __is_same(T, __nv_bfloat16) ? 1u : 0u;
            constexpr uint32_t DESC = 1u << 4 | FMT << 7 | FMT << 10 | (128u >> 4) << 24;
            constexpr uint32_t DESC_S = DESC | (uint32_t)(KEYS >> 3) << 17, DESC_O = DESC | 1u << 16 | (uint32_t)(DP >> 3) << 17;
            const uint32_t qa = (sq + r * M::Q) >> 4 | 1u << 16, k0 = sk >> 4 | 1u << 16, v0 = sv >> 4 | (uint32_t)(M::SUBK / 16) << 16;
            const uint32_t s_col = tmem + M::S_COL + r * KEYS, p_col = tmem + M::P_COL + r * KEYS / 2, o_col = tmem + M::O_COL + r * DP;
            // One lane does it all: it is alone in what follows, so that nothing has to be agreed on
            // between two instructions.
            if (elected()) {
                uint32_t fixes = 0;                                        // parity of v_fixed of a stage, a bit each
                uint32_t k_st = 0, k_par = 0, v_st = 0, v_par = 0;         // stages of the next scores and outputs, and their barriers' parities
                uint32_t scores = 0, done = 0, nq = 0;                     // score tiles, products and units
                bool ok = true;
                for (int k = 0, u; ok && (u = unit_at(k)) < C.units; ++k) {
                    const Unit U = unit_of<KEYS, TILES>(A, C, u, rank, box);
                    const Span span = span_of(U, C, r);
                    const Reach reach = reach_of<KEYS>(A, U.r, span);
                    const Idle idle = idle_of<KEYS>(A, U.r);
                    uint32_t more = 0;                                     // O has a product of this unit
                    if (span.last >= 0) ok = bar_wait(q_full + 8 * r, nq++ & 1, &stop, limit);
                    // the scores of tile i + 1, then the outputs of tile i
                    for (int i = U.begin - 1; i < U.end && ok; ++i) {
                        if (i + 1 < U.end) {
                            ok = wait_for(k_full + 8 * k_st, k_par, &stop, limit);
                            if (reach.some(i + 1)) {
                                if (scores > 0) ok = ok && wait_for(s_free + 8 * r, (scores - 1) & 1, &stop, limit);
                                if (!ok) break;
                                const uint32_t ka = k0 + k_st * (M::KV / 16);
                                tc_after();
#pragma unroll
                                for (int k = 0; k < DP / 16; ++k)
                                    tc_mma_ss(s_col, desc_of(qa + ((k >> 2) * M::SUBQ + (k & 3) * 32) / 16),
                                              desc_of(ka + ((k >> 2) * M::SUBK + (k & 3) * 32) / 16), DESC_S, k > 0);
                                tc_commit(s_full + 8 * r);
                                tc_commit(k_empty + 8 * k_st);
                                ++scores;
                            } else {
                                if (!ok) break;
                                bar_arrive(k_empty + 8 * k_st);
                            }
                            if (++k_st == ST) {
                                k_st = 0;
                                k_par ^= 1;
                            }
                        }
                        if (span.last >= 0 && (i + 2 == U.end || U.begin == U.end)) tc_commit(q_empty + 8 * r);
                        if (i < U.begin) continue;
                        ok = wait_for(v_full + 8 * v_st, v_par, &stop, limit);
                        if (idle.any(i)) {
                            ok = ok && bar_wait(v_fixed + 8 * v_st, fixes >> v_st & 1u, &stop, limit);
                            fixes ^= 1u << v_st;
                        }
                        if (reach.some(i)) {
                            ok = ok && wait_for(p_full + 8 * r, done & 1, &stop, limit);
                            if (!ok) break;
                            const uint32_t va = v0 + v_st * (M::KV / 16);
                            tc_after();
#pragma unroll
                            for (int k = 0; k < KEYS / 16; ++k) tc_mma_ts(o_col, p_col + 8 * k, desc_of(va + k * 2048 / 16), DESC_O, k > 0 ? 1u : more);
                            tc_commit(o_done + 8 * r);
                            tc_commit(v_empty + 8 * v_st);
                            ++done;
                            more = 1;
                        } else {
                            if (!ok) break;
                            bar_arrive(v_empty + 8 * v_st);
                        }
                        if (++v_st == ST) {
                            v_st = 0;
                            v_par ^= 1;
                        }
                    }
                }
                // products under way end before their memory is given back
                tc_commit(last_bar);
                int last = 0;
                bar_wait(last_bar, 0, &last, limit);
            }
            __syncwarp();
        } else if (warp == M::CLEAR) {
            // ---- clear what no row of the unit sees in V: copied with a box, or behind the line ----
            int n = 0;
            bool ok = true;
            for (int k = 0, u; ok && (u = unit_at(k)) < C.units; ++k) {
                const Unit U = unit_of<KEYS, TILES>(A, C, u, rank, box);
                const Idle idle = idle_of<KEYS>(A, U.r);
                for (int i = U.begin; i < U.end && ok; ++i, ++n) {
                    const int st = n % ST;
                    ok = __all_sync(~0u, bar_wait(v_full + 8 * st, n / ST & 1, &stop, limit));
                    if (!ok) break;
                    if (idle.any(i)) {
                        for (int k0 = 0; k0 < KEYS; k0 += 32) {
                            const int v = i * KEYS + k0 + lane;
                            unsigned clear = __ballot_sync(~0u, k0 + lane < KEYS && (v >= U.r.n || !seen_by_any(A, U.r, U.r.real(v))));
                            for (; clear; clear &= clear - 1) {
                                const uint32_t at = sv + st * M::KV + (k0 + __ffs(clear) - 1) * 128;
                                if (lane < DP / 8)
                                    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at + (lane >> 3) * M::SUBK + ((lane & 7) << 4)), "r"(0) : "memory");
                            }
                        }
                        async_fence();
                        __syncwarp();
                        if (lane == 0) bar_arrive(v_fixed + 8 * st);
                    }
                    __syncwarp();
                    if (lane == 0) bar_arrive(v_empty + 8 * st);
                }
            }
        }
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    if (warp == M::ISSUE) {
        tc_after();
        tc_free(tmem);
    }
    if (tid == 0 && stop) ran_out = 1;
}

constexpr int JOIN_NT = 128, JOIN_SPLIT = 16;

// Joins the parts of a unit, a row by each warp: the lanes read the parts' maxima and sums, then
// all add up the parts' outputs in order, several loads at a time.
template <class T, int DP, int TILES>
__global__ void __launch_bounds__(JOIN_NT) k_window_join(Win A, Cut C)
{
    const dbs_window_args &a = A.a;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, i = (int)(blockIdx.x * (JOIN_NT / 32) + (threadIdx.x >> 5)), u = i / (TILES * 128), tile_row = i % (TILES * 128);
    const uint32_t heads = (uint32_t)a.kv_heads, per = (uint32_t)a.batch * heads, g = (uint32_t)u / per, bh = (uint32_t)u - g * per;
    const int64_t b = bh / heads;
    const int hk = (int)(bh % heads), row = tile_row % 128, dt = row / A.group;
    const int t0 = (C.groups - 1 - (int)g) * TILES * C.tokens, t = t0 + tile_row / 128 * C.tokens + dt, h = hk * A.group + row - dt * A.group;
    if (dt >= C.tokens || t >= a.tokens) return;
    const Seq s = sequence(A, b);
    const float *const parts = part_of<DP, TILES>(C, u, 0);
    constexpr int64_t PART = part_floats<DP, TILES>();
    const bool in = lane < C.split;
    const float m = in ? __ldcg(parts + lane * PART + TILES * 128 * DP + tile_row) : -INFINITY;
    float l = in ? __ldcg(parts + lane * PART + TILES * 128 * (DP + 1) + tile_row) : 0.f, top = m;
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    const float f = weight_of(m, l, top);
    l = weighed(f, l);
#pragma unroll
    for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
    if (t >= s.tokens || s.first + t < 0) l = 0.f;
    float o[8] = {};
#pragma unroll 4
    for (int k = 0; k < C.split; ++k) {
        const float fk = __shfl_sync(~0u, f, k);
#pragma unroll
        for (int e = 0; e < DP / 32; ++e) {
            const float x = lane + 32 * e < a.head_dim ? __ldcg(parts + k * PART + tile_row * DP + lane + 32 * e) : 0.f;
            o[e] += fk * x;
        }
    }
    bool odd = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (l == 0.f) o[e] = 0.f;
        odd |= !isfinite(o[e]);
    }
    store_row<T>(a, b, t, h, top, l, o);
    if (l == l && __any_sync(~0u, odd) && spoiled<T>(A, range_of(A, s, t0, t0 + TILES * C.tokens - 1, 1), b, hk, s.first + t)) {
        float m1, l1;
        row_by_warp<T, true>(A, s, b, t, h, 0, 1, m1, l1, o);
        store_out<T>(a, b, t, h, l1, o);
    }
}

bool args_ok(const dbs_window_args *a)
{
    constexpr int64_t INTS = int64_t(1) << 31;
    if (!a || (a->dtype != DBS_F16 && a->dtype != DBS_BF16) || a->head_dim < 1 || a->head_dim > 256 || a->kv_heads < 1 ||
        a->kv_heads > 65536 || a->q_heads < a->kv_heads || a->q_heads > 65536 || a->q_heads % a->kv_heads || a->batch < 0 ||
        a->batch >= INTS || a->tokens < 0 || a->tokens > INTS - 1024 || a->pages < 0 || a->page_size < 0 || a->max_pages < 0 ||
        a->page_size >= INTS || a->max_pages >= INTS || a->pages >= INTS || a->window < 1 || a->sinks < 0 || !std::isfinite(a->scale))
        return false;
    if (a->batch == 0 || a->tokens == 0) return true;
    if (a->batch * a->tokens >= INTS || a->batch * a->tokens * a->q_heads >= INTS) return false;
    const int64_t entries = a->max_pages * a->page_size;
    if (entries > INTS - 1024) return false;                             // (an entry's number and a tile's end are ints)
    if (!a->q || !a->out || !a->kv_lens) return false;
    if (entries > 0 && (!a->k || !a->v || a->pages < 1)) return false;
    for (int64_t stride : {a->q_batch, a->q_token, a->q_head, a->k_page, a->k_entry, a->k_head, a->v_page, a->v_entry, a->v_head,
                           a->page_row, a->o_batch, a->o_token, a->o_head})
        if (stride < 0) return false;
    // heads of out that share memory, or are the inputs'
    const int64_t pages = entries > 0 ? a->pages : 0;
    const Places out(a->out, 2, a->head_dim, {{a->batch, a->o_batch}, {a->tokens, a->o_token}, {a->q_heads, a->o_head}});
    if (!out.own || out.meets({a->q, 2, a->head_dim, {{a->batch, a->q_batch}, {a->tokens, a->q_token}, {a->q_heads, a->q_head}}}) ||
        out.meets({a->k, 2, a->head_dim, {{pages, a->k_page}, {a->page_size, a->k_entry}, {a->kv_heads, a->k_head}}}) ||
        out.meets({a->v, 2, a->head_dim, {{pages, a->v_page}, {a->page_size, a->v_entry}, {a->kv_heads, a->v_head}}}))
        return false;
    if (!a->page_table && (a->max_pages > 1 || (entries > 0 && a->pages < a->batch))) return false;
    return true;
}

// ---- host ----

// Entries that a unit of `tokens` tokens may have, all that the line may hold.
int64_t line_of(const dbs_window_args &a, int64_t tokens)
{
    const int64_t entries = a.max_pages * a.page_size;
    return a.window >= entries || a.sinks >= entries || a.window + a.sinks + tokens >= entries ? entries : a.window + a.sinks + tokens - 1;
}

template <class T, int DP, bool BOXES>
dbs_status launch_few(const Win &A, const Maps &maps, cudaStream_t s)
{
    using F = Few<DP>;
    static Once once;
    const int sms = multiprocessors();
    if (sms == 0) return DBS_ERR_CUDA;
    const int64_t rows = A.a.tokens * A.group, groups = (rows + FEW_ROWS - 1) / FEW_ROWS, units = A.a.batch * A.a.kv_heads * groups;
    // Blocks of a unit: enough to fill the GPU's multiprocessors twice, up to four with a turn of its entries each,
    // eight with more than one, more with four or more: a turn takes 1.2 us, a join of eight or sixteen blocks
    // longer.  (One token, 8 kv heads of 128: 200 entries 6.8 us, in one block 8.1; 1024 in eight blocks 7.5, in
    // sixteen 8.0; 8192 in sixteen 13.6, in four 30; 32768 34.9 and 105.)
    const int64_t turns = (line_of(A.a, FEW_ROWS) + FEW_KEYS - 1) / FEW_KEYS;
    const int most = DP == 256 ? 8 : FEW_SPLIT;
    int split = 1;
    while (split < most && units * split * 2 <= 2 * sms && (split < 4 ? turns > split : split < 8 ? turns > 2 * split : turns >= 4 * split))
        split *= 2;
    if (!room_for(once, k_window_few<T, DP, BOXES>, F::SMEM, true)) return DBS_ERR_CUDA;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(units * split));
    c.blockDim = FEW_NT;
    c.dynamicSmemBytes = F::SMEM;
    c.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)split;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    cudaLaunchKernelEx(&c, k_window_few<T, DP, BOXES>, A, (int)groups, split, maps);
    return launched();
}

// Q's rows as boxes of a row tile: 64 columns of a kv head's query heads of `tokens` tokens.
bool make_q_map(const dbs_window_args &a, int group, int tokens, CUtensorMap &map)
{
    const cuuint64_t dims[4] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.q_heads, (cuuint64_t)a.tokens, (cuuint64_t)a.batch};
    return map_of(map, a.dtype, a.q, dims, {a.q_head, a.q_token, a.q_batch}, {64, (cuuint32_t)group, (cuuint32_t)tokens, 1});
}

template <class T, int DP, int TILES>
dbs_status launch_many(const Win &A, Cut C, const ManyMaps &maps, cudaStream_t s)
{
    using M = Many<DP, TILES>;
    static Once once;
    if (!room_for(once, k_window_many<T, DP, TILES>, M::SMEM, false, TILES == 2 ? M::REGS : 0)) return DBS_ERR_CUDA;
    const int sms = multiprocessors();
    k_window_many<T, DP, TILES><<<C.split > 1 ? C.units * C.split : C.units < sms ? C.units : sms, M::NT, M::SMEM, s>>>(A, C, maps);
    const dbs_status st = launched();
    if (st != DBS_OK || C.split == 1) return st;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(C.units * TILES * 128 / (JOIN_NT / 32)));
    c.blockDim = JOIN_NT;
    c.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, k_window_join<T, DP, TILES>, A, C) == cudaSuccess ? DBS_OK : (cudaGetLastError(), DBS_ERR_CUDA);
}

// How a call runs.
struct Plan {
    bool rows, many;           // any alignment; 128 rows at a time
    ManyMaps maps;             // of `many`, with Q; of the kernel for few rows without
    bool boxes;                // there are maps
    Cut cut;                   // of `many`
    int64_t scratch;           // bytes
};

dbs_status plan_of(const dbs_window_args &a, Plan &P)
{
    P.rows = !on_vectors(a);
    P.many = P.boxes = false;
    P.scratch = 0;
    if (P.rows) return DBS_OK;
    const int sms = multiprocessors(), group = a.q_heads / a.kv_heads, dp = a.head_dim <= 64 ? 64 : a.head_dim <= 128 ? 128 : 256;
    if (sms == 0) return DBS_ERR_CUDA;
    // Many rows of a kv head: 128 at a time, if K, V and Q can be copied as boxes (sinks and the
    // window's start round to them).  Heads of 128, 8 of kv, 16 rows, one sequence of 8192 entries and 32 of 4096: 16.8 us and 103, by
    // 16 at a time 15.0 and 97; 24 rows 16.8 and 103, by 16 at a time 26 and 141; 64 rows 18.7 and 107, 22 and 277.
    if (a.tokens * group > FEW_ROWS && group <= 128 && a.scale > 0 && make_maps(a, a.sinks > 0 || dp == 128 ? 16 : dp == 256 ? 64 : 32, P.maps.kv) &&
        make_q_map(a, group, 128 / group, P.maps.q)) {
        const int tiles = dp == 256 ? 1 : 2, keys = dp == 64 ? 96 : dp == 128 ? 80 : 64;
        Cut &C = P.cut;
        C.tokens = 128 / group;
        C.groups = (int)((a.tokens + tiles * C.tokens - 1) / (tiles * C.tokens));
        C.units = (int)(a.batch * a.kv_heads * C.groups);
        C.scratch = nullptr;
        // Blocks of a unit: as many as find room at once, with two tiles each at least (64 tokens, 32/8 heads, window 4096:
        // 22 us, in one block 62; 8 sequences of 8 tokens over 2111 entries 24 and 29).
        const int64_t line = (line_of(a, tiles * C.tokens) + keys - 1) / keys;
        int64_t split = sms / C.units;
        split = split < line / 2 ? split : line / 2;
        C.split = (int)(split < 1 ? 1 : split < JOIN_SPLIT ? split : JOIN_SPLIT);
        if (C.split > 1) P.scratch = (int64_t)C.units * C.split * tiles * 128 * (dp + 2) * (int64_t)sizeof(float);
        P.many = P.boxes = true;
        return DBS_OK;
    }
    P.boxes = make_maps(a, FEW_STEP, P.maps.kv);
    return DBS_OK;
}

template <class T, int DP>
dbs_status launch_size(const Win &A, const Plan &P, cudaStream_t s)
{
    if (P.many) return launch_many<T, DP, DP == 256 ? 1 : 2>(A, P.cut, P.maps, s);
    return P.boxes ? launch_few<T, DP, true>(A, P.maps.kv, s) : launch_few<T, DP, false>(A, P.maps.kv, s);
}

template <class T>
dbs_status launch(const Win &A, const Plan &P, cudaStream_t s)
{
    if (P.rows) {
        k_window_rows<T><<<(unsigned)(A.a.batch * A.a.tokens * A.a.q_heads), ROW_NT, 0, s>>>(A);
        return launched();
    }
    const int d = A.a.head_dim;
    return d <= 64 ? launch_size<T, 64>(A, P, s) : d <= 128 ? launch_size<T, 128>(A, P, s) : launch_size<T, 256>(A, P, s);
}

}  // namespace

namespace dbs::ops {
dbs_status window_waits_since(cudaStream_t s) { return waits_since(s); }
}  // namespace dbs::ops

extern "C" {

dbs_status dbs_window_attention_scratch(const dbs_window_args *a, int64_t *bytes)
{
    if (!bytes || !args_ok(a)) return DBS_ERR_INVALID_ARG;
    *bytes = 0;
    if (a->batch == 0 || a->tokens == 0) return DBS_OK;
    Plan P;
    const dbs_status st = plan_of(*a, P);
    if (st == DBS_OK) *bytes = P.scratch;
    return st;
}

dbs_status dbs_window_attention(const dbs_window_args *a, void *stream)
{
    if (!args_ok(a)) return DBS_ERR_INVALID_ARG;
    if (a->batch == 0 || a->tokens == 0) return DBS_OK;
    Plan P;
    const dbs_status st = plan_of(*a, P);
    if (st != DBS_OK) return st;
    if (P.scratch > 0 && (!a->scratch || (reinterpret_cast<uintptr_t>(a->scratch) & 31u) || a->scratch_bytes < P.scratch)) return DBS_ERR_INVALID_ARG;
    P.cut.scratch = (float *)a->scratch;
    constexpr int64_t MOST = 0x7fffffff - 1023;                          // (as many entries as there may be)
    const Win A{*a, a->scale * 1.4426950408889634f, (int)(a->window < MOST ? a->window : MOST), (int)(a->sinks < MOST ? a->sinks : MOST),
                a->q_heads / a->kv_heads, wide_out(a->out, a->o_batch, a->o_token, a->o_head), waits()};
    return a->dtype == DBS_F16 ? launch<__half>(A, P, (cudaStream_t)stream) : launch<__nv_bfloat16>(A, P, (cudaStream_t)stream);
}

}  // extern "C"
