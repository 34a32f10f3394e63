// Attention with a sliding window and sinks over a (paged) cache
// (dbs_window_attention, sm_103a): softmax over the entries a token sees, with the
// running maximum and sum held in fp32.
#include "ops_dev.h"
#include "tc_dev.h"

#include <cmath>

using namespace dbs::ops;

namespace {

struct Win {
    dbs_window_args a;
    float scale_log2;          // scale * log2(e): probabilities are powers of two
    int window, sinks;         // (at most 2^31 - 1)
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

// Where entry j of sequence b lies: its page, and its place in it.
struct Place {
    int64_t page;
    uint32_t in;
};

__device__ __forceinline__ Place place_of(const dbs_window_args &a, int64_t b, int j)
{
    if (!a.page_table) return {b, (uint32_t)j};
    const uint32_t size = (uint32_t)a.page_size, n = (uint32_t)j / size;
    const int64_t p = a.page_table[b * a.page_row + n];
    return {p < 0 ? 0 : p >= a.pages ? a.pages - 1 : p, (uint32_t)j - n * size};
}

// The first entry of the window of a token at position p (p >= 0).
__device__ __forceinline__ int window_start(const Win &A, int p) { return p >= A.window ? p - A.window + 1 : 0; }

// One query row by one warp, entry by entry (every step-th of those it sees, from the
// part-th on), touching only what the row sees.
template <class T>
__device__ __forceinline__ void row_by_warp(const Win &A, const Seq &s, int64_t b, int t, int h, int part, int step, float &m, float &l,
                                            float (&o)[8])
{
    const dbs_window_args &a = A.a;
    const int lane = threadIdx.x & 31, hk = h / A.group;
    const T *q = (const T *)a.q + b * a.q_batch + t * a.q_token + h * a.q_head;
    float qr[8];
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        qr[e] = lane + 32 * e < a.head_dim ? to_f32(q[lane + 32 * e]) : 0.f;
        o[e] = 0.f;
    }
    const int p = s.first + t;
    if (t >= s.tokens || p < 0) return;
    const int lo = window_start(A, p), sinks = A.sinks < lo ? A.sinks : lo, n = sinks + p + 1 - lo;
    for (int i = part; i < n; i += step) {
        const Place at = place_of(a, b, i < sinks ? i : lo + i - sinks);
        const T *k = (const T *)a.k + at.page * a.k_page + at.in * a.k_entry + hk * a.k_head;
        const T *v = (const T *)a.v + at.page * a.v_page + at.in * a.v_entry + hk * a.v_head;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (lane + 32 * e < a.head_dim) x = fmaf(qr[e], to_f32(k[lane + 32 * e]), x);
#pragma unroll
        for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
        x *= A.scale_log2;
        const float top = fmaxf(m, x);
        // all scores -inf so far: nothing is carried and nothing counts
        const float keep = m == -INFINITY ? 0.f : exp2f(m - top);
        const float pr = x == -INFINITY ? 0.f : exp2f(x - top);
        l = l * keep + pr;
        m = top;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (lane + 32 * e < a.head_dim) o[e] = fmaf(pr, to_f32(v[lane + 32 * e]), o[e] * keep);
    }
}

// Writes a row from its sums: out = o / l, lse = (m + log2 l) ln 2.
template <class T>
__device__ __forceinline__ void store_row(const Win &A, int64_t b, int t, int h, float m, float l, const float (&o)[8])
{
    const dbs_window_args &a = A.a;
    const int lane = threadIdx.x & 31;
    T *out = (T *)a.out + b * a.o_batch + t * a.o_token + h * a.o_head;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (lane + 32 * e < a.head_dim) out[lane + 32 * e] = from_f32<T>(l == 0.f ? 0.f : o[e] / l);
    if (a.lse && lane == 0) a.lse[(b * a.tokens + t) * a.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

constexpr int ROW_NT = 128;

// Any head size and alignment: one block per query row, its warps take every fourth
// entry, a lane every 32nd value.
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
            // a maximum of -inf: nothing there, or a NaN that has to stay
            const float f = s_m[w] == -INFINITY ? (s_l[w] != s_l[w] ? 1.f : 0.f) : exp2f(s_m[w] - top);
            sum += f * s_l[w];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] += f == 0.f ? 0.f : f * s_o[w][lane + 32 * e];
        }
        store_row<T>(A, b, t, (int)h, top, sum, o);
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
    r.lo = window_start(A, r.first) / grain * grain;
    if (A.sinks < r.lo) r.sinks = (A.sinks + grain - 1) / grain * grain;
    if (A.sinks >= r.lo || r.sinks >= r.lo) r.sinks = r.lo = 0;
    r.n = r.sinks + r.hi - r.lo;
    return r;
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
// through shared memory; a row whose result is not finite, because of an entry that others see or
// of one of its own, is made anew by a warp from what it sees alone.

// ---- few rows: every warp streams its own entries ----

// Tensor maps of K and V: [pages, entries, heads, head_dim], boxes of 64 columns of one head
// of `box` entries.
struct Maps {
    CUtensorMap k, v;
    int box;
};

__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap *map, int d, int head, int entry, int page, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
                 "l"(map), "r"(bar), "r"(d), "r"(head), "r"(entry), "r"(page) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool take)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <class T> __device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (__is_same(T, __half))
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float remote(const void *p, int block)
{
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(block));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() { asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory"); }

constexpr int FEW_NT = 128, FEW_W = FEW_NT / 32;
constexpr int FEW_ROWS = 16;               // one matrix instruction's rows
constexpr int FEW_STEP = 16;               // entries of a stage of a warp
constexpr int FEW_KEYS = FEW_W * FEW_STEP;
constexpr int FEW_SPLIT = 16;              // blocks of a cluster, at most

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
// windows are read, by latency for one.
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
            const float f = s_m[w][r] == -INFINITY ? (s_l[w][r] != s_l[w][r] ? 1.f : 0.f) : exp2f(s_m[w][r] - top);
            const float *po = (const float *)(ring + w * F::RING) + r * DP;
            sum += f * s_l[w][r];
#pragma unroll
            for (int e = 0; e < DP / 32; ++e) oo[e] += f == 0.f ? 0.f : f * po[lane + 32 * e];
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
        const float f = m == -INFINITY ? (l != l ? 1.f : 0.f) : exp2f(m - top);
        l = f == 0.f ? 0.f : f * l;
#pragma unroll
        for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
#pragma unroll
        for (int k = 0; k < FEW_SPLIT; ++k) {
            const float fk = __shfl_sync(~0u, f, k);
            out += fk == 0.f ? 0.f : fk * v[k];
        }
        if (row.p < 0) l = out = 0.f;
        if (l == l && __any_sync(~0u, col < a.head_dim && !isfinite(out))) {
            float ol[8], m1, l1;
            row_by_warp<T>(A, s, b, row.t, row.h, 0, 1, m1, l1, ol);
#pragma unroll
            for (int e = 0; e < 8; ++e) out = e == e0 ? ol[e] : out;
            l = l1;
            top = m1;
        }
        if (col < a.head_dim) ((T *)a.out + b * a.o_batch + row.t * a.o_token + row.h * a.o_head)[col] = from_f32<T>(l == 0.f ? 0.f : out / l);
        if (a.lse && e0 == 0 && lane == 0) a.lse[(b * a.tokens + row.t) * a.q_heads + row.h] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
    }
    // (no block ends while another one reads its shared memory)
    if (split > 1) cluster_sync();
    if (threadIdx.x == 0 && stop) ran_out = 1;
}

bool args_ok(const dbs_window_args *a)
{
    constexpr int64_t INTS = int64_t(1) << 31;
    if (!a || (a->dtype != DBS_F16 && a->dtype != DBS_BF16) || a->head_dim < 1 || a->head_dim > 256 || a->kv_heads < 1 ||
        a->kv_heads > 65536 || a->q_heads < a->kv_heads || a->q_heads > 65536 || a->q_heads % a->kv_heads || a->batch < 0 ||
        a->batch >= INTS || a->tokens < 0 || a->tokens >= INTS || a->pages < 0 || a->page_size < 0 || a->max_pages < 0 ||
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
    // heads of out that share memory
    if ((a->q_heads > 1 && a->o_head < a->head_dim) || (a->tokens > 1 && a->o_token < a->head_dim) ||
        (a->batch > 1 && a->o_batch < a->head_dim))
        return false;
    if (!a->page_table && (a->max_pages > 1 || (entries > 0 && a->pages < a->batch))) return false;
    return true;
}

// ---- host ----

bool aligned8(int64_t v) { return (v & 7) == 0; }

// 16-byte copies of heads: every head starts on such a boundary.
bool on_vectors(const dbs_window_args &a)
{
    return a.head_dim % 8 == 0 && aligned16(a.q) && aligned16(a.k) && aligned16(a.v) && aligned8(a.q_batch) && aligned8(a.q_token) &&
           aligned8(a.q_head) && aligned8(a.k_page) && aligned8(a.k_entry) && aligned8(a.k_head) && aligned8(a.v_page) &&
           aligned8(a.v_entry) && aligned8(a.v_head);
}

// Boxes of the caches, of `most` entries or as many as divide a page, or false where pages or
// strides do not allow them.
bool make_maps(const dbs_window_args &a, int most, Maps &M)
{
    const encode_tiled_fn encode = encode_tiled();
    if (!encode || a.page_size < 1 || a.pages < 1 || a.max_pages < 1) return false;
    // a sequence's own page is one run of entries; pages of a table split into boxes
    M.box = most;
    if (a.page_table)
        while (M.box >= 8 && a.page_size % M.box) M.box /= 2;
    if (M.box < 8) return false;
    for (int i = 0; i < 2; ++i) {
        const cuuint64_t dims[4] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.kv_heads, (cuuint64_t)a.page_size, (cuuint64_t)a.pages};
        const int64_t by[3] = {i ? a.v_head : a.k_head, i ? a.v_entry : a.k_entry, i ? a.v_page : a.k_page};
        const cuuint32_t box[4] = {64, 1, (cuuint32_t)M.box, 1}, ones[4] = {1, 1, 1, 1};
        cuuint64_t strides[3];
        for (int d = 0; d < 3; ++d) {
            // (a dimension of one entry has any stride)
            const int64_t bytes = dims[d + 1] == 1 ? 16 * a.head_dim : by[d] * 2;
            if (bytes <= 0 || bytes >= int64_t(1) << 40 || dims[d + 1] >= cuuint64_t(1) << 31) return false;
            strides[d] = (cuuint64_t)bytes;
        }
        if (encode(i ? &M.v : &M.k, a.dtype == DBS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                   const_cast<void *>(i ? a.v : a.k), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    return true;
}

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
    if (units * FEW_SPLIT >= int64_t(1) << 31) return DBS_ERR_INVALID_ARG;
    // Blocks of a unit: enough to fill the GPU's multiprocessors twice, with two turns of
    // its entries each at least.
    const int64_t turns = (line_of(A.a, FEW_ROWS) + FEW_KEYS - 1) / FEW_KEYS;
    const int most = DP == 256 ? 8 : FEW_SPLIT;
    int split = 1;
    while (split < most && units * split * 2 <= 2 * sms && turns >= 4 * split) split *= 2;
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

template <class T, int DP>
dbs_status launch_size(const Win &A, cudaStream_t s)
{
    Maps maps{};
    return make_maps(A.a, FEW_STEP, maps) ? launch_few<T, DP, true>(A, maps, s) : launch_few<T, DP, false>(A, maps, s);
}

template <class T>
dbs_status launch(const Win &A, cudaStream_t s)
{
    if (!on_vectors(A.a)) {
        k_window_rows<T><<<(unsigned)(A.a.batch * A.a.tokens * A.a.q_heads), ROW_NT, 0, s>>>(A);
        return launched();
    }
    const int d = A.a.head_dim;
    return d <= 64 ? launch_size<T, 64>(A, s) : d <= 128 ? launch_size<T, 128>(A, s) : launch_size<T, 256>(A, s);
}

}  // namespace

namespace dbs::ops {
dbs_status window_waits_since(cudaStream_t s) { return waits_since(s); }
}  // namespace dbs::ops

extern "C" dbs_status dbs_window_attention(const dbs_window_args *a, void *stream)
{
    if (!args_ok(a)) return DBS_ERR_INVALID_ARG;
    if (a->batch == 0 || a->tokens == 0) return DBS_OK;
    constexpr int64_t MOST = 0x7fffffff;
    const bool wide_out = aligned16(a->out) && aligned8(a->o_batch) && aligned8(a->o_token) && aligned8(a->o_head);
    const Win A{*a, a->scale * 1.4426950408889634f, (int)(a->window < MOST ? a->window : MOST), (int)(a->sinks < MOST ? a->sinks : MOST),
                a->q_heads / a->kv_heads, wide_out, waits()};
    return a->dtype == DBS_F16 ? launch<__half>(A, (cudaStream_t)stream) : launch<__nv_bfloat16>(A, (cudaStream_t)stream);
}
