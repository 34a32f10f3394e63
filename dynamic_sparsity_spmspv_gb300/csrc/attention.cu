// Attention of drafted tokens over a (paged) cache (dbs_tree_attention,
// sm_103a): softmax over the entries a token sees, with the running maximum
// and sum held in fp32.
#include "ops_dev.h"
#include "tc_dev.h"

#include <cmath>

using namespace dbs::ops;

namespace {

struct Attn {
    dbs_attention_args a;
    float scale_log2;          // scale * log2(e): probabilities are powers of two
    int words;                 // 64-bit mask words per token
    bool wide_out;             // heads of out start on 16-byte boundaries
    int group;                 // query heads of a kv head
    Waits waits;
};

// What sequence b holds, with every length clamped to its range.
struct Seq {
    int kv, first;             // entries; index of the first drafted one (may be < 0)
    int tree;                  // drafted tokens
};

__device__ __forceinline__ Seq sequence(const Attn &A, int64_t b)
{
    const dbs_attention_args &a = A.a;
    Seq s;
    const int64_t room = a.max_pages * a.page_size;
    int64_t kv = a.kv_lens[b], t = a.tree_lens ? a.tree_lens[b] : a.tokens;
    s.kv = (int)(kv < 0 ? 0 : kv > room ? room : kv);
    s.tree = (int)(t < 0 ? 0 : t > a.tokens ? a.tokens : t);
    s.first = s.kv - s.tree;
    return s;
}

// Where entry j of sequence b lies: its page, and its place in it.
struct Place {
    int64_t page;
    uint32_t in;
};

__device__ __forceinline__ Place place_of(const dbs_attention_args &a, int64_t b, int j)
{
    if (!a.page_table) return {b, (uint32_t)j};
    const uint32_t size = (uint32_t)a.page_size, n = (uint32_t)j / size;
    const int64_t p = a.page_table[b * a.page_row + n];
    return {p < 0 ? 0 : p >= a.pages ? a.pages - 1 : p, (uint32_t)j - n * size};
}

// Whether token t of sequence b sees drafted entry i (0 <= i < tree).
__device__ __forceinline__ bool sees(const Attn &A, int64_t b, int t, int i)
{
    if (!A.a.tree) return i <= t;
    return (uint64_t)A.a.tree[(b * A.a.tokens + t) * A.words + (i >> 6)] >> (i & 63) & 1u;
}

// Row `r` of a unit's rows: R = token * G + head within the group.
struct Row {
    int t, h;
    bool inside;               // a row of the call (R < tokens * G)
};

__device__ __forceinline__ Row row_of(const Attn &A, int hk, int64_t R)
{
    const uint32_t G = (uint32_t)A.group, t = (uint32_t)R / G;             // (tokens * G < 2^27)
    Row r;
    r.t = (int)t;
    r.h = hk * (int)G + (int)((uint32_t)R - t * G);
    r.inside = R < A.a.tokens * G;
    return r;
}

// Visibility of the 32 entries from drafted index `node` on (bit k: entry
// node + k) for token t.  Entries below 0 are the earlier part of the cache.
__device__ __forceinline__ uint32_t sees32(const Attn &A, int64_t b, int t, int tree, int node)
{
    if (t >= tree || node >= tree) return 0u;
    if (node <= -32) return ~0u;
    uint32_t m;
    if (!A.a.tree) {
        const int n = t - node + 1;                  // the first n entries
        m = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
    } else {
        const uint64_t *w = (const uint64_t *)A.a.tree + (b * A.a.tokens + t) * A.words;
        if (node < 0) {
            m = (uint32_t)(w[0] << -node) | ((1u << -node) - 1u);
        } else {
            const int i = node >> 6, sh = node & 63;
            uint64_t v = w[i] >> sh;
            if (sh > 32 && i + 1 < A.words) v |= w[i + 1] << (64 - sh);
            m = (uint32_t)v;
        }
    }
    const int left = tree - node;                    // drafted entries end here
    return left >= 32 ? m : m & ((1u << left) - 1u);
}

// One query row by one warp, entry by entry, touching only what the row sees.
template <class T>
__device__ __forceinline__ void row_by_warp(const Attn &A, int64_t b, int t, int h, int j0, int step, float &m, float &l,
                                         float (&o)[8])
{
    const dbs_attention_args &a = A.a;
    const int lane = threadIdx.x & 31, hk = h / (a.q_heads / a.kv_heads);
    const Seq s = sequence(A, b);
    const T *q = (const T *)a.q + b * a.q_batch + t * a.q_token + h * a.q_head;
    float qr[8];
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        qr[e] = lane + 32 * e < a.head_dim ? to_f32(q[lane + 32 * e]) : 0.f;
        o[e] = 0.f;
    }
    if (t >= s.tree) return;
    for (int j = j0; j < s.kv; j += step) {
        if (j >= s.first && !sees(A, b, t, j - s.first)) continue;
        const Place at = place_of(a, b, j);
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

// The matrix products give every row every entry of a tile, with probability
// 0 where it is not seen, and 0 * NaN is NaN.  So a NaN or infinity in the
// drafted part of V (the part that rows see differently) is replaced by 0 on
// its way through shared memory, the unit is marked, and the rows that do see
// such a value get it here, in the end: a positive probability times it is the
// value itself, whatever the order.
template <class T> struct Odd;
template <> struct Odd<__half> { static constexpr uint32_t exp = 0x7c00u; };
template <> struct Odd<__nv_bfloat16> { static constexpr uint32_t exp = 0x7f80u; };

// Clears what is not finite in two packed values; returns whether there was any.
template <class T>
__device__ __forceinline__ bool clear_odd(uint32_t &w)
{
    const bool lo = (w & Odd<T>::exp) == Odd<T>::exp, hi = (w >> 16 & Odd<T>::exp) == Odd<T>::exp;
    if (lo) w &= 0xffff0000u;
    if (hi) w &= 0x0000ffffu;
    return lo || hi;
}

struct Eight {
    float v[8];
};

// (by value, so that the caller's sums stay in registers)
template <class T>
__device__ __noinline__ Eight add_odd(const Attn &A, int64_t b, int t, int hk, Eight o)
{
    const dbs_attention_args &a = A.a;
    const int lane = threadIdx.x & 31;
    const Seq s = sequence(A, b);
    for (int i = s.first < 0 ? -s.first : 0; i < s.tree; ++i) {
        if (!sees(A, b, t, i)) continue;
        const Place at = place_of(a, b, s.first + i);
        const T *v = (const T *)a.v + at.page * a.v_page + at.in * a.v_entry + hk * a.v_head;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (lane + 32 * e < a.head_dim) {
                const float x = to_f32(v[lane + 32 * e]);
                if (!isfinite(x)) o.v[e] += x;
            }
    }
    return o;
}

// Writes a row from its sums: out = o / l, lse = (m + log2 l) ln 2.
template <class T>
__device__ __forceinline__ void store_row(const Attn &A, int64_t b, int t, int h, float m, float l, const float (&o)[8])
{
    const dbs_attention_args &a = A.a;
    const int lane = threadIdx.x & 31;
    T *out = (T *)a.out + b * a.o_batch + t * a.o_token + h * a.o_head;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (lane + 32 * e < a.head_dim) out[lane + 32 * e] = from_f32<T>(l == 0.f ? 0.f : o[e] / l);
    if (a.lse && lane == 0) a.lse[(b * a.tokens + t) * a.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

constexpr int ROW_NT = 128;

// Any head size and alignment: one block per query row, its warps take every
// fourth entry, a lane every 32nd value.  Every row reads the cache again, from L2
// (one token, 32 heads, 2001 entries: 426 us; k_attn_few 10).
template <class T>
__global__ void __launch_bounds__(ROW_NT) k_attn_rows(Attn A)
{
    const dbs_attention_args &a = A.a;
    constexpr int W = ROW_NT / 32;
    __shared__ float s_m[W], s_l[W], s_o[W][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t rows = a.batch * a.tokens * a.q_heads;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int h = (int)(r % a.q_heads);
        const int64_t bt = r / a.q_heads, b = bt / a.tokens;
        const int t = (int)(bt % a.tokens);
        float o[8], m, l;
        row_by_warp<T>(A, b, t, h, warp, W, m, l, o);
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) s_o[warp][lane + 32 * e] = o[e];
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
        __syncthreads();
        if (warp == 0) {
            float top = -INFINITY, sum = 0.f, f;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 0.f;
            for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w]);
            for (int w = 0; w < W; ++w) {
                // a maximum of -inf: nothing there, or a NaN that has to stay
                f = s_m[w] == -INFINITY ? (s_l[w] != s_l[w] ? 1.f : 0.f) : exp2f(s_m[w] - top);
                sum += f * s_l[w];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] += f == 0.f ? 0.f : f * s_o[w][lane + 32 * e];
            }
            store_row<T>(A, b, t, h, top, sum, o);
        }
    }
}

// ---- how the work is shared out ----
//
// A unit is one kv head of one sequence and up to `rows` of its query rows; its
// work is its tiles of `keys` entries (one at least), each weighing as many as
// the 128-row blocks that the unit fills (a count, not a time: see k_attn_many).  All units lie in one line, of which
// every block takes an equal, contiguous piece, whatever the lengths: a piece
// covers whole units and at most two in part (the first and the last).  Whole
// ones are written at once, parts go to the block's two slots of scratch and are
// joined by k_attn_join.
struct Share {
    int keys, rows, groups;    // entries of a tile; query rows of a unit; units of a kv head
    int heavy, last;           // weight of a tile: of a kv head's units but the last, of the last
    float *scratch;
    int4 *units;               // of every unit: the first block that works on it, its slot there, the number of blocks

    __host__ __device__ int per_head() const { return heavy * (groups - 1) + last; }
    // Blocks that get a piece: none of them shorter than a tile.
    __device__ int64_t blocks(int64_t total, int64_t grid) const
    {
        const int64_t most = total / (heavy > last ? heavy : last);
        return most < grid ? most : grid;
    }
};

__device__ __forceinline__ int tiles_of(const Share &S, const Seq &s)
{
    return s.kv <= S.keys ? 1 : (int)((uint32_t)(s.kv + S.keys - 1) / (uint32_t)S.keys);
}
// (32-bit divisions where they do)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
__device__ __forceinline__ int64_t piece(int64_t total, int64_t c, int64_t blocks) { return quotient(c * total, blocks); }
// The block whose piece holds position x.
__device__ __forceinline__ int64_t block_of(int64_t total, int64_t x, int64_t blocks) { return quotient((x + 1) * blocks - 1, total); }

// A slot of scratch: rows x head_dim sums, the rows' maxima and sums, and the
// mark of a V that is not finite.
__host__ __device__ __forceinline__ int64_t slot_floats(int rows, int head_dim) { return (int64_t)rows * (head_dim + 2) + 8; }
__device__ __forceinline__ float *slot_of(const Attn &A, const Share &S, int64_t block, int slot)
{
    return S.scratch + (block * 2 + slot) * slot_floats(S.rows, A.a.head_dim);
}

// A piece's part of one unit.
struct Segment {
    Seq s;
    int64_t b;
    int hk, group;             // kv head, group of its rows
    int j0, j1;                // entries
    int tiles;                 // 0: the piece ends within the unit's next tile, which the following block has
    bool whole;                // the unit's only part
    int slot;                  // of scratch, if not
    int64_t u0;                // the unit in the line, and its weight
    int weight;
};

// Lengths of the first sequences, kept in shared memory by a block.
constexpr int NEAR = 128;
struct Near {
    int kv[NEAR], tree[NEAR];
};

__device__ __forceinline__ Seq sequence(const Attn &A, const Near &near, int64_t b)
{
    if (b >= NEAR) return sequence(A, b);
    return {near.kv[b], near.kv[b] - near.tree[b], near.tree[b]};
}

// Walks a block's piece, unit by unit.
struct Walk {
    int64_t x, end, b, u0, first, total, blocks;
    int hk, group;
    __device__ __forceinline__ bool next(const Attn &A, const Share &S, const Near &near, Segment &g)
    {
        while (x < end) {
            g.s = sequence(A, near, b);
            const int n = tiles_of(S, g.s), w = group == S.groups - 1 ? S.last : S.heavy;
            const int64_t u1 = u0 + (int64_t)n * w, e = end < u1 ? end : u1;
            const int t0 = w == 1 ? (int)(x - u0) : (int)((x - u0 + w - 1) >> 1), t1 = w == 1 ? (int)(e - u0) : (int)((e - u0 + w - 1) >> 1);
            g.b = b;
            g.hk = hk;
            g.group = group;
            g.tiles = t1 - t0;
            g.whole = g.tiles == n;
            g.slot = first >= u0 ? 0 : 1;
            g.j0 = t0 * S.keys;
            g.j1 = (int64_t)t1 * S.keys < g.s.kv ? t1 * S.keys : g.s.kv;
            g.u0 = u0;
            g.weight = n * w;
            x = e;
            if (x == u1) {
                u0 = u1;
                if (++group == S.groups) {
                    group = 0;
                    if (++hk == A.a.kv_heads) {
                        hk = 0;
                        ++b;
                    }
                }
            }
            if (g.tiles > 0) return true;
        }
        return false;
    }
    // For the join, by the block with the unit's first tile: who works on it.
    __device__ __forceinline__ void record(const Attn &A, const Share &S, const Segment &g) const
    {
        if (g.j0 != 0) return;
        const int w = g.group == S.groups - 1 ? S.last : S.heavy;
        int64_t c1 = g.whole ? blockIdx.x : block_of(total, g.u0 + g.weight - 1, blocks);
        // the last block has no tile if its piece begins within the last one
        while (w > 1 && c1 > blockIdx.x && (piece(total, c1, blocks) - g.u0 + w - 1) / w >= g.weight / w) --c1;
        S.units[(g.b * A.a.kv_heads + g.hk) * S.groups + g.group] = make_int4((int)blockIdx.x, g.slot, (int)(c1 - blockIdx.x) + 1, 0);
    }
};

// Where this block's piece begins.  Up to NEAR sequences every warp finds out
// for itself from the lengths in shared memory, a few sequences a lane; of more
// the block adds up the lengths in turns.
template <int NT>
__device__ __forceinline__ Walk start(const Attn &A, const Share &S, int64_t *red, Near &near)
{
    const int64_t B = A.a.batch;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Walk w;
    for (int i = threadIdx.x; i < NEAR && i < B; i += NT) {
        const Seq s = sequence(A, i);
        near.kv[i] = s.kv;
        near.tree[i] = s.tree;
    }
    __syncthreads();
    const int64_t per = (int64_t)A.a.kv_heads * S.per_head();
    auto tiles = [&](int64_t i) { return i < B ? (int64_t)tiles_of(S, sequence(A, near, i)) * per : 0; };
    auto scan = [&](int64_t v) {                             // sums up to and with each lane
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(~0u, v, d);
            if (lane >= d) v += o;
        }
        return v;
    };
    int64_t at = 0;
    if (B <= NEAR) {
        constexpr int E = NEAR / 32;
        int64_t n[E], sum = 0;
#pragma unroll
        for (int k = 0; k < E; ++k) sum += n[k] = tiles(lane * E + k);
        int64_t upto = scan(sum);
        w.total = __shfl_sync(~0u, upto, 31);
        w.blocks = S.blocks(w.total, gridDim.x);
        w.x = blockIdx.x < w.blocks ? piece(w.total, blockIdx.x, w.blocks) : w.total;
        w.b = 0;
        if (w.x < w.total) {
            const int who = __ffs(__ballot_sync(~0u, w.x < upto)) - 1;
            upto -= sum;                                     // before this lane's
            int64_t mine = lane * E;
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (mine == lane * E + k && w.x >= upto + n[k]) {
                    upto += n[k];
                    ++mine;
                }
            at = __shfl_sync(~0u, upto, who);
            w.b = __shfl_sync(~0u, mine, who);
        }
    } else {
        int64_t sum = 0;
        for (int64_t i = threadIdx.x; i < B; i += NT) sum += tiles(i);
        sum = __shfl_sync(~0u, scan(sum), 31);
        if (lane == 0) red[warp] = sum;
        __syncthreads();
        w.total = 0;
        for (int k = 0; k < NT / 32; ++k) w.total += red[k];
        w.blocks = S.blocks(w.total, gridDim.x);
        w.x = blockIdx.x < w.blocks ? piece(w.total, blockIdx.x, w.blocks) : w.total;
        w.b = 0;
        // (every warp for itself, 32 sequences at a time)
        if (w.x < w.total)
            for (;; w.b += 32) {
                const int64_t n = tiles(w.b + lane), upto = scan(n), all = __shfl_sync(~0u, upto, 31);
                if (w.x < at + all) {
                    const int who = __ffs(__ballot_sync(~0u, w.x < at + upto)) - 1;
                    at += __shfl_sync(~0u, upto - n, who);
                    w.b += who;
                    break;
                }
                at += all;
            }
    }
    w.first = w.x;
    w.end = blockIdx.x < w.blocks ? piece(w.total, blockIdx.x + 1, w.blocks) : w.x;
    if (w.x < w.end) {
        const int n = tiles_of(S, sequence(A, near, w.b));
        const int64_t head = (int64_t)n * S.per_head(), big = (int64_t)n * S.heavy;
        w.hk = (int)quotient(w.x - at, head);
        const int64_t rest = w.x - at - w.hk * head;
        w.group = S.groups == 1 ? 0 : (int)quotient(rest, big);
        if (w.group > S.groups - 1) w.group = S.groups - 1;
        w.u0 = at + w.hk * head + w.group * big;
    }
    return w;
}

constexpr int JOIN_NT = 128, JOIN_W = JOIN_NT / 32;

// Joins the parts of a unit that more than one block worked on; a row by `split`
// warps (all four of a block while there are few rows, else one).  A row's
// warps read the parts' maxima and sums (a lane a part), each adds up its share
// of the parts' outputs, several loads at a time, and the warps' sums are added
// in order.  Bound by the latency of that chain.
template <class T>
__global__ void __launch_bounds__(JOIN_NT) k_attn_join(Attn A, Share S, int rows, int split)
{
    const dbs_attention_args &a = A.a;
    __shared__ float s_o[JOIN_W][256];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t per = (uint32_t)a.kv_heads * S.groups;
    const uint32_t b = blockIdx.x / per, u = blockIdx.x % per;
    const int hk = (int)(u / S.groups), group = (int)(u % S.groups);
    const int4 unit = S.units[blockIdx.x];
    const Seq s = sequence(A, b);
    const int parts = unit.z, mine = warp % split;
    if (parts == 1) return;
    const int64_t size = slot_floats(S.rows, a.head_dim), stat = (int64_t)S.rows * a.head_dim;
    // the unit may be the second of its first block, and is the first of the others
    const float *p0 = slot_of(A, S, unit.x, unit.y), *rest = slot_of(A, S, unit.x, 0);
    for (int r0 = blockIdx.y * (JOIN_W / split); r0 < rows; r0 += gridDim.y * (JOIN_W / split)) {
        const int r = r0 + warp / split;
        const Row row = row_of(A, hk, (int64_t)group * S.rows + r);
        const bool here = r < rows && row.inside;
        float top = -INFINITY, sum = 0.f, o[8] = {};
        bool odd = false;
        if (here && row.t < s.tree) {
            for (int base = 0; base < parts; base += 32) {
                float m = -INFINITY, l = 0.f;
                if (base + lane < parts) {
                    const float *st = (base + lane ? rest + 2 * size * (base + lane) : p0) + stat;
                    m = st[r];
                    l = st[S.rows + r];
                    odd |= st[2 * S.rows] != 0.f;
                }
                float now = fmaxf(top, m);
#pragma unroll
                for (int d = 16; d; d >>= 1) now = fmaxf(now, __shfl_xor_sync(~0u, now, d));
                const float keep = top == -INFINITY ? 0.f : exp2f(top - now);
                top = now;
                const float f = m == -INFINITY ? 0.f : exp2f(m - top);
                l = l != l ? l : f * l;
#pragma unroll
                for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
                sum = sum * keep + l;
                const int now_parts = parts - base < 32 ? parts - base : 32;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] *= keep;
                for (int i = mine; i < now_parts; i += 4 * split) {
                    float v[4][8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = base + (i + k * split < now_parts ? i + k * split : i);
                        const float *p = (c ? rest + 2 * size * c : p0) + (int64_t)r * a.head_dim;
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[k][e] = lane + 32 * e < a.head_dim ? p[lane + 32 * e] : 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float fi = __shfl_sync(~0u, f, (i + k * split) & 31);
                        if (i + k * split >= now_parts) break;
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] += fi == 0.f ? 0.f : fi * v[k][e];
                    }
                }
            }
        }
        if (split > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (lane + 32 * e < a.head_dim) s_o[warp][lane + 32 * e] = o[e];
            __syncthreads();
            if (mine == 0)
                for (int k = 1; k < split; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (lane + 32 * e < a.head_dim) o[e] += s_o[warp + k][lane + 32 * e];
        }
        if (!here || mine != 0) continue;
        if (__any_sync(~0u, odd)) {
            Eight q;
#pragma unroll
            for (int e = 0; e < 8; ++e) q.v[e] = o[e];
            q = add_odd<T>(A, b, row.t, hk, q);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = q.v[e];
        }
        store_row<T>(A, b, row.t, row.h, top, sum, o);
    }
}

// ---- few rows: every warp streams its own entries ----

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
template <class T> __device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <> __device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <> __device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int FEW_NT = 128, FEW_W = FEW_NT / 32;
constexpr int FEW_ROWS = 16;               // one matrix instruction's rows
constexpr int FEW_STEP = 16;               // entries of a stage of a warp
constexpr int FEW_KEYS = FEW_W * FEW_STEP;
constexpr int FEW_STAGES = 3;
constexpr int FEW_SPLIT = 16;      // blocks of a cluster, at most

template <int DP> constexpr int few_smem() { return FEW_W * FEW_STAGES * 2 * FEW_STEP * DP * 2; }

// 16 query rows against a piece of the cache.  The four warps take turns of 16
// entries, each with its own ring of K and V stages, running maximum, sum and
// output, so no block-wide wait runs in the loop; they are joined at the end of
// a unit.  A maximum is replaced only when it grew by more than 2^8, so the
// output is hardly ever rescaled (probabilities stay below 2^8, exact in
// proportion).
//
// Two ways to share out the work: pieces of the line (CLUSTER = false), or, for few
// units, the blocks of a cluster for each, which take equal parts of its entries and
// join them through their shared memory, in the same launch.
template <class T, int DP, bool CLUSTER>
__global__ void __launch_bounds__(FEW_NT) k_attn_few(Attn A, Share S, int split)
{
    const dbs_attention_args &a = A.a;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ int64_t red[FEW_W];
    __shared__ Near near;
    __shared__ float s_m[FEW_W][FEW_ROWS], s_l[FEW_W][FEW_ROWS];
    __shared__ int s_odd[FEW_W];
    __shared__ float j_m[CLUSTER ? FEW_ROWS : 1], j_l[CLUSTER ? FEW_ROWS : 1];                 // of the block's rows, for the cluster
    __shared__ int j_odd;
    constexpr int RB = DP * 2, CH = DP / 8, HALF = FEW_STEP * RB;   // bytes and 16-byte chunks of an entry; of a stage's K
    constexpr int KK = DP / 16, NN = DP / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q4 = lane & 3;
    unsigned char *mine = ring + warp * (FEW_STAGES * 2 * HALF);
    // a row's joined sums, in the ring of the warp that joins it, behind that warp's own
    auto joined = [&](int r) { return r % FEW_W * (FEW_STAGES * 2 * HALF) + (FEW_ROWS + r / FEW_W) * DP * 4; };
    static_assert((FEW_ROWS + FEW_ROWS / FEW_W) * DP * 4 <= FEW_STAGES * 2 * HALF, "room behind a warp's sums");
    const uint32_t base = smem_addr(mine);
    const int chunks = a.head_dim / 8;
    const int rank = CLUSTER ? (int)(blockIdx.x % split) : 0;
    Walk walk;
    Segment seg;
    if constexpr (CLUSTER) {
        const uint32_t unit = blockIdx.x / split, per = (uint32_t)a.kv_heads * S.groups, u = unit % per;
        seg.b = unit / per;
        seg.hk = (int)(u / S.groups);
        seg.group = (int)(u % S.groups);
        seg.s = sequence(A, seg.b);
        const int n = tiles_of(S, seg.s);
        seg.j0 = (int)((int64_t)n * rank / split) * S.keys;
        seg.j1 = (int)((int64_t)n * (rank + 1) / split) * S.keys;
        seg.j1 = seg.j1 < seg.s.kv ? seg.j1 : seg.s.kv;
        seg.whole = false;
    } else {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the join waits for this grid's end)
        walk = start<FEW_NT>(A, S, red, near);
    }
    {
        while (CLUSTER || walk.next(A, S, near, seg)) {
            if (!CLUSTER && threadIdx.x == 0) walk.record(A, S, seg);
            const Seq &s = seg.s;
            const int64_t b = seg.b;
            const int hk = seg.hk, j0 = seg.j0, j1 = seg.j1;
            const int64_t R0 = (int64_t)seg.group * FEW_ROWS;
            const int steps = j1 > j0 + warp * FEW_STEP ? (j1 - j0 - warp * FEW_STEP + FEW_KEYS - 1) / FEW_KEYS : 0;

            // stage `i` of this warp: lane l < 16 finds entry l, all lanes copy
            auto fetch = [&](int i) {
                if (i < steps) {
                    const int j = j0 + i * FEW_KEYS + warp * FEW_STEP + (lane & 15);
                    const bool in = j < j1;
                    const Place at_j = place_of(a, b, in ? j : j1 - 1);
                    const int64_t ok = at_j.page * a.k_page + at_j.in * a.k_entry, ov = at_j.page * a.v_page + at_j.in * a.v_entry;
                    const unsigned ins = __ballot_sync(~0u, in);
                    const T *k = (const T *)a.k + hk * a.k_head, *v = (const T *)a.v + hk * a.v_head;
                    const uint32_t st = base + (i % FEW_STAGES) * (2 * HALF);
#pragma unroll
                    for (int c0 = 0; c0 < FEW_STEP * CH; c0 += 32) {
                        const int row = (c0 + lane) / CH, c = (c0 + lane) % CH;
                        const int64_t rk = __shfl_sync(~0u, ok, row), rv = __shfl_sync(~0u, ov, row);
                        const bool take = (ins >> row & 1u) && c < chunks;
                        const uint32_t to = st + row * RB + ((c ^ (row & 7)) << 4);
                        cp16(to, take ? (const void *)(k + rk + c * 8) : (const void *)a.k, take);
                        cp16(to + HALF, take ? (const void *)(v + rv + c * 8) : (const void *)a.v, take);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
#pragma unroll
            for (int i = 0; i < FEW_STAGES - 1; ++i) fetch(i);

            // query rows g and g + 8 as matrix fragments
            const Row ra = row_of(A, hk, R0 + g), rb = row_of(A, hk, R0 + g + 8);
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
            bool odd = false;
            float o[NN][4], ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
#pragma unroll
            for (int i = 0; i < NN; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

            for (int i = 0; i < steps; ++i) {
                fetch(i + FEW_STAGES - 1);
                asm volatile("cp.async.wait_group %0;" ::"n"(FEW_STAGES - 1) : "memory");
                __syncwarp();
                const uint32_t st = base + (i % FEW_STAGES) * (2 * HALF);
                float sc[2][4] = {};
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    // matrices: entries 0-7 and 8-15, halves of 16 columns
                    uint32_t r[4];
                    const int row = (lane & 7) + ((lane >> 4) << 3), c = 2 * k + ((lane >> 3) & 1);
                    ldsm4(r, st + row * RB + ((c ^ (row & 7)) << 4));
                    mma16816<T>(sc[0], qf[k], r[0], r[1]);
                    mma16816<T>(sc[1], qf[k], r[2], r[3]);
                }
                const int j = j0 + i * FEW_KEYS + warp * FEW_STEP;
                uint32_t va = ~0u, vb = ~0u;
                if (j + FEW_STEP > s.first) {
                    bool found = false;
#pragma unroll
                    for (int c0 = lane; c0 < FEW_STEP * CH; c0 += 32) {
                        uint4 *w = (uint4 *)(mine + (i % FEW_STAGES) * (2 * HALF) + HALF + (c0 << 4));
                        uint4 x = *w;
                        const bool any = (int)clear_odd<T>(x.x) | (int)clear_odd<T>(x.y) | (int)clear_odd<T>(x.z) | (int)clear_odd<T>(x.w);
                        if (any && j + c0 / CH >= s.first) {
                            *w = x;
                            found = true;
                        }
                    }
                    odd |= __any_sync(~0u, found);
                    va = sees32(A, b, ra.t, s.tree, j - s.first);
                    vb = sees32(A, b, rb.t, s.tree, j - s.first);
                }
                float ta = -INFINITY, tb = -INFINITY;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int bit = 8 * h + 2 * q4 + e;
                        sc[h][e] = va >> bit & 1u ? sc[h][e] * A.scale_log2 : -INFINITY;
                        sc[h][e + 2] = vb >> bit & 1u ? sc[h][e + 2] * A.scale_log2 : -INFINITY;
                        ta = fmaxf(ta, sc[h][e]);
                        tb = fmaxf(tb, sc[h][e + 2]);
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
                // sums take them as they are); two pieces of each would cost a second product.  Error against 64
                // bits, relative: one token of 2001 entries, bf16, 0.0022 (0.0016 with fp32 probabilities)
                const uint32_t pf[4] = {pack2<T>(sc[0][0], sc[0][1]), pack2<T>(sc[0][2], sc[0][3]), pack2<T>(sc[1][0], sc[1][1]),
                                        pack2<T>(sc[1][2], sc[1][3])};
#pragma unroll
                for (int k = 0; k < NN; k += 2) {
                    // matrices: entries 0-7 and 8-15 of two groups of 8 columns
                    uint32_t r[4];
                    const int row = (lane & 7) + (((lane >> 3) & 1) << 3), c = k + (lane >> 4);
                    ldsm4t(r, st + HALF + row * RB + ((c ^ (row & 7)) << 4));
                    mma16816<T>(o[k], pf, r[0], r[1]);
                    mma16816<T>(o[k + 1], pf, r[2], r[3]);
                }
                __syncwarp();
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
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
            if (lane == 0) s_odd[warp] = odd;
            if (q4 == 0) {
                s_m[warp][g] = ma;
                s_l[warp][g] = la;
                s_m[warp][g + 8] = mb;
                s_l[warp][g + 8] = lb;
            }
            __syncthreads();
            const bool whole = seg.whole;
            odd = (s_odd[0] | s_odd[1] | s_odd[2] | s_odd[3]) != 0;
            float *part = CLUSTER ? nullptr : slot_of(A, S, blockIdx.x, seg.slot);
            for (int r = warp; r < FEW_ROWS; r += FEW_W) {
                const Row row = row_of(A, hk, R0 + r);
                if (!row.inside) break;
                float top = -INFINITY, sum = 0.f, oo[8] = {};
#pragma unroll
                for (int w = 0; w < FEW_W; ++w) top = fmaxf(top, s_m[w][r]);
#pragma unroll
                for (int w = 0; w < FEW_W; ++w) {
                    const float f = s_m[w][r] == -INFINITY ? (s_l[w][r] != s_l[w][r] ? 1.f : 0.f) : exp2f(s_m[w][r] - top);
                    const float *po = (const float *)(ring + w * (FEW_STAGES * 2 * HALF)) + r * DP;
                    sum += f * s_l[w][r];
#pragma unroll
                    for (int e = 0; e < DP / 32; ++e) oo[e] += f == 0.f ? 0.f : f * po[lane + 32 * e];
                }
                if (CLUSTER) {
#pragma unroll
                    for (int e = 0; e < DP / 32; ++e) ((float *)(ring + joined(r)))[lane + 32 * e] = oo[e];
                    if (lane == 0) {
                        j_m[r] = top;
                        j_l[r] = sum;
                    }
                } else if (whole) {
                    if (row.t >= s.tree) {
                        sum = 0.f;
                    } else if (odd) {
                        Eight w;
#pragma unroll
                        for (int e = 0; e < 8; ++e) w.v[e] = oo[e];
                        w = add_odd<T>(A, b, row.t, hk, w);
#pragma unroll
                        for (int e = 0; e < 8; ++e) oo[e] = w.v[e];
                    }
                    store_row<T>(A, b, row.t, row.h, top, sum, oo);
                } else {
#pragma unroll
                    for (int e = 0; e < DP / 32; ++e)
                        if (lane + 32 * e < a.head_dim) part[(int64_t)r * a.head_dim + lane + 32 * e] = oo[e];
                    if (lane == 0) {
                        part[(int64_t)FEW_ROWS * a.head_dim + r] = top;
                        part[(int64_t)FEW_ROWS * a.head_dim + FEW_ROWS + r] = sum;
                        if (r == 0) part[(int64_t)FEW_ROWS * a.head_dim + 2 * FEW_ROWS] = odd;
                    }
                }
            }
            if constexpr (CLUSTER) {
                if (threadIdx.x == 0) j_odd = odd;
                asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
                // 32 columns of a row for each of the cluster's warps in turn
                auto from = [&](const void *p, int block) {
                    uint32_t at;
                    float v;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(block));
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
                    return v;
                };
                const int64_t left = (int64_t)a.tokens * A.group - R0;
                const int rows = (int)(left < FEW_ROWS ? left : FEW_ROWS);
                for (int i = rank * FEW_W + warp; i < rows * (DP / 32); i += split * FEW_W) {
                    const int r = i / (DP / 32), e0 = i % (DP / 32);
                    const Row row = row_of(A, hk, R0 + r);
                    const bool in = lane < split;
                    const float m = in ? from(j_m + r, lane) : -INFINITY;
                    float l = in ? from(j_l + r, lane) : 0.f;
                    const bool found = in && __float_as_int(from(&j_odd, lane)) != 0;
                    float v[FEW_SPLIT], o = 0.f, top = m;
#pragma unroll
                    for (int k = 0; k < FEW_SPLIT; ++k) v[k] = k < split ? from((const float *)(ring + joined(r)) + lane + 32 * e0, k) : 0.f;
#pragma unroll
                    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                    const float f = m == -INFINITY ? (l != l ? 1.f : 0.f) : exp2f(m - top);
                    l = f == 0.f ? 0.f : f * l;
#pragma unroll
                    for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
#pragma unroll
                    for (int k = 0; k < FEW_SPLIT; ++k) {
                        const float fk = __shfl_sync(~0u, f, k);
                        o += fk == 0.f ? 0.f : fk * v[k];
                    }
                    if (row.t >= s.tree) {
                        l = 0.f;
                    } else if (__any_sync(~0u, found)) {
                        Eight w;
#pragma unroll
                        for (int e = 0; e < 8; ++e) w.v[e] = e == e0 ? o : 0.f;
                        w = add_odd<T>(A, b, row.t, hk, w);
#pragma unroll
                        for (int e = 0; e < 8; ++e) o = e == e0 ? w.v[e] : o;
                    }
                    if (lane + 32 * e0 < a.head_dim) ((T *)a.out + b * a.o_batch + row.t * a.o_token + row.h * a.o_head)[lane + 32 * e0] = from_f32<T>(l == 0.f ? 0.f : o / l);
                    if (a.lse && e0 == 0 && lane == 0) a.lse[(b * a.tokens + row.t) * a.q_heads + row.h] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
                }
                // (no block ends while another one reads its shared memory)
                asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
                break;
            }
            __syncthreads();       // the rings are free again
        }
    }
}

// ---- many rows: tcgen05 ----
//
// 128 query rows against tiles of entries on the fifth-generation tensor cores:
// S = Q K^T and O += P V with both accumulators in tensor memory (a row per
// lane), Q, K and V in shared memory in the 128-byte swizzle (K row by row, V
// as it lies, its entries as the contraction's dimension), and P rounded to the
// caches' type, as the matrix instruction has one type for both operands (error against
// 64 bits: trees of 48, f16, 0.00029, with fp32 probabilities 0.00021).  Warps have roles: two fetch K and V, two load Q, one for each 128
// rows issues the matrix instructions, two look through the drafted part of V, and
// four for each 128 rows do the softmax, a thread a row.  S has two buffers, so the
// scores of the next tile of entries are made under the softmax of one.
// With one row tile P is written over S.  With two (TILES = 2), which share a tile
// of K and V, tensor memory holds scores of 64 entries for each, P goes to shared
// memory, so that scores wait for no product, and the warps that fetch and issue
// leave registers to those of the softmax, which then read S once.
//
// K and V come by tiled copies (TMA) of boxes of as many entries as divide a
// page, eight at least; caches whose pages do not split into eights come by
// 16-byte asynchronous copies, which reach about half of the memory's rate (an SM's
// copies in flight are the limit).
//
// 16 trees of 12 tokens, 8 kv heads, 128 MB of caches: 54 us.  A tile of 128 entries
// takes 1.15 us, less than its copy at the memory's rate; what is lost is the start
// (9 us until the first scores, of which 4 the first copies) and 5 us for each of a
// block's two or three units (masked tile, last product, output, first scores).
// 4 trees of 48 tokens over 32768 entries, 384 rows to a kv head: 169 us, 32% of the
// tensor cores' rate.  Two row tiles take 1.1 us for 64 entries where a block has 862
// such tiles (2 x 1024 tokens over 32768 entries, 32/8 heads: 950 us, 61%); the products
// alone would take 0.67: the softmax's own chain (scores, maximum, powers, sum, stores)
// bounds it.  With 108 a block the start, the units' ends and the join cost a third
// (1024 tokens over 8192 entries: 34%).  A lone row tile, the rest of a kv head's rows,
// has the same chain: 384 rows (48 tokens, 32/4 heads) take longer than 512 (L2 flushed:
// 185 us and 168), although the line gives it half of a pair's weight.  With P over S and
// tiles of 128 entries 173 us; P over S and tiles of 64: 177; one warp issuing for both
// row tiles: 179.  A share of the powers of two by polynomial made it slower (186 us and
// more).
//
// Every wait on a barrier has a limit; a block whose wait runs out stops, leaves NaN in
// the rows of all units, or parts of units, that it had not finished, and says so.

template <int DP, int TILES> struct Many {
    static constexpr int KEYS = DP == 256 || TILES == 2 ? 64 : 128;
    static constexpr int STAGES = DP == 256 ? 2 : TILES == 2 ? 4 : 3;       // of K, and of V
    static constexpr int SB = 2;                                          // score buffers of a row tile
    static constexpr int SUBQ = 128 * 128, SUBK = KEYS * 128;             // 64 columns of a tile, in bytes
    static constexpr bool PS = TILES == 2;                                // P in shared memory, not over S
    static constexpr int Q = DP / 64 * SUBQ, KV = DP / 64 * SUBK, P = PS ? 128 * KEYS * 2 : 0;
    static constexpr int NT = 32 * (4 * TILES + 4 + TILES + 2);
    static constexpr int FETCH = 4 * TILES, LOAD = FETCH + 2, ISSUE = FETCH + 4, MEND = ISSUE + TILES;   // first warps of the roles
    // registers of a thread at launch (TILES = 2), and once the warps that fetch and
    // issue have left some to those of the softmax, two fours of warps each
    static constexpr int REGS = 128, FEW = 112, MANY = 2 * REGS - FEW;
    static constexpr int S_COL = 0, O_COL = TILES * SB * KEYS;
    static constexpr int SMEM = TILES * (Q + P) + STAGES * 2 * KV + 1024;
};
static_assert(!Many<128, 2>::PS || Many<128, 2>::KEYS == 64, "a row of P is a row of the swizzle");
static_assert(Many<128, 2>::O_COL + 2 * 128 <= 512 && Many<256, 1>::O_COL + 256 <= 512, "tensor memory");

// 32 bytes, a whole sector, at once.
__device__ __forceinline__ void store32(void *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f, uint32_t g, uint32_t h)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h) : "memory");
}
// (to 2 units of the last place, and 0 below 2^-126: far below the 16 bits that P keeps)
__device__ __forceinline__ float pow2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Tensor maps of K and V: [pages, entries, heads, head_dim], boxes of 64 columns
// of one head of `box` entries.
struct Maps {
    CUtensorMap k, v;
    int box;
};

__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap *map, int d, int head, int entry, int page, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
                 "l"(map), "r"(bar), "r"(d), "r"(head), "r"(entry), "r"(page) : "memory");
}
// After a wait ran out, for the units that are left of a block's piece: who works on
// them, for the join, by one warp; and NaN in their rows, or, of a part, sums that the
// join makes NaN of, a row by each softmax thread (row `row` of row tile `r`).  (The first is
// inlined: the issuing warps have given registers away, a call might need them.)
__device__ __forceinline__ void record_rest(const Attn &A, const Share &S, const Near &near, Walk walk)
{
    Segment seg;
    while (walk.next(A, S, near, seg))
        if ((threadIdx.x & 31) == 0) walk.record(A, S, seg);
}
template <class T, int TILES>
__device__ __noinline__ void leave_nan(const Attn &A, const Share &S, const Near &near, Walk walk, int r, int row)
{
    const dbs_attention_args &a = A.a;
    const float nan = nanf("");
    Segment seg;
    while (walk.next(A, S, near, seg)) {
        const int slot_row = r * 128 + row;
        const Row me = row_of(A, seg.hk, (int64_t)seg.group * (128 * TILES) + slot_row);
        if (!me.inside) continue;
        if (seg.whole) {
            T *out = (T *)a.out + seg.b * a.o_batch + me.t * a.o_token + me.h * a.o_head;
            for (int d = 0; d < a.head_dim; ++d) out[d] = from_f32<T>(nan);
            if (a.lse) a.lse[(seg.b * a.tokens + me.t) * a.q_heads + me.h] = nan;
        } else {
            float *st = slot_of(A, S, blockIdx.x, seg.slot) + (int64_t)S.rows * a.head_dim;
            st[slot_row] = -INFINITY;
            st[S.rows + slot_row] = nan;
            if (slot_row == 0) st[2 * S.rows] = 0.f;
        }
    }
}

template <class T, int DP, int TILES, bool BOXES>
__global__ void __launch_bounds__(Many<DP, TILES>::NT, 1) k_attn_many(Attn A, Share S, const __grid_constant__ Maps maps)
{
    using M = Many<DP, TILES>;
    constexpr int KEYS = M::KEYS, ST = M::STAGES, SB = M::SB, CH = DP / 8;
    const dbs_attention_args &a = A.a;
    extern __shared__ unsigned char raw[];
    __shared__ int64_t red[M::NT / 32];
    __shared__ Near near;
    __shared__ __align__(8) uint64_t bars[6 * ST + TILES * (SB + 5)];
    __shared__ uint32_t tmem_at;
    __shared__ int stop;
    __shared__ int odd_seg[8];                       // segments (their number + 1) whose V is not finite somewhere
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t sq = base, sk = base + TILES * M::Q, sv = sk + ST * M::KV, sp = sv + ST * M::KV;
    const uint32_t bar0 = smem_addr(bars);
    const uint32_t k_full = bar0, k_empty = k_full + 8 * ST, v_full = k_empty + 8 * ST, v_empty = v_full + 8 * ST;
    const uint32_t s_full = v_empty + 8 * ST, q_full = s_full + 8 * TILES * SB, p_ready = q_full + 8 * TILES, o_done = p_ready + 8 * TILES;
    const uint32_t last_bar = o_done + 8 * TILES, v_fixed = last_bar + 8 * TILES, v_odd = v_fixed + 8 * ST, q_empty = v_odd + 8 * ST;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");       // (the join waits for this grid's end)
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            bar_init(k_full + 8 * i, BOXES ? 1 : 32);
            bar_init(k_empty + 8 * i, TILES);
            bar_init(v_full + 8 * i, BOXES ? 1 : 32);
            bar_init(v_fixed + 8 * i, 64);
            bar_init(v_odd + 8 * i, 1);
            bar_init(v_empty + 8 * i, TILES);
        }
        for (int i = 0; i < TILES * SB; ++i) bar_init(s_full + 8 * i, 1);
        for (int i = 0; i < TILES; ++i) {
            bar_init(q_full + 8 * i, 64);
            bar_init(q_empty + 8 * i, 1);
            bar_init(p_ready + 8 * i, 128);
            bar_init(o_done + 8 * i, 1);
            bar_init(last_bar + 8 * i, 1);
        }
        stop = 0;
        for (int i = 0; i < 8; ++i) odd_seg[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == M::ISSUE) {
        tc_alloc(smem_addr(&tmem_at));
    }
    Walk walk = start<M::NT>(A, S, red, near);
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tmem_at;
    // row tiles in use of a unit
    const int G = a.q_heads / a.kv_heads;
    const int64_t all_rows = a.tokens * G;
    auto tiles_in = [&](const Segment &g) {
        const int64_t left = all_rows - (int64_t)g.group * (128 * TILES);
        return TILES == 1 || left <= 128 ? 1 : 2;
    };
    Segment seg;

    if (warp < M::FETCH) {
        // ---- softmax: a thread has a row ----
        more_registers<TILES == 2 ? M::MANY : 0>();
        const int r = warp >> 2, row = (warp & 3) * 32 + lane;             // row tile, row in it
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
        const uint32_t o_at = tmem + lanes + M::O_COL + r * DP;
        int it = 0, number = 0;                                            // tiles done; segments
        bool ok = true;
        while (ok && walk.next(A, S, near, seg)) {
            const int number_now = number++;
            if (r >= tiles_in(seg)) continue;                              // the unit has one row tile: the other's barriers rest
            const int64_t b = seg.b;
            const Seq s = seg.s;
            const Row me = row_of(A, seg.hk, (int64_t)seg.group * (128 * TILES) + r * 128 + row);
            const bool busy = __any_sync(~0u, me.inside);
            float m = -INFINITY, l = 0.f;
            for (int t = 0; t < seg.tiles; ++t, ++it) {
                const int buf = it & 1;
                ok = __all_sync(~0u, bar_wait(s_full + 8 * (r * SB + buf), it >> 1 & 1, &stop, A.waits.limit));
                if (!ok) break;
                tc_after();
                const uint32_t s_at = tmem + lanes + M::S_COL + (r * SB + buf) * KEYS;
                const int j0 = seg.j0 + t * KEYS;
                const bool masked = j0 + KEYS > s.first;
                bool settled = t == 0;                                     // the product before this one is known to be in O
                if (busy) {
                    // 64 entries at a time; of more, read twice: first for the maximum, then for P
                    // (loops kept rolled: the roles share the instruction cache)
                    auto load = [&](float (&v)[64], int c) {
                        tc_ld(v, s_at + 64 * c);
                        if (masked) {
                            const uint32_t lo = sees32(A, b, me.t, s.tree, j0 + 64 * c - s.first);
                            const uint32_t hi = sees32(A, b, me.t, s.tree, j0 + 64 * c + 32 - s.first);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                v[e] = lo >> e & 1u ? v[e] : -INFINITY;
                                v[e + 32] = hi >> e & 1u ? v[e + 32] : -INFINITY;
                            }
                        }
                    };
                    float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    float v[64];
#pragma unroll 1
                    for (int c = 0; c < KEYS / 64; ++c) {
                        load(v, c);
#pragma unroll
                        for (int e = 0; e < 64; ++e) t4[e & 3] = fmaxf(t4[e & 3], v[e]);
                    }
                    const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * A.scale_log2;      // (scale > 0 here)
                    // replace the maximum only when it grew by more than 2^8
                    const bool grew = top > m + 8.f || (m == -INFINITY && top > m);
                    if (__any_sync(~0u, grew)) {
                        const float f = grew ? (m == -INFINITY ? 0.f : exp2f(m - top)) : 1.f;
                        if (grew) m = top;
                        l *= f;
                        if (t > 0) {
                            // the output so far, once the product before this one is in it
                            ok = __all_sync(~0u, bar_wait(o_done + 8 * r, (it - 1) & 1, &stop, A.waits.limit));
                            if (!ok) break;
                            settled = true;
                            tc_after();
#pragma unroll 1
                            for (int c = 0; c < DP / 32; ++c) {
                                float o[32];
                                uint32_t w[32];
                                tc_ld(o, o_at + 32 * c);
#pragma unroll
                                for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * f);
                                tc_st(o_at + 32 * c, w);
                            }
                            tc_wait_st();
                        }
                    }
                    const float shift = m == -INFINITY ? 0.f : m;
                    if (M::PS && !settled) {
                        // P's place is free once the product before this one is done
                        ok = __all_sync(~0u, bar_wait(o_done + 8 * r, (it - 1) & 1, &stop, A.waits.limit));
                        if (!ok) break;
                        settled = true;
                    }
                    float l4[4] = {l, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int c = 0; c < KEYS / 64; ++c) {
                        uint32_t w[32];
                        if (KEYS > 64) load(v, c);
#pragma unroll
                        for (int e = 0; e < 64; ++e) {
                            v[e] = pow2(fmaf(v[e], A.scale_log2, -shift));
                            l4[e & 3] += v[e];
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e) w[e] = pack2<T>(v[2 * e], v[2 * e + 1]);
                        if constexpr (M::PS) {
                            const uint32_t at = sp + r * M::P + row * 128;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + ((e ^ (row & 7)) << 4)), "r"(w[4 * e]), "r"(w[4 * e + 1]),
                                             "r"(w[4 * e + 2]), "r"(w[4 * e + 3]) : "memory");
                        } else {
                            tc_st(s_at + 32 * c, w);
                        }
                    }
                    l = (l4[0] + l4[1]) + (l4[2] + l4[3]);
                    if constexpr (M::PS) async_fence();
                    else tc_wait_st();
                }
                // (every phase of o_done is waited for while the next cannot end)
                if (!settled) ok = __all_sync(~0u, bar_wait(o_done + 8 * r, (it - 1) & 1, &stop, A.waits.limit));
                if (!ok) break;
                tc_before();
                bar_arrive(p_ready + 8 * r);
            }
            // the unit's (or the part's) output
            if (ok) ok = __all_sync(~0u, bar_wait(o_done + 8 * r, (it - 1) & 1, &stop, A.waits.limit));
            tc_after();
            const bool odd = ok && *(volatile int *)&odd_seg[number_now & 7] == number_now + 1;
            if (!busy) continue;
            float *part = slot_of(A, S, blockIdx.x, seg.slot);
            const int slot_row = r * 128 + row;
            const bool none = me.t >= s.tree || l == 0.f;
            const float fine = ok ? 1.f : nanf("");
            const float by = seg.whole ? (none ? 0.f : 1.f / l) * fine : fine;
            T *out = (T *)a.out + b * a.o_batch + me.t * a.o_token + me.h * a.o_head;
#pragma unroll 1
            for (int c = 0; c < DP / 32; ++c) {
                float v[32];
                tc_ld(v, o_at + 32 * c);
                if (!me.inside) continue;
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = seg.whole && none && ok ? 0.f : v[e] * by;
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    const int d = 32 * c + e;
                    if (d >= a.head_dim) break;
                    if (!seg.whole) {
                        store32(part + (int64_t)slot_row * a.head_dim + d, __float_as_uint(v[e]), __float_as_uint(v[e + 1]), __float_as_uint(v[e + 2]),
                                __float_as_uint(v[e + 3]), __float_as_uint(v[e + 4]), __float_as_uint(v[e + 5]), __float_as_uint(v[e + 6]),
                                __float_as_uint(v[e + 7]));
                    } else if (A.wide_out) {
                        *(uint4 *)(out + d) = make_uint4(pack2<T>(v[e], v[e + 1]), pack2<T>(v[e + 2], v[e + 3]), pack2<T>(v[e + 4], v[e + 5]),
                                                         pack2<T>(v[e + 6], v[e + 7]));
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) out[d + k] = from_f32<T>(v[e + k]);
                    }
                }
            }
            tc_before();
            if (me.inside) {
                if (!seg.whole) {
                    float *st = part + (int64_t)S.rows * a.head_dim;
                    st[slot_row] = m;
                    st[S.rows + slot_row] = l * fine;
                    if (slot_row == 0) st[2 * S.rows] = odd;
                } else if (a.lse) {
                    a.lse[(b * a.tokens + me.t) * a.q_heads + me.h] = !ok ? fine : none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                }
            }
            if (odd && seg.whole) {
                __syncwarp();
                for (int i = 0; i < 32; ++i) {
                    const Row other = row_of(A, seg.hk, (int64_t)seg.group * (128 * TILES) + r * 128 + (warp & 3) * 32 + i);
                    if (!other.inside || other.t >= s.tree) continue;
                    T *o = (T *)a.out + b * a.o_batch + other.t * a.o_token + other.h * a.o_head;
                    Eight w;
#pragma unroll
                    for (int e = 0; e < 8; ++e) w.v[e] = lane + 32 * e < a.head_dim ? to_f32(o[lane + 32 * e]) : 0.f;
                    w = add_odd<T>(A, b, other.t, seg.hk, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (lane + 32 * e < a.head_dim) o[lane + 32 * e] = from_f32<T>(w.v[e]);
                }
            }
        }
        if (!ok) leave_nan<T, TILES>(A, S, near, walk, r, row);
    } else if (fewer_registers<TILES == 2 ? M::FEW : 0>(), BOXES && warp < M::FETCH + 2) {
        // ---- fetch: one warp K, one V, a lane a box ----
        const bool is_v = warp > M::FETCH;
        const uint32_t store = is_v ? sv : sk, full = is_v ? v_full : k_full, empty = is_v ? v_empty : k_empty;
        const CUtensorMap *const map = is_v ? &maps.v : &maps.k;
        const int box = maps.box, boxes = KEYS / box;                      // (8 to 128 entries; 1 to 16 boxes)
        const uint32_t vain = vain_bytes(A.waits);
        int n = 0;
        bool ok = true;
        while (ok && walk.next(A, S, near, seg)) {
            Place at = {0, 0};
            auto find = [&](int t) {
                const int j = seg.j0 + t * KEYS + lane * box;
                if (lane < boxes && j < seg.j1) at = place_of(a, seg.b, j);
            };
            find(0);
            for (int t = 0; t < seg.tiles && ok; ++t, ++n) {
                const int st = n % ST, j = seg.j0 + t * KEYS;
                ok = __all_sync(~0u, bar_wait(empty + 8 * st, (n / ST + 1) & 1, &stop, A.waits.limit));   // the first round finds it free
                if (!ok) break;
                const bool mine = lane < boxes && j + lane * box < seg.j1;
                const int count = __popc(__ballot_sync(~0u, mine));
                if (lane == 0) bar_expect(full + 8 * st, (uint32_t)(count * box * 128 * (DP / 64)) + vain);
                __syncwarp();
                if (mine)
#pragma unroll
                    for (int c = 0; c < DP / 64; ++c)
                        box_load(store + st * M::KV + c * M::SUBK + lane * box * 128, map, 64 * c, seg.hk, (int)at.in, (int)at.page, full + 8 * st);
                __syncwarp();
                if (is_v && lane == 0 && j + KEYS > seg.s.first) bar_arrive(v_odd + 8 * st);      // a tile to look through
                if (t + 1 < seg.tiles) find(t + 1);
            }
        }
        // copies under way end before their memory is given back
        for (int i = n > ST ? n - ST : 0; i < n; ++i) {
            int last = 0;
            bar_wait(full + 8 * (i % ST), i / ST & 1, &last, A.waits.limit);
        }
    } else if (warp >= M::LOAD && warp < M::ISSUE) {
        // ---- Q ----
        const int p = tid - 32 * M::LOAD, c = p % CH, r0 = p / CH;
        constexpr int RS = 64 / CH;
        int units[TILES] = {};
        bool ok = true;
        while (ok && walk.next(A, S, near, seg)) {
            const int used = tiles_in(seg);
#pragma unroll
            for (int r = 0; r < TILES; ++r) {
                if (r >= used || !ok) continue;
                // rows past the call's are left as they are: a row's results depend on it alone
                const int64_t R0 = (int64_t)seg.group * (128 * TILES) + r * 128;
                const int rows = all_rows - R0 < 128 ? (int)(all_rows - R0) : 128;
                const T *q = (const T *)a.q + seg.b * a.q_batch + 8 * c;
                bool free = false;
#pragma unroll 1
                for (int i0 = 0; i0 < rows; i0 += 16 * RS) {
                    uint4 x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int to = i0 + i * RS + r0;
                        const Row row = row_of(A, seg.hk, R0 + to);
                        x[i] = make_uint4(0, 0, 0, 0);
                        if (to < rows && 8 * c < a.head_dim) x[i] = *(const uint4 *)(q + row.t * a.q_token + row.h * a.q_head);
                    }
                    if (!free) {
                        // free once the segment before has its scores
                        ok = __all_sync(~0u, bar_wait(q_empty + 8 * r, (units[r]++ + 1) & 1, &stop, A.waits.limit));
                        free = true;
                        if (!ok) break;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int to = i0 + i * RS + r0;
                        const uint32_t at = sq + r * M::Q + (c >> 3) * M::SUBQ + to * 128 + (((c & 7) ^ (to & 7)) << 4);
                        if (to < rows)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x[i].x), "r"(x[i].y), "r"(x[i].z), "r"(x[i].w) : "memory");
                    }
                }
                if (!ok) continue;                                         // (no queries came)
                async_fence();
                bar_arrive(q_full + 8 * r);
            }
        }
    } else if (warp >= M::MEND) {
        // ---- of the tiles with drafted entries: what lies behind the last entry of V
        // becomes 0, and so does what is not finite in drafted ones ----
        const int p = tid - 32 * M::MEND, c = p % CH, r0 = p / CH;
        constexpr int RS = 64 / CH;
        int n = 0, number = 0;
        uint32_t seen = 0;                                                 // parity of v_odd of a stage, a bit each
        bool ok = BOXES;                                                   // (else the fetching warps do it)
        while (ok && walk.next(A, S, near, seg)) {
            for (int t = 0; t < seg.tiles && ok; ++t, ++n) {
                const int j0 = seg.j0 + t * KEYS, st = n % ST;
                if (j0 + KEYS <= seg.s.first) continue;
                // (first that the stage's copies are this tile's, then that they have arrived)
                ok = __all_sync(~0u, bar_wait(v_odd + 8 * st, seen >> st & 1u, &stop, A.waits.limit));
                seen ^= 1u << st;
                if (ok) ok = __all_sync(~0u, bar_wait(v_full + 8 * st, n / ST & 1, &stop, A.waits.limit));
                if (!ok) break;
                bool found = false;
#pragma unroll 4
                for (int row = r0; row < KEYS; row += RS) {
                    const uint32_t at = sv + st * M::KV + (c >> 3) * M::SUBK + row * 128 + (((c & 7) ^ (row & 7)) << 4);
                    uint4 x;
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
                    const bool behind = j0 + row >= seg.s.kv;
                    const bool any = (int)clear_odd<T>(x.x) | (int)clear_odd<T>(x.y) | (int)clear_odd<T>(x.z) | (int)clear_odd<T>(x.w);
                    if (behind) x = make_uint4(0, 0, 0, 0);
                    if (behind || (any && j0 + row >= seg.s.first))
                        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
                    found |= any && !behind && j0 + row >= seg.s.first;
                }
                if (found) *(volatile int *)&odd_seg[number & 7] = number + 1;
                async_fence();
                bar_arrive(v_fixed + 8 * st);
            }
            ++number;
        }
    } else if (!BOXES && warp >= M::FETCH && warp < M::ISSUE) {
        // ---- fetch: one warp K, one V.  A lane finds one entry in 32, all copy.  Stages are filled as they come
        // free, and announced in order, as soon as they have arrived.
        constexpr int RS = 32 / CH, PL = KEYS / 32;                        // entries of one copy of all lanes; of a lane
        const bool is_v = warp > M::FETCH;
        const int chunks = a.head_dim / 8, c = lane % CH, r0 = lane / CH;
        const uint32_t sub = (c >> 3) * M::SUBK, store = (is_v ? sv : sk) + sub;
        const uint32_t full = is_v ? v_full : k_full, empty = is_v ? v_empty : k_empty;
        const int64_t st_page = is_v ? a.v_page : a.k_page, st_entry = is_v ? a.v_entry : a.k_entry, st_head = is_v ? a.v_head : a.k_head;
        const T *const src = (const T *)(is_v ? a.v : a.k) + c * 8;
        const bool vain = vain_bytes(A.waits) != 0;
        int n = 0, announced = 0, number = 0;                              // tiles fetched, announced; segments
        struct Mark { int first, j0, number; };
        Mark marks[ST];                                                    // of the tiles under way
#pragma unroll
        for (int i = 0; i < ST; ++i) marks[i] = {0, 0, 0};
        auto announce = [&]() {
            // all but the (n - announced - 1) newest copies have arrived
            if (n - announced == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
            else if (ST == 2 || n - announced == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else if (ST == 3 || n - announced == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
            else asm volatile("cp.async.wait_group 3;" ::: "memory");
            const int st = announced % ST;
            Mark m = marks[0];
#pragma unroll
            for (int i = 1; i < ST; ++i)
                if (st == i) m = marks[i];
            if (is_v && m.j0 + KEYS > m.first) {
                bool found = false;
#pragma unroll 4
                for (int i = 0; i < KEYS / RS; ++i) {
                    const int row = r0 + i * RS;
                    const uint32_t at = store + st * M::KV + row * 128 + (((c & 7) ^ (row & 7)) << 4);
                    uint4 x;
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
                    const bool any = (int)clear_odd<T>(x.x) | (int)clear_odd<T>(x.y) | (int)clear_odd<T>(x.z) | (int)clear_odd<T>(x.w);
                    if (any && m.j0 + row >= m.first) {
                        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
                        found = true;
                    }
                }
                if (found) *(volatile int *)&odd_seg[m.number & 7] = m.number + 1;
            }
            async_fence();
            if (!vain) bar_arrive(full + 8 * st);
            ++announced;
        };
        bool ok = true;
        while (ok && walk.next(A, S, near, seg)) {
            const T *const from = src + seg.hk * st_head;
            int64_t off[PL];                                               // of this lane's entries of the next tile
            unsigned in[PL];
            auto find = [&](int t) {
#pragma unroll
                for (int i = 0; i < PL; ++i) {
                    const int j = seg.j0 + t * KEYS + 32 * i + lane;
                    Place at = {0, 0};                                     // (a cache without entries has no place, and may have no page table)
                    if (j < seg.j1) at = place_of(a, seg.b, j);
                    in[i] = __ballot_sync(~0u, j < seg.j1);
                    off[i] = at.page * st_page + at.in * st_entry;
                }
            };
            find(0);
            for (int t = 0; t < seg.tiles && ok; ++t) {
                const int st = n % ST;
                const uint32_t parity = (n / ST + 1) & 1;                  // of the stage's release; the first round finds it free
                // what has been fetched is announced before this warp waits for a stage
                while (announced < n && !__all_sync(~0u, bar_test(empty + 8 * st, parity))) announce();
                ok = __all_sync(~0u, bar_wait(empty + 8 * st, parity, &stop, A.waits.limit));
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < ST; ++i)
                    if (st == i) marks[i] = {seg.s.first, seg.j0 + t * KEYS, number};
                const uint32_t to = store + st * M::KV;
#pragma unroll
                for (int i = 0; i < KEYS / RS; ++i) {
                    const int row = i * RS + lane / CH;
                    const int64_t o = __shfl_sync(~0u, off[i * RS / 32], row & 31);
                    const bool take = (in[i * RS / 32] >> (row & 31) & 1u) && c < chunks;
                    cp16(to + row * 128 + (((c & 7) ^ (row & 7)) << 4), take ? (const void *)(from + o) : a.q, take);   // (some address to read nothing from)
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                ++n;
                if (t + 1 < seg.tiles) find(t + 1);
            }
            ++number;
        }
        if (ok)
            while (announced < n) announce();
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp >= M::ISSUE && warp < M::MEND) {
        // ---- issue the products: a warp for each row tile ----
        const int r = warp - M::ISSUE;
        constexpr uint32_t FMT = __is_same(T, __nv_bfloat16) ? 1u : 0u;
        constexpr uint32_t DESC = 1u << 4 | FMT << 7 | FMT << 10 | (128u >> 4) << 24;
        constexpr uint32_t DESC_S = DESC | (uint32_t)(KEYS >> 3) << 17, DESC_O = DESC | 1u << 16 | (uint32_t)(DP >> 3) << 17;
        uint32_t fixes = 0;                                                // parity of the repairs of a stage, a bit each
        int n0 = 0, it = 0, units = 0;                                     // first tile; score tiles, segments
        bool ok = true;
        while (ok && walk.next(A, S, near, seg)) {
            if (r == 0 && lane == 0) walk.record(A, S, seg);
            // scores against tile t of the segment
            auto scores = [&](int t) {
                const int st = (n0 + t) % ST;
                if (ok) ok = __all_sync(~0u, bar_wait(k_full + 8 * st, (n0 + t) / ST & 1, &stop, A.waits.limit));
                // the scores' columns are free once the product that read P from them is done
                // (the next segment waits for the last one's: two phases of a barrier are
                // never told apart)
                // (with P elsewhere: once the softmax has read them, which the product before waited for)
                if (!M::PS && it > 0 && ok) ok = __all_sync(~0u, bar_wait(o_done + 8 * r, (it - (t > 0 ? SB : 1)) & 1, &stop, A.waits.limit));
                if (!ok) return;
                tc_after();
                const uint32_t d = __shfl_sync(~0u, tmem + M::S_COL + (r * SB + (it & 1)) * KEYS, 0);
                const uint32_t qa = desc_lo(sq + r * M::Q, 16), ka = desc_lo(sk + st * M::KV, 16);
                uint64_t qd[DP / 16], kd[DP / 16];
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    qd[k] = desc_of(qa + ((k >> 2) * M::SUBQ + (k & 3) * 32) / 16);
                    kd[k] = desc_of(ka + ((k >> 2) * M::SUBK + (k & 3) * 32) / 16);
                }
                if (elected()) {
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) tc_mma_ss(d, qd[k], kd[k], DESC_S, k > 0);
                    tc_commit(s_full + 8 * (r * SB + (it & 1)));
                    tc_commit(k_empty + 8 * st);
                    if (t == seg.tiles - 1) tc_commit(q_empty + 8 * r);
                }
                ++it;
                __syncwarp();
            };
            auto outputs = [&](int t) {
                const int st = (n0 + t) % ST, done = it - (t + 1 < seg.tiles ? 2 : 1);   // this tile's number
                if (ok) ok = __all_sync(~0u, bar_wait(v_full + 8 * st, (n0 + t) / ST & 1, &stop, A.waits.limit));
                if (BOXES && ok && seg.j0 + (t + 1) * KEYS > seg.s.first) {
                    ok = __all_sync(~0u, bar_wait(v_fixed + 8 * st, fixes >> st & 1u, &stop, A.waits.limit));
                    fixes ^= 1u << st;
                }
                if (ok) ok = __all_sync(~0u, bar_wait(p_ready + 8 * r, done & 1, &stop, A.waits.limit));
                if (!ok) return;
                tc_after();
                const uint32_t d = __shfl_sync(~0u, tmem + M::O_COL + r * DP, 0);
                const uint32_t pa = __shfl_sync(~0u, tmem + M::S_COL + (r * SB + (done & 1)) * KEYS, 0);
                const uint32_t va = desc_lo(sv + st * M::KV, M::SUBK), more = __shfl_sync(~0u, t, 0) > 0;
                const uint32_t pl = desc_lo(sp + r * M::P, 16);
                uint64_t vd[KEYS / 16], pd[KEYS / 16];
#pragma unroll
                for (int k = 0; k < KEYS / 16; ++k) {
                    vd[k] = desc_of(va + k * 2048 / 16);
                    pd[k] = desc_of(pl + k * 32 / 16);
                }
                if (elected()) {
#pragma unroll
                    for (int k = 0; k < KEYS / 16; ++k) {
                        if (M::PS) tc_mma_ss(d, pd[k], vd[k], DESC_O, k > 0 ? 1u : more);
                        else tc_mma_ts(d, pa + 8 * k, vd[k], DESC_O, k > 0 ? 1u : more);
                    }
                    tc_commit(o_done + 8 * r);
                    tc_commit(v_empty + 8 * st);
                }
                __syncwarp();
            };
            if (r < tiles_in(seg)) {
                ok = __all_sync(~0u, bar_wait(q_full + 8 * r, units++ & 1, &stop, A.waits.limit));
                if (ok) scores(0);
                for (int t = 0; t < seg.tiles && ok; ++t) {
                    if (t + 1 < seg.tiles) scores(t + 1);
                    if (ok) outputs(t);
                }
            } else {
                // the unit has one row tile: the stages are released as they come
                for (int t = 0; t < seg.tiles && ok; ++t) {
                    const int st = (n0 + t) % ST;
                    ok = __all_sync(~0u, bar_wait(k_full + 8 * st, (n0 + t) / ST & 1, &stop, A.waits.limit) && bar_wait(v_full + 8 * st, (n0 + t) / ST & 1, &stop, A.waits.limit));
                    if (!ok) break;
                    if (lane == 0) {
                        bar_arrive(k_empty + 8 * st);
                        bar_arrive(v_empty + 8 * st);
                    }
                    if (BOXES && seg.j0 + (t + 1) * KEYS > seg.s.first) fixes ^= 1u << st;
                }
            }
            n0 += seg.tiles;
        }
        if (!ok) {
            if (r == 0) record_rest(A, S, near, walk);
            // products under way end before their memory is given back
            if (lane == 0) tc_commit(last_bar + 8 * r);
            __syncwarp();
            int last = 0;
            bar_wait(last_bar + 8 * r, 0, &last, A.waits.limit);
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

// ---- host ----

// How a call runs: the kernel, its grid and its scratch.
struct Plan {
    bool rows, many;           // any alignment; 128 rows at a time
    int dp, blocks;
    int split;                 // blocks of a cluster for each unit of few rows; 0: pieces of the line
    Share share;
    int64_t slots, scratch;    // bytes of scratch: the slots, and all
};

bool aligned8(int64_t v) { return (v & 7) == 0; }

dbs_status plan_of(const dbs_attention_args &a, Plan &P)
{
    P = Plan{};
    const int64_t entries = a.max_pages * a.page_size, rows = a.tokens * (a.q_heads / a.kv_heads);
    // 16-byte copies of heads: every head starts on such a boundary
    P.rows = a.head_dim % 8 || !aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned8(a.q_batch) ||
             !aligned8(a.q_token) || !aligned8(a.q_head) || !aligned8(a.k_page) || !aligned8(a.k_entry) ||
             !aligned8(a.k_head) || !aligned8(a.v_page) || !aligned8(a.v_entry) || !aligned8(a.v_head);
    if (P.rows) return DBS_OK;
    const int sms = multiprocessors();
    if (sms == 0) return DBS_ERR_CUDA;
    P.dp = a.head_dim <= 64 ? 64 : a.head_dim <= 128 ? 128 : 256;
    // up to 16 rows of a kv head fit one instruction of k_attn_few, which reads
    // the cache once for each 16
    P.many = rows > FEW_ROWS && a.scale > 0;
    Share &S = P.share;
    int per_sm = P.dp == 64 ? 4 : P.dp == 128 ? 2 : 1;
    if (P.many) {
        const int tiles = P.dp == 256 || rows <= 128 ? 1 : 2;
        S.keys = P.dp == 256 || tiles == 2 ? 64 : 128;
        S.rows = 128 * tiles;
        S.heavy = tiles;
        per_sm = 1;
    } else {
        S.keys = FEW_KEYS;
        S.rows = FEW_ROWS;
        S.heavy = 1;
    }
    S.groups = (int)((rows + S.rows - 1) / S.rows);
    S.last = P.many ? (int)((rows - (int64_t)(S.groups - 1) * S.rows + 127) / 128) : 1;
    const int64_t most = a.batch * a.kv_heads * S.groups * (entries < S.keys ? 1 : (entries + S.keys - 1) / S.keys);
    P.blocks = (int)(most < sms * per_sm ? most : sms * per_sm);
    // Few units of few rows: a cluster for each, as large as all find room at once,
    // instead of a second launch that joins the line's pieces (one token, 8 kv heads:
    // 2000 entries 11 and 14 us, 8192 entries 17 and 20; four sequences of 2000: 14 and
    // 20).  Where a block would have 2048 entries or more the line's even pieces are
    // faster (32768 entries: 44 and 40 us).  Blocks that fill an SM make clusters of
    // sixteen hard to place (head_dim 256, 3000 entries: 24 us, of eight 19).
    const int64_t units = a.batch * a.kv_heads * S.groups;
    if (!P.many) {
        int c = 1;
        while (c < (per_sm == 1 ? 8 : FEW_SPLIT) && units * 2 * c <= sms * per_sm) c *= 2;
        if (c > 1 && entries < (int64_t)c * 2048) {
            P.split = c;
            P.blocks = (int)(units * c);
            return DBS_OK;
        }
    }
    P.slots = (int64_t)P.blocks * 2 * slot_floats(S.rows, a.head_dim) * 4;
    P.scratch = P.slots + a.batch * a.kv_heads * S.groups * (int64_t)sizeof(int4);
    return DBS_OK;
}

// Rows of a call's largest unit.
int64_t rows_of_unit(const Attn &A, const Plan &P)
{
    const int64_t rows = A.a.tokens * (A.a.q_heads / A.a.kv_heads);
    return rows < P.share.rows ? rows : P.share.rows;
}

// The joining kernel, started while the first one ends.
template <class T>
dbs_status launch_join(const Attn &A, const Plan &P, cudaStream_t s)
{
    // whole blocks for a row while all rows find room on the GPU at once (8 blocks
    // an SM), and no more blocks than that: each finds its unit's place anew
    const int64_t units = A.a.batch * A.a.kv_heads * P.share.groups, rows = rows_of_unit(A, P), room = (int64_t)multiprocessors() * 8;
    const int split = units * rows <= room ? JOIN_W : 1;
    const int64_t turns = (rows + JOIN_W / split - 1) / (JOIN_W / split), most = room / units > 0 ? room / units : 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)units, (unsigned)(turns < most ? turns : most));
    c.blockDim = JOIN_NT;
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, k_attn_join<T>, A, P.share, (int)rows, split) == cudaSuccess ? DBS_OK : (cudaGetLastError(), DBS_ERR_CUDA);
}

template <class T, int DP>
dbs_status launch_few(const Attn &A, const Plan &P, cudaStream_t s)
{
    static Once once, once_cluster;
    if (P.split) {
        if (!room_for(once_cluster, k_attn_few<T, DP, true>, few_smem<DP>(), true)) return DBS_ERR_CUDA;
        cudaLaunchConfig_t c{};
        c.gridDim = dim3((unsigned)P.blocks);
        c.blockDim = FEW_NT;
        c.dynamicSmemBytes = few_smem<DP>();
        c.stream = s;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = (unsigned)P.split;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        c.attrs = &at;
        c.numAttrs = 1;
        cudaLaunchKernelEx(&c, k_attn_few<T, DP, true>, A, P.share, P.split);
        return launched();
    }
    if (!room_for(once, k_attn_few<T, DP, false>, few_smem<DP>())) return DBS_ERR_CUDA;
    k_attn_few<T, DP, false><<<P.blocks, FEW_NT, few_smem<DP>(), s>>>(A, P.share, 0);
    const dbs_status st = launched();
    return st == DBS_OK ? launch_join<T>(A, P, s) : st;
}

// Boxes of the caches, or false where pages or strides do not allow them.
bool make_maps(const dbs_attention_args &a, int keys, Maps &M)
{
    const encode_tiled_fn encode = encode_tiled();
    if (!encode || a.page_size < 1 || a.pages < 1) return false;
    // a sequence's own page is one run of entries; pages of a table split into boxes
    M.box = keys;
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

template <class T, int DP, int TILES, bool BOXES>
dbs_status launch_kind(const Attn &A, const Plan &P, const Maps &maps, cudaStream_t s)
{
    using M = Many<DP, TILES>;
    static Once once;
    if (!room_for(once, k_attn_many<T, DP, TILES, BOXES>, M::SMEM, false, TILES == 2 ? M::REGS : 0)) return DBS_ERR_CUDA;
    k_attn_many<T, DP, TILES, BOXES><<<P.blocks, M::NT, M::SMEM, s>>>(A, P.share, maps);
    const dbs_status st = launched();
    return st == DBS_OK ? launch_join<T>(A, P, s) : st;
}

template <class T, int DP, int TILES>
dbs_status launch_many(const Attn &A, const Plan &P, cudaStream_t s)
{
    Maps maps{};
    return make_maps(A.a, P.share.keys, maps) ? launch_kind<T, DP, TILES, true>(A, P, maps, s) : launch_kind<T, DP, TILES, false>(A, P, maps, s);
}

template <class T>
dbs_status launch(const Attn &A, const Plan &P, cudaStream_t s)
{
    if (P.rows) {
        const int64_t rows = A.a.batch * A.a.tokens * A.a.q_heads;
        k_attn_rows<T><<<(unsigned)(rows < (1 << 30) ? rows : (1 << 30)), ROW_NT, 0, s>>>(A);
        return launched();
    }
    if (P.many) {
        if (P.dp == 256) return launch_many<T, 256, 1>(A, P, s);
        if (P.share.heavy == 1) return P.dp == 64 ? launch_many<T, 64, 1>(A, P, s) : launch_many<T, 128, 1>(A, P, s);
        return P.dp == 64 ? launch_many<T, 64, 2>(A, P, s) : launch_many<T, 128, 2>(A, P, s);
    }
    return P.dp == 64 ? launch_few<T, 64>(A, P, s) : P.dp == 128 ? launch_few<T, 128>(A, P, s) : launch_few<T, 256>(A, P, s);
}

bool args_ok(const dbs_attention_args *a)
{
    if (!a || (a->dtype != DBS_F16 && a->dtype != DBS_BF16) || a->head_dim < 1 || a->head_dim > 256 || a->kv_heads < 1 ||
        a->kv_heads > 65536 || a->q_heads < a->kv_heads || a->q_heads > 65536 || a->q_heads % a->kv_heads || a->batch < 0 ||
        a->batch >= (int64_t(1) << 24) || a->tokens < 0 || a->tokens > 1024 || a->pages < 0 || a->page_size < 0 ||
        a->max_pages < 0 || a->page_size >= (int64_t(1) << 31) || a->max_pages >= (int64_t(1) << 31) ||
        a->pages >= (int64_t(1) << 40) || !std::isfinite(a->scale))
        return false;
    if (a->batch == 0 || a->tokens == 0) return true;
    const int64_t entries = a->max_pages * a->page_size;
    if (entries > (int64_t(1) << 31) - 1024) return false;               // (an entry's number and a tile's end are ints)
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

}  // namespace

extern "C" {

dbs_status dbs_operators_check(void *stream)
{
    const dbs_status here = waits_since((cudaStream_t)stream), w4 = w4_waits_since((cudaStream_t)stream);
    return here == DBS_ERR_CUDA ? here : w4 != DBS_OK ? w4 : here;
}

dbs_status dbs_debug_operator_waits(int64_t limit_ns, int32_t block)
{
    if (limit_ns < 1 || limit_ns > 2000000000 || block < -2) return DBS_ERR_INVALID_ARG;
    wait_limit.store((uint32_t)limit_ns, std::memory_order_relaxed);
    wait_vain.store(block, std::memory_order_relaxed);
    return DBS_OK;
}

dbs_status dbs_tree_attention_scratch(const dbs_attention_args *a, int64_t *bytes)
{
    if (!bytes || !args_ok(a)) return DBS_ERR_INVALID_ARG;
    *bytes = 0;
    if (a->batch == 0 || a->tokens == 0) return DBS_OK;
    Plan P;
    const dbs_status st = plan_of(*a, P);
    if (st == DBS_OK) *bytes = P.scratch;
    return st;
}

dbs_status dbs_tree_attention(const dbs_attention_args *a, void *stream)
{
    if (!args_ok(a)) return DBS_ERR_INVALID_ARG;
    if (a->batch == 0 || a->tokens == 0) return DBS_OK;
    Plan P;
    const dbs_status st = plan_of(*a, P);
    if (st != DBS_OK) return st;
    if (P.scratch > 0 && (!a->scratch || (reinterpret_cast<uintptr_t>(a->scratch) & 31u) || a->scratch_bytes < P.scratch)) return DBS_ERR_INVALID_ARG;
    const bool wide_out = aligned16(a->out) && aligned8(a->o_batch) && aligned8(a->o_token) && aligned8(a->o_head);
    const Attn A{*a, a->scale * 1.4426950408889634f, (int)((a->tokens + 63) / 64), wide_out, a->q_heads / a->kv_heads, waits()};
    P.share.scratch = (float *)a->scratch;
    P.share.units = (int4 *)((char *)a->scratch + P.slots);
    return a->dtype == DBS_F16 ? launch<__half>(A, P, (cudaStream_t)stream) : launch<__nv_bfloat16>(A, P, (cudaStream_t)stream);
}

}  // extern "C"
