// Attention of drafted tokens over a (paged) cache (dbs_tree_attention,
// sm_103a): softmax over the entries a token sees, with the running maximum
// and sum held in fp32.
#include "ops_dev.h"

#include <cmath>

using namespace dbs::ops;

namespace {

struct Attn {
    dbs_attention_args a;
    float scale_log2;          // scale * log2(e): probabilities are powers of two
    int words;                 // 64-bit mask words per token
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
    const int G = A.a.q_heads / A.a.kv_heads;
    Row r;
    r.t = (int)(R / G);
    r.h = hk * G + (int)(R % G);
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
// fourth entry.
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
// A unit is one kv head of one sequence and up to `rows` of its query rows;
// its work is its tiles of `keys` entries (one at least).  All units' tiles lie
// in one line, of which every block takes an equal, contiguous piece, whatever
// the lengths: a piece covers whole units and at most two in part (the first
// and the last).  Whole ones are written at once, parts go to the block's two
// slots of scratch and are joined by k_attn_join.
struct Share {
    int keys, rows, groups;    // entries of a tile; query rows of a unit; units of a kv head
    float *scratch;
};

struct Line {
    int64_t total, at;         // tiles of all; tiles before sequence b
};

__device__ __forceinline__ int tiles_of(const Share &S, const Seq &s)
{
    return s.kv <= S.keys ? 1 : (int)((uint32_t)(s.kv + S.keys - 1) / (uint32_t)S.keys);
}
__device__ __forceinline__ int64_t tiles_of(const Attn &A, const Share &S, int64_t b) { return tiles_of(S, sequence(A, b)); }

// Sum of `v` over the block (every thread gets it); `red` holds a word per warp.
template <int NT>
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t *red)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < NT / 32; ++w) v += red[w];
    return v;
}

// Tiles before sequence `b`, and of all.
template <int NT>
__device__ Line line_at(const Attn &A, const Share &S, int64_t b, int64_t *red)
{
    const int64_t per = (int64_t)A.a.kv_heads * S.groups;
    Line L{0, 0};
    if (A.a.batch == 1) {
        L.total = tiles_of(A, S, 0) * per;
        return L;
    }
    int64_t all = 0, before = 0;
    for (int64_t i = threadIdx.x; i < A.a.batch; i += NT) {
        const int64_t n = tiles_of(A, S, i) * per;
        all += n;
        if (i < b) before += n;
    }
    L.total = block_sum<NT>(all, red);
    L.at = block_sum<NT>(before, red);
    return L;
}

// The sequence that holds tile x, and the tiles before it.
template <int NT>
__device__ int64_t sequence_of(const Attn &A, const Share &S, int64_t x, int64_t &at, int64_t *red)
{
    const int64_t per = (int64_t)A.a.kv_heads * S.groups;
    at = 0;
    if (A.a.batch == 1) return 0;
    __shared__ int64_t hit, hit_at;
    for (int64_t base = 0; base < A.a.batch; base += NT) {
        const int64_t i = base + threadIdx.x;
        const int64_t n = i < A.a.batch ? tiles_of(A, S, i) * per : 0;
        int64_t inc = n;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(~0u, inc, d);
            if (lane >= d) inc += o;
        }
        __syncthreads();
        if (lane == 31) red[warp] = inc;
        __syncthreads();
        int64_t add = at, sum = 0;
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp) add += red[w];
            sum += red[w];
        }
        if (x < at + sum) {
            if (x >= add + inc - n && x < add + inc) {
                hit = i;
                hit_at = add + inc - n;
            }
            __syncthreads();
            at = hit_at;
            return hit;
        }
        at += sum;
    }
    return A.a.batch - 1;      // not reached: x < total
}

__device__ __forceinline__ int64_t piece(int64_t total, int64_t c, int64_t blocks) { return c * total / blocks; }
// The block whose piece holds tile x.
__device__ __forceinline__ int64_t block_of(int64_t total, int64_t x, int64_t blocks) { return ((x + 1) * blocks - 1) / total; }

// A slot of scratch: rows x head_dim sums, the rows' maxima and sums, and the
// mark of a V that is not finite.
__host__ __device__ __forceinline__ int64_t slot_floats(int rows, int head_dim) { return (int64_t)rows * (head_dim + 2) + 4; }
__device__ __forceinline__ float *slot_of(const Attn &A, const Share &S, int64_t block, int slot)
{
    return S.scratch + (block * 2 + slot) * slot_floats(S.rows, A.a.head_dim);
}

constexpr int JOIN_NT = 128;

// Joins the parts of a unit that more than one block worked on; one warp per
// row.  The parts' maxima and sums are read by the lanes at once, their outputs
// in the order of the cache.
template <class T>
__global__ void __launch_bounds__(JOIN_NT) k_attn_join(Attn A, Share S, int grid)
{
    const dbs_attention_args &a = A.a;
    __shared__ int64_t red[JOIN_NT / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t per = (uint32_t)a.kv_heads * S.groups;
    const uint32_t b = blockIdx.x / per, u = blockIdx.x % per;
    const Line L = line_at<JOIN_NT>(A, S, b, red);
    const Seq s = sequence(A, b);
    const int n = tiles_of(S, s);
    const int64_t x0 = L.at + (int64_t)u * n;
    const int64_t blocks = L.total < grid ? L.total : grid;
    const int64_t c0 = block_of(L.total, x0, blocks), c1 = block_of(L.total, x0 + n - 1, blocks);
    if (c0 == c1) return;
    const int hk = (int)(u / S.groups), r = blockIdx.y * (JOIN_NT / 32) + warp;
    if (r >= S.rows) return;
    const Row row = row_of(A, hk, (int64_t)(u % S.groups) * S.rows + r);
    if (!row.inside) return;
    float top = -INFINITY, sum = 0.f, o[8] = {};
    if (row.t < s.tree) {
        const int parts = (int)(c1 - c0) + 1;
        const int64_t size = slot_floats(S.rows, a.head_dim);
        // the unit may be the second of its first block, and is the first of the others
        const float *p0 = slot_of(A, S, c0, piece(L.total, c0, blocks) >= x0 ? 0 : 1), *rest = slot_of(A, S, c0, 0);
        const int64_t stat = (int64_t)S.rows * a.head_dim;
        for (int i = lane; i < parts; i += 32) top = fmaxf(top, (i ? rest + 2 * size * i : p0)[stat + r]);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        bool odd = false;
        for (int base = 0; base < parts; base += 32) {
            float f = 0.f, l = 0.f;
            if (base + lane < parts) {
                const float *st = (base + lane ? rest + 2 * size * (base + lane) : p0) + stat;
                const float m = st[r];
                l = st[S.rows + r];
                odd |= st[2 * S.rows] != 0.f;
                f = m == -INFINITY ? 0.f : exp2f(m - top);
                l = l != l ? l : f * l;
            }
            const int now = parts - base < 32 ? parts - base : 32;
            for (int i = 0; i < now; i += 4) {
                float v[4][8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = base + (i + k < now ? i + k : i);
                    const float *p = (c ? rest + 2 * size * c : p0) + (int64_t)r * a.head_dim;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[k][e] = lane + 32 * e < a.head_dim ? p[lane + 32 * e] : 0.f;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (i + k >= now) break;
                    const float fi = __shfl_sync(~0u, f, i + k);
                    sum += __shfl_sync(~0u, l, i + k);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] += fi == 0.f ? 0.f : fi * v[k][e];
                }
            }
        }
        if (__any_sync(~0u, odd)) {
            Eight w;
#pragma unroll
            for (int e = 0; e < 8; ++e) w.v[e] = o[e];
            w = add_odd<T>(A, b, row.t, hk, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = w.v[e];
        }
    }
    store_row<T>(A, b, row.t, row.h, top, sum, o);
}

// ---- few rows: every warp streams its own entries ----

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
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

template <int DP> constexpr int few_smem() { return FEW_W * FEW_STAGES * 2 * FEW_STEP * DP * 2; }

// 16 query rows against a piece of the cache.  The four warps take turns of 16
// entries, each with its own ring of K and V stages, running maximum, sum and
// output, so no block-wide wait runs in the loop; they are joined at the end of
// a unit.  A maximum is replaced only when it grew by more than 2^8, so the
// output is hardly ever rescaled (probabilities stay below 2^8, exact in
// proportion).
template <class T, int DP>
__global__ void __launch_bounds__(FEW_NT) k_attn_few(Attn A, Share S)
{
    const dbs_attention_args &a = A.a;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ int64_t red[FEW_W];
    __shared__ float s_m[FEW_W][FEW_ROWS], s_l[FEW_W][FEW_ROWS];
    __shared__ int s_odd[FEW_W];
    constexpr int RB = DP * 2, CH = DP / 8, HALF = FEW_STEP * RB;   // bytes and 16-byte chunks of an entry; of a stage's K
    constexpr int KK = DP / 16, NN = DP / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q4 = lane & 3;
    unsigned char *mine = ring + warp * (FEW_STAGES * 2 * HALF);
    const uint32_t base = smem_addr(mine);
    const int chunks = a.head_dim / 8;
    const int64_t per = (int64_t)a.kv_heads * S.groups;
    const int64_t total = line_at<FEW_NT>(A, S, 0, red).total;
    const int64_t blocks = total < gridDim.x ? total : gridDim.x;      // no empty pieces
    if (blockIdx.x < blocks) {
        int64_t x = piece(total, blockIdx.x, blocks);
        const int64_t end = piece(total, blockIdx.x + 1, blocks);
        int64_t at, b = sequence_of<FEW_NT>(A, S, x, at, red);
        bool first_piece = true;
        while (x < end) {
            const Seq s = sequence(A, b);
            const int n = tiles_of(S, s);
            const int64_t u = (x - at) / n;
            const int t0 = (int)(x - at - u * n), count = n - t0 < end - x ? n - t0 : (int)(end - x);
            const int hk = (int)((uint32_t)u / (uint32_t)S.groups);
            const int64_t R0 = (int64_t)((uint32_t)u % (uint32_t)S.groups) * FEW_ROWS;
            const int j0 = t0 * FEW_KEYS, j1 = (int64_t)(t0 + count) * FEW_KEYS < s.kv ? (t0 + count) * FEW_KEYS : s.kv;
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
                // probabilities rounded once to the caches' type for the second product
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
            const bool whole = count == n;
            odd = (s_odd[0] | s_odd[1] | s_odd[2] | s_odd[3]) != 0;
            float *part = slot_of(A, S, blockIdx.x, first_piece ? 0 : 1);
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
                if (whole) {
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
            __syncthreads();       // the rings are free again
            first_piece = false;
            x += count;
            if (x - at == n * per) {
                at = x;
                ++b;
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---- host ----

// How a call runs: the kernel, its grid and its scratch.
struct Plan {
    bool rows;                 // any alignment
    int dp, blocks;
    Share share;
    int64_t scratch;
};

bool aligned8(int64_t v) { return (v & 7) == 0; }

dbs_status plan_of(const dbs_attention_args &a, Plan &P)
{
    P = Plan{};
    const int64_t entries = a.max_pages * a.page_size;
    // 16-byte copies of heads: every head starts on such a boundary
    P.rows = a.head_dim % 8 || !aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned8(a.q_batch) ||
             !aligned8(a.q_token) || !aligned8(a.q_head) || !aligned8(a.k_page) || !aligned8(a.k_entry) ||
             !aligned8(a.k_head) || !aligned8(a.v_page) || !aligned8(a.v_entry) || !aligned8(a.v_head);
    if (P.rows) return DBS_OK;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return DBS_ERR_CUDA;
    }
    P.dp = a.head_dim <= 64 ? 64 : a.head_dim <= 128 ? 128 : 256;
    P.share.keys = FEW_KEYS;
    P.share.rows = FEW_ROWS;
    P.share.groups = (int)((a.tokens * (a.q_heads / a.kv_heads) + FEW_ROWS - 1) / FEW_ROWS);
    const int per_sm = P.dp == 64 ? 4 : P.dp == 128 ? 2 : 1;
    const int64_t most = a.batch * a.kv_heads * P.share.groups * (entries < FEW_KEYS ? 1 : (entries + FEW_KEYS - 1) / FEW_KEYS);
    P.blocks = (int)(most < sms * per_sm ? most : sms * per_sm);
    P.scratch = (int64_t)P.blocks * 2 * slot_floats(FEW_ROWS, a.head_dim) * 4;
    return DBS_OK;
}

// The joining kernel, started while the first one ends.
template <class T>
dbs_status launch_join(const Attn &A, const Plan &P, cudaStream_t s)
{
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(A.a.batch * A.a.kv_heads * P.share.groups), (unsigned)((P.share.rows + JOIN_NT / 32 - 1) / (JOIN_NT / 32)));
    c.blockDim = JOIN_NT;
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, k_attn_join<T>, A, P.share, P.blocks) == cudaSuccess ? DBS_OK : (cudaGetLastError(), DBS_ERR_CUDA);
}

template <class T, int DP>
dbs_status launch_few(const Attn &A, const Plan &P, cudaStream_t s)
{
    if (cudaFuncSetAttribute(k_attn_few<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, few_smem<DP>()) != cudaSuccess) {
        cudaGetLastError();
        return DBS_ERR_CUDA;
    }
    k_attn_few<T, DP><<<P.blocks, FEW_NT, few_smem<DP>(), s>>>(A, P.share);
    const dbs_status st = launched();
    return st == DBS_OK ? launch_join<T>(A, P, s) : st;
}

template <class T>
dbs_status launch(const Attn &A, const Plan &P, cudaStream_t s)
{
    if (P.rows) {
        const int64_t rows = A.a.batch * A.a.tokens * A.a.q_heads;
        k_attn_rows<T><<<(unsigned)(rows < (1 << 30) ? rows : (1 << 30)), ROW_NT, 0, s>>>(A);
        return launched();
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
    if (entries >= (int64_t(1) << 31)) return false;
    if (!a->q || !a->out || !a->kv_lens) return false;
    if (entries > 0 && (!a->k || !a->v || a->pages < 1)) return false;
    if (!a->page_table && (a->max_pages > 1 || (entries > 0 && a->pages < a->batch))) return false;
    return true;
}

}  // namespace

extern "C" {

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
    if (P.scratch > 0 && (!a->scratch || !aligned16(a->scratch) || a->scratch_bytes < P.scratch)) return DBS_ERR_INVALID_ARG;
    Attn A{*a, a->scale * 1.4426950408889634f, (int)((a->tokens + 63) / 64)};
    P.share.scratch = (float *)a->scratch;
    return a->dtype == DBS_F16 ? launch<__half>(A, P, (cudaStream_t)stream) : launch<__nv_bfloat16>(A, P, (cudaStream_t)stream);
}

}  // extern "C"
