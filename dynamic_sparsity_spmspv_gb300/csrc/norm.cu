// Norms of queries and keys with their rotation in one pass (dbs_norm_rotary) and
// its gradient (dbs_norm_rotary_gradient, sm_103a).
#include <cmath>

#include "places.h"
#include "vec_dev.h"

using namespace dbs::ops;

namespace {

constexpr int NT = 256;
// Blocks of a multiprocessor, heads whose loads are issued together, and heads of a thread at most, for
// heads of one unit a lane.  Forward the next heads are loaded before these are worked on (16,382 tokens of 40 heads of
// 128, bf16: 2, 3 and 12 60 us, 2, 3 and 8 61, 2, 2 and 8 66, 3, 1 and 8 67, 2, 4 and 16 78 (registers spilled);
// without that 3, 2 and 8 71).  The gradient has registers left for it in 16 bits only (8192 tokens of 32 heads of 96, f32: 2, 2 and
// 8 64 us, 2, 2 and 4 66, 2, 4 and 8 72, 2, 1 and 8 79, 3, 2 and 8 89 (spilled); loading ahead 76; of 40 heads of 128, bf16: 62,
// without loading ahead 74, with 1 head 72, 4 heads 90, 3 blocks 89, a span of 4 71).
constexpr int FORWARD_BLOCKS = 2, FORWARD_HEADS = 3, FORWARD_SPAN = 12, BACKWARD_BLOCKS = 2, BACKWARD_HEADS = 2, BACKWARD_SPAN = 8;

// What a lane moves at once: N values, 16 or 8 bytes, or one where rows are not aligned for that.
template <class T, int N> struct Piece {
    using type = uint4;
};
template <class T> struct Piece<T, 1> {
    using type = typename Vec<T, false>::type;
};
template <> struct Piece<__half, 4> {
    using type = uint2;
};
template <> struct Piece<__nv_bfloat16, 4> {
    using type = uint2;
};
using dbs::ops::open;
using dbs::ops::shut;
template <class T> __device__ __forceinline__ void open(const uint2 &w, float (&v)[4])
{
    open2<T>(w.x, v, 0);
    open2<T>(w.y, v, 1);
}
template <class T> __device__ __forceinline__ void shut(const float (&v)[4], uint2 &w) { w = make_uint2(shut2<T>(v, 0), shut2<T>(v, 1)); }

// A unit of a head is what one lane holds of it: two pieces, `a` and `b`.  Of the turned entries
// they are the halves of N pairs, or, interleaved, a piece of pairs from the first half of the
// turned entries and one from the second (none where their number is odd); of the rest likewise one
// from each half.  So the lanes of each access are neighbours in memory (with both pieces in a row an
// access has half of each sector).  A head is
// spread over L lanes of a warp (a power of two), K units each: its sums need log2 L exchanges and no shared
// memory, and it is read once.
struct Head {
    int head_dim, dim;
    int units, turned, rest;           // of a head, of its turned entries, of the others
    int lanes;                         // L
    float part;                        // 1 / head_dim
};

template <class T, bool INTERLEAVED, int N> struct Unit {
    static constexpr bool RUNS = INTERLEAVED && N > 1;     // pairs within a piece
    int a, b;
    bool some, both, turned;
    __device__ __forceinline__ Unit(const Head &H, int c)
    {
        some = c < H.units;
        turned = c < H.turned;
        const int r = c - H.turned;
        a = !turned ? H.dim + r * N : INTERLEAVED && N == 1 ? 2 * c : c * N;
        b = !turned ? a + H.rest * N : RUNS ? a + H.turned * N : INTERLEAVED ? a + 1 : a + H.dim / 2;
        both = some && b < (turned ? H.dim : H.head_dim);
    }
    // The pair whose angle value e of the N is (of pairs within pieces: half of them in each).
    __device__ __forceinline__ int pair(int e) const { return RUNS ? (e < N / 2 ? a / 2 + e : b / 2 + e - N / 2) : INTERLEAVED ? a / 2 : a + e; }
};

template <int N> Head head_of(int head_dim, int dim)
{
    Head H{head_dim, dim, 0, (dim / N + 1) / 2, ((head_dim - dim) / N + 1) / 2, 1, 1.f / (float)head_dim};
    H.units = H.turned + H.rest;
    while (H.lanes < 32 && H.lanes < H.units) H.lanes *= 2;
    return H;
}

template <class T, bool INTERLEAVED, int N, int K> struct Lane {
    using VT = typename Piece<T, N>::type;
    using U = Unit<T, INTERLEAVED, N>;
    static constexpr int RUN = U::RUNS ? N / 2 : N, F = RUN < 4 ? RUN : 4;     // angles in a row, of one load

    // The units' cosines and sines (1 and 0 of what is not turned).
    static __device__ __forceinline__ void angles(const Head &H, int lane, const float *table, int64_t rows, int64_t pos, float sign,
                                                  float (&cs)[K][N], float (&sn)[K][N])
    {
        const bool ok = pos >= 0 && pos < rows;
        const int half = H.dim / 2;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const U u(H, lane + k * H.lanes);
#pragma unroll
            for (int q = 0; q < N; q += F) {
                struct alignas(4 * F) Floats {
                    float v[F];
                };
                Floats c4, s4;
                const bool in = u.turned && (q < RUN || u.both);
                if (in && ok) {
                    const float *row = table + pos * H.dim + u.pair(q);
                    c4 = *(const Floats *)row;
                    s4 = *(const Floats *)(row + half);
                }
#pragma unroll
                for (int e = 0; e < F; ++e) {
                    cs[k][q + e] = !in ? 1.f : ok ? c4.v[e] : nanf("");
                    sn[k][q + e] = !in ? 0.f : ok ? sign * s4.v[e] : nanf("");
                }
            }
        }
    }
    // (`vectors`: the weight is of the heads' type and on 16-byte boundaries)
    static __device__ __forceinline__ void weights(const Head &H, int lane, const void *w, dbs_dtype type, bool vectors, float (&v)[K][2 * N])
    {
        if (N > 1 && vectors) {
            VT x[K][2];
            load(H, lane, (const T *)w, x);
#pragma unroll
            for (int k = 0; k < K; ++k) opened(x[k], v[k]);
            return;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const U u(H, lane + k * H.lanes);
#pragma unroll
            for (int e = 0; e < 2 * N; ++e) {
                const int at = e < N ? u.a + e : u.b + e - N;
                v[k][e] = 1.f;
                if (w && (e < N ? u.some : u.both))
                    v[k][e] = type == DBS_F32   ? ((const float *)w)[at]
                              : type == DBS_F16 ? to_f32(((const __half *)w)[at])
                                                : to_f32(((const __nv_bfloat16 *)w)[at]);
            }
        }
    }
    // The lane's units: where its pieces are.
    struct Units {
        int a[K], b[K];
        bool some[K], both[K], turned[K];
        __device__ __forceinline__ Units(const Head &H, int lane)
        {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const U u(H, lane + k * H.lanes);
                a[k] = u.a;
                b[k] = u.b;
                some[k] = u.some;
                both[k] = u.both;
                turned[k] = u.turned;
            }
        }
    };
    static __device__ __forceinline__ void load(const Units &u, const T *p, VT (&x)[K][2])
    {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k][0] = x[k][1] = VT{};
            if (u.some[k]) x[k][0] = *(const VT *)(p + u.a[k]);
            if (u.both[k]) x[k][1] = *(const VT *)(p + u.b[k]);
        }
    }
    static __device__ __forceinline__ void store(const Units &u, T *p, const VT (&x)[K][2])
    {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (u.some[k]) *(VT *)(p + u.a[k]) = x[k][0];
            if (u.both[k]) *(VT *)(p + u.b[k]) = x[k][1];
        }
    }
    static __device__ __forceinline__ void load(const Head &H, int lane, const T *p, VT (&x)[K][2])
    {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const U u(H, lane + k * H.lanes);
            x[k][0] = x[k][1] = VT{};
            if (u.some) x[k][0] = *(const VT *)(p + u.a);
            if (u.both) x[k][1] = *(const VT *)(p + u.b);
        }
    }
    static __device__ __forceinline__ void opened(const VT (&x)[2], float (&v)[2 * N])
    {
        float a[N], b[N];
        open<T>(x[0], a);
        open<T>(x[1], b);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            v[e] = a[e];
            v[N + e] = b[e];
        }
    }
    // A unit's values two by two, so that an instruction works on two: N words.
    static __device__ __forceinline__ void paired(const float (&v)[2 * N], uint64_t (&p)[N])
    {
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = two(v[2 * j], v[2 * j + 1]);
    }
    static __device__ __forceinline__ void opened(const VT (&x)[2], uint64_t (&p)[N])
    {
        float v[2 * N];
        opened(x, v);
        paired(v, p);
    }
    static __device__ __forceinline__ void closed(const uint64_t (&p)[N], VT (&x)[2])
    {
        float v[2 * N], a[N], b[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float2 f = apart(p[j]);
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            a[e] = v[e];
            b[e] = v[N + e];
        }
        shut<T>(a, x[0]);
        shut<T>(b, x[1]);
    }
    // What every value (of a pair that turns) takes of itself and of its partner: (a, b) becomes
    // (a wa cos - b wb sin, a wa sin + b wb cos).
    static constexpr bool WITHIN = U::RUNS || N == 1;      // a word holds both of a pair
    static __device__ __forceinline__ void turns(const float (&cs)[N], const float (&sn)[N], const float (&w)[2 * N], uint64_t (&own)[N], uint64_t (&other)[N])
    {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = 2 * j;
            if (WITHIN) {
                own[j] = two(cs[j] * w[e], cs[j] * w[e + 1]);
                other[j] = two(-sn[j] * w[e + 1], sn[j] * w[e]);
            } else if (e < N) {
                own[j] = two(cs[e] * w[e], cs[e + 1] * w[e + 1]);
                other[j] = two(-sn[e] * w[N + e], -sn[e + 1] * w[N + e + 1]);
            } else {
                own[j] = two(cs[e - N] * w[e], cs[e - N + 1] * w[e + 1]);
                other[j] = two(sn[e - N] * w[e - N], sn[e - N + 1] * w[e - N + 1]);
            }
        }
    }
    // (what is not turned takes nothing of others, whatever they hold)
    static __device__ __forceinline__ void turn(uint64_t (&p)[N], const uint64_t (&own)[N], const uint64_t (&other)[N], bool turned)
    {
        uint64_t q[N];
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = mul_two(p[j], own[j]);
        if (turned)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float2 f = apart(p[j]);
                q[j] = fma_two(WITHIN ? two(f.y, f.x) : p[(j + N / 2) % N], other[j], q[j]);
            }
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = q[j];
    }
    static __device__ __forceinline__ float both(uint64_t v)
    {
        const float2 f = apart(v);
        return f.x + f.y;
    }
    // (mean + eps)^(-1/2), the function's value with one step of Newton's method
    static __device__ __forceinline__ float root(const Head &H, float sum, float eps)
    {
        const float v = fmaf(sum, H.part, eps), r = rsqrtf(v), better = r * fmaf(-0.5f * v * r, r, 1.5f);
        return better == better ? better : r;              // (0 and infinity have no step)
    }
    // (every lane of the warp takes part; each head's lanes get their own sum)
    static __device__ __forceinline__ float sum(const Head &H, float v)
    {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
            if (d < H.lanes) v += __shfl_xor_sync(~0u, v, d);
        return v;
    }
};

// ---- forward ----

struct Norm {
    dbs_norm_heads part[3];
    bool vectors[3];                   // of the weights
    int32_t nparts;
    Head head, copy;                   // of the groups that are normed, and copied
    int64_t tokens, total;             // tokens of a sequence, tokens of all
    float eps;
    const float *table;
    int64_t table_rows;
    const int32_t *positions, *slots;
    int64_t page_size, slots_end;
};

// blockIdx.y: the chunks of `span` heads of every group; blockIdx.x: the tokens, L
// lanes each.  A group of lanes keeps its token's angles and its weights for up to
// `span` heads, HEADS of whose loads are issued together, while the HEADS before them are worked on.  Bound by HBM:
// every entry is read and written once (338 MB in 60 us, 83% of the memory's rate).
template <class T, bool INTERLEAVED, int N, int K>
__global__ void __launch_bounds__(NT, K == 1 ? FORWARD_BLOCKS : 1) k_norm_rotary(Norm A, int span)
{
    using L = Lane<T, INTERLEAVED, N, K>;
    constexpr int HEADS = K == 1 ? FORWARD_HEADS : 1;
    int y = blockIdx.y, p = 0;
    for (;; ++p) {
        const int chunks = (A.part[p].heads.heads + span - 1) / span;
        if (y < chunks) break;
        y -= chunks;
    }
    const dbs_rotary_heads &P = A.part[p].heads;
    const bool norm = P.rotate != 0;
    const Head H = norm ? A.head : A.copy;
    const int h0 = y * span, heads = P.heads - h0 < span ? P.heads - h0 : span;
    const uint32_t i = blockIdx.x * NT + threadIdx.x, tok = i / (uint32_t)H.lanes;
    const int lane = (int)(i & (uint32_t)(H.lanes - 1));
    if ((i & ~31u) / (uint32_t)H.lanes >= A.total) return;             // (whole warps: the others take part in the sums)
    const bool in = tok < A.total;
    const uint32_t b = in ? tok / (uint32_t)A.tokens : 0u, t = in ? tok - b * (uint32_t)A.tokens : 0u;
    const T *src = (const T *)P.in + b * P.in_batch + t * P.in_token + h0 * P.in_head;
    T *dst = (T *)P.out + h0 * P.out_head;
    bool write = in;
    if (P.to_slots) {
        const int64_t slot = in ? A.slots[tok] : -1;
        write = slot >= 0 && slot < A.slots_end;
        const uint32_t size = (uint32_t)A.page_size, at = write ? (uint32_t)slot : 0u, page = at / size;
        dst += page * P.out_batch + (at - page * size) * P.out_token;
    } else {
        dst += b * P.out_batch + t * P.out_token;
    }
    const typename L::Units units(H, lane);
    typename L::VT x[HEADS][K][2], next[HEADS][K][2];
    auto fetch = [&](int h, typename L::VT (&to)[HEADS][K][2]) {
#pragma unroll
        for (int k = 0; k < HEADS; ++k)
            if (h + k < heads) L::load(units, src + k * P.in_head, to[k]);
        src += HEADS * P.in_head;
    };
    fetch(0, x);
    uint64_t own[K][N], other[K][N];
    if (norm) {
        float cs[K][N], sn[K][N], w[K][2 * N];
        L::angles(H, lane, A.table, A.table_rows, H.dim && in ? A.positions[tok] : 0, 1.f, cs, sn);
        L::weights(H, lane, A.part[p].weight, A.part[p].weight_dtype, A.vectors[p], w);
#pragma unroll
        for (int c = 0; c < K; ++c) L::turns(cs[c], sn[c], w[c], own[c], other[c]);
    }
#pragma unroll 1
    for (int h = 0; h < heads; h += HEADS) {
        fetch(h + HEADS, next);
#pragma unroll
        for (int k = 0; k < HEADS; ++k) {
            if (h + k >= heads) break;
            if (norm) {
                uint64_t v[K][N], ss = 0;
#pragma unroll
                for (int c = 0; c < K; ++c) {
                    L::opened(x[k][c], v[c]);
#pragma unroll
                    for (int j = 0; j < N; ++j) ss = fma_two(v[c][j], v[c][j], ss);
                }
                const float r = L::root(H, L::sum(H, L::both(ss)), A.eps);
                const uint64_t r2 = two(r, r);
#pragma unroll
                for (int c = 0; c < K; ++c) {
#pragma unroll
                    for (int j = 0; j < N; ++j) v[c][j] = mul_two(v[c][j], r2);
                    L::turn(v[c], own[c], other[c], units.turned[c]);
                    L::closed(v[c], x[k][c]);
                }
            }
            if (write) L::store(units, dst + k * P.out_head, x[k]);
        }
#pragma unroll
        for (int k = 0; k < HEADS; ++k)
#pragma unroll
            for (int c = 0; c < K; ++c) {
                x[k][c][0] = next[k][c][0];
                x[k][c][1] = next[k][c][1];
            }
        dst += HEADS * P.out_head;
    }
}

template <class T, bool INTERLEAVED, int N, int K>
dbs_status launch_norm(Norm &A, int head_dim, int dim, cudaStream_t s)
{
    A.head = head_of<N>(head_dim, dim);
    A.copy = head_of<N>(head_dim, 0);
    const int lanes = A.head.lanes > A.copy.lanes ? A.head.lanes : A.copy.lanes;
    const int64_t room = (int64_t)multiprocessors() * 2048;
    if (room == 0) return DBS_ERR_CUDA;
    // Heads of a thread: many, so that angles and weights are read once for all of them,
    // and fewer while that leaves some of the GPU's threads idle.
    int span = FORWARD_SPAN, chunks = 0;
    for (;; span /= 2) {
        chunks = 0;
        for (int p = 0; p < A.nparts; ++p) chunks += (A.part[p].heads.heads + span - 1) / span;
        if (span == 1 || A.total * lanes * chunks >= room) break;          // (at most 3 * 16384 chunks)
    }
    k_norm_rotary<T, INTERLEAVED, N, K><<<dim3((unsigned)((A.total * lanes + NT - 1) / NT), (unsigned)chunks), NT, 0, s>>>(A, span);
    return launched();
}

// ---- gradient ----

struct Gradient {
    dbs_norm_gradient_heads part[2];
    bool vectors[2];
    int32_t nparts, blocks[2];         // blocks of each group of heads
    Head head;
    int64_t tokens, total;
    float eps;
    const float *table;
    int64_t table_rows;
    const int32_t *positions;
    float *scratch;                    // [part][block][head_dim]
    int room;                          // blocks that scratch holds of a part
};

// A group of lanes takes a token's heads, HEADS at a time, then the next token that is
// the grid's turn; what the heads give to weight' stays in its registers.  In the end the block's
// groups are added up in their order and written to scratch, and k_norm_weight adds the blocks.
// Two entries are read and one is written (f32, 303 MB in 66 us, 67% of the memory's rate; bf16, 8192 tokens of 40 heads of
// 128, 252 MB in 62 us, 60%).  Bound by latencies with 16 warps, more of which registers do not allow: in fp32 by the memory's,
// whose loads wait for the heads before them (issue 37% of the active cycles, 4.5 warps waiting for memory at each instruction); in
// 16 bits, with the next heads under way, by those of its instructions, 234 of a warp for two heads and their sums
// over lanes (issue 58%; waiting for an instruction before 1.9, for exchanges 1.1, for memory 1.1).
template <class T, bool INTERLEAVED, int N, int K>
__global__ void __launch_bounds__(NT, K == 1 ? BACKWARD_BLOCKS : 1) k_norm_gradient(Gradient A, int span)
{
    using L = Lane<T, INTERLEAVED, N, K>;
    constexpr int HEADS = K == 1 ? BACKWARD_HEADS : 1;
    constexpr bool AHEAD = sizeof(T) == 2;                 // (the next heads are loaded before these are worked on)
    extern __shared__ float sums[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int p = (int)blockIdx.x >= A.blocks[0], block = (int)blockIdx.x - (p ? A.blocks[0] : 0);
    const dbs_norm_gradient_heads &P = A.part[p];
    const Head H = A.head;
    const int lane = threadIdx.x & (H.lanes - 1), group = threadIdx.x / H.lanes, groups = NT / H.lanes;
    const uint32_t chunks = (uint32_t)((P.heads + span - 1) / span);
    const int64_t items = A.total * chunks, step = (int64_t)A.blocks[p] * groups;
    // (all lanes of a warp go the same number of turns)
    const int first = (threadIdx.x & ~31) / H.lanes;
    const typename L::Units units(H, lane);
    uint64_t w[K][N], dw[K][N];
    {
        float f[K][2 * N];
        L::weights(H, lane, P.weight, P.weight_dtype, A.vectors[p], f);
#pragma unroll
        for (int c = 0; c < K; ++c) {
            L::paired(f[c], w[c]);
#pragma unroll
            for (int j = 0; j < N; ++j) dw[c][j] = 0;
        }
    }
    for (int64_t i0 = (int64_t)block * groups + first; i0 < items; i0 += step) {
        const int64_t i = i0 + (group - first);
        const bool in = i < items;
        // (neighbours have neighbouring tokens: 66 us, with a token's chunks side by side 68)
        const uint32_t chunk = in ? (uint32_t)(i / A.total) : 0u, tok = in ? (uint32_t)(i - chunk * A.total) : 0u;
        const uint32_t b = tok / (uint32_t)A.tokens, t = tok - b * (uint32_t)A.tokens;
        const int h0 = (int)chunk * span, heads = P.heads - h0 < span ? P.heads - h0 : span;
        const T *g = (const T *)P.grad + b * P.grad_batch + t * P.grad_token + h0 * P.grad_head;
        const T *x = (const T *)P.in + b * P.in_batch + t * P.in_token + h0 * P.in_head;
        T *out = (T *)P.out + b * P.out_batch + t * P.out_token + h0 * P.out_head;
        using Set = typename L::VT[HEADS][K][2];
        Set gv, xv, gn, xn;
        auto fetch = [&](int h, Set &to_g, Set &to_x) {
#pragma unroll
            for (int k = 0; k < HEADS; ++k)
                if (in && h + k < heads) {
                    L::load(units, g + k * P.grad_head, to_g[k]);
                    L::load(units, x + k * P.in_head, to_x[k]);
                }
            g += HEADS * P.grad_head;
            x += HEADS * P.in_head;
        };
        fetch(0, gv, xv);
        uint64_t own[K][N], other[K][N];
        {
            float cs[K][N], sn[K][N], ones[2 * N];
            L::angles(H, lane, A.table, A.table_rows, H.dim ? A.positions[tok] : 0, -1.f, cs, sn);
#pragma unroll
            for (int e = 0; e < 2 * N; ++e) ones[e] = 1.f;
#pragma unroll
            for (int c = 0; c < K; ++c) L::turns(cs[c], sn[c], ones, own[c], other[c]);
        }
#pragma unroll 1
        for (int h = 0; h < span; h += HEADS) {
            if (AHEAD) fetch(h + HEADS, gn, xn);
            else if (h) fetch(h, gv, xv);
#pragma unroll
            for (int k = 0; k < HEADS; ++k) {
                const bool live = in && h + k < heads;
                uint64_t gf[K][N], xf[K][N], ss = 0, dot = 0;
#pragma unroll
                for (int c = 0; c < K; ++c) {
                    L::opened(gv[k][c], gf[c]);
                    L::opened(xv[k][c], xf[c]);
                    L::turn(gf[c], own[c], other[c], units.turned[c]);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        ss = fma_two(xf[c][j], xf[c][j], ss);
                        dot = fma_two(mul_two(w[c][j], gf[c][j]), xf[c][j], dot);
                    }
                }
                const float r = L::root(H, L::sum(H, L::both(ss)), A.eps), f = -L::sum(H, L::both(dot)) * r * r * H.part;
                if (!live) continue;
                const uint64_t r2 = two(r, r), f2 = two(f, f);
#pragma unroll
                for (int c = 0; c < K; ++c) {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        dw[c][j] = fma_two(gf[c][j], mul_two(xf[c][j], r2), dw[c][j]);
                        gf[c][j] = mul_two(r2, fma_two(xf[c][j], f2, mul_two(w[c][j], gf[c][j])));
                    }
                    L::closed(gf[c], gv[k][c]);
                }
                L::store(units, out + k * P.out_head, gv[k]);
            }
            if (AHEAD)
#pragma unroll
                for (int k = 0; k < HEADS; ++k)
#pragma unroll
                    for (int c = 0; c < K; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            gv[k][c][e] = gn[k][c][e];
                            xv[k][c][e] = xn[k][c][e];
                        }
            out += HEADS * P.out_head;
        }
    }
    if (!P.weight_grad) return;
#pragma unroll
    for (int c = 0; c < K; ++c) {
        const typename L::U u(H, lane + c * H.lanes);
#pragma unroll
        for (int e = 0; e < 2 * N; ++e) {
            const float2 f = apart(dw[c][e / 2]);
            if (e < N ? u.some : u.both) sums[group * H.head_dim + (e < N ? u.a + e : u.b + e - N)] = e & 1 ? f.y : f.x;
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < H.head_dim; d += NT) {
        float s = 0.f;
        for (int k = 0; k < groups; ++k) s += sums[k * H.head_dim + d];
        A.scratch[((int64_t)p * A.room + block) * H.head_dim + d] = s;
    }
}

// The blocks' sums of 32 columns, by 32 warps in turn, then theirs in order.
__global__ void __launch_bounds__(1024) k_norm_weight(Gradient A, int head_dim)
{
    __shared__ float part[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const dbs_norm_gradient_heads &P = A.part[blockIdx.y];
    if (!P.weight_grad) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
    const float *from = A.scratch + (int64_t)blockIdx.y * A.room * head_dim;
    float s = 0.f;
    if (d < head_dim)
#pragma unroll 16
        for (int k = warp; k < A.blocks[blockIdx.y]; k += 32) s += __ldcg(from + (int64_t)k * head_dim + d);
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && d < head_dim) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) s += part[k][lane];
        P.weight_grad[d] = s;
    }
}


template <class T, bool INTERLEAVED, int N, int K>
dbs_status launch_gradient(Gradient &A, int head_dim, int dim, cudaStream_t s)
{
    A.head = head_of<N>(head_dim, dim);
    const int sms = multiprocessors(), groups = NT / A.head.lanes;
    if (sms == 0) return DBS_ERR_CUDA;
    A.room = sms * BACKWARD_BLOCKS;
    // Heads of a turn: as for the forward pass
    int span = BACKWARD_SPAN;
    int64_t heads = 0;
    for (int p = 0; p < A.nparts; ++p) heads += A.part[p].heads;
    for (; span > 1; span /= 2) {
        int64_t items = 0;
        for (int p = 0; p < A.nparts; ++p) items += A.total * ((A.part[p].heads + span - 1) / span);
        if (items >= (int64_t)A.room * groups) break;
    }
    int blocks = 0;
    bool sum = false;
    for (int p = 0; p < A.nparts; ++p) {
        const int64_t items = A.total * ((A.part[p].heads + span - 1) / span), most = (items + groups - 1) / groups;
        // (no more blocks than find room at once, in both groups together: one more would run when the others have ended)
        int64_t share = heads ? (int64_t)A.room * A.part[p].heads / heads : 0;
        if (share == 0) share = 1;
        A.blocks[p] = (int)(most < share ? most : share);
        blocks += A.blocks[p];
        sum = sum || A.part[p].weight_grad;
    }
    if (blocks) {
        const int smem = groups * head_dim * (int)sizeof(float);
        k_norm_gradient<T, INTERLEAVED, N, K><<<blocks, NT, smem, s>>>(A, span);
        const dbs_status st = launched();
        if (st != DBS_OK) return st;
    }
    if (!sum) return DBS_OK;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)((head_dim + 31) / 32), (unsigned)A.nparts);
    c.blockDim = 1024;
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = blocks ? 1 : 0;
    return cudaLaunchKernelEx(&c, k_norm_weight, A, head_dim) == cudaSuccess ? DBS_OK : (cudaGetLastError(), DBS_ERR_CUDA);
}

// Pieces of N values: every head on such a boundary, and whole pieces in each part of a head.
template <int N> bool whole_pieces(int head_dim, int dim, bool interleaved, const float *table)
{
    return dim % (interleaved ? N : 2 * N) == 0 && head_dim % N == 0 && aligned16(table);
}
template <class T, int N> bool on_pieces(const void *p, int64_t b, int64_t t, int64_t h)
{
    return (reinterpret_cast<uintptr_t>(p) & (N * sizeof(T) - 1)) == 0 && ((b | t | h) & (N - 1)) == 0;
}

// Values of a piece.  Forward 16 bytes of them.  The gradient holds twice as much of a head
// beside its weights and their sums, so it takes half as many of 16 bits (with 16 bytes of them, and one block of a
// multiprocessor instead of two: 59 us for 62 above, 53 for 55 with heads of 256, as many with heads of 96).
template <class T> constexpr int FORWARD = 16 / (int)sizeof(T);
template <class T> constexpr int BACKWARD = 4;

// The kernel for a head's size: units of a lane (at most 1024 entries, and the last piece of each part may
// have no second).  The gradient's kernels of many units, for heads above 256 entries, spill registers (2048 tokens of 10 heads of
// 512: bf16 81 us, f32 97, floors 9 and 18; of 1024 91 and 120).
template <class T, bool INTERLEAVED> dbs_status norm_of(Norm &A, int head_dim, int dim, bool wide, cudaStream_t s)
{
    constexpr int N = FORWARD<T>;
    if (wide) return head_of<N>(head_dim, dim).units <= 32 ? launch_norm<T, INTERLEAVED, N, 1>(A, head_dim, dim, s)
                                                           : launch_norm<T, INTERLEAVED, N, 16 / N + 1>(A, head_dim, dim, s);
    return head_of<1>(head_dim, dim).units <= 128 ? launch_norm<T, INTERLEAVED, 1, 4>(A, head_dim, dim, s)
                                                  : launch_norm<T, INTERLEAVED, 1, 16>(A, head_dim, dim, s);
}
template <class T, bool INTERLEAVED> dbs_status gradient_of(Gradient &A, int head_dim, int dim, bool wide, cudaStream_t s)
{
    constexpr int N = BACKWARD<T>;
    if (wide) return head_of<N>(head_dim, dim).units <= 32 ? launch_gradient<T, INTERLEAVED, N, 1>(A, head_dim, dim, s)
                                                           : launch_gradient<T, INTERLEAVED, N, 16 / N + 1>(A, head_dim, dim, s);
    return head_of<1>(head_dim, dim).units <= 128 ? launch_gradient<T, INTERLEAVED, 1, 4>(A, head_dim, dim, s)
                                                  : launch_gradient<T, INTERLEAVED, 1, 16>(A, head_dim, dim, s);
}

template <class T> bool type_is(dbs_dtype t)
{
    return t == (sizeof(T) == 4 ? DBS_F32 : __is_same(T, __half) ? DBS_F16 : DBS_BF16);
}
template <class T> dbs_status norm(Norm &A, int head_dim, int dim, bool interleaved, cudaStream_t s)
{
    constexpr int N = FORWARD<T>;
    bool wide = whole_pieces<N>(head_dim, dim, interleaved, A.table);
    for (int p = 0; p < A.nparts; ++p) {
        const dbs_rotary_heads &P = A.part[p].heads;
        wide = wide && on_pieces<T, N>(P.in, P.in_batch, P.in_token, P.in_head) && on_pieces<T, N>(P.out, P.out_batch, P.out_token, P.out_head);
        A.vectors[p] = A.part[p].weight && type_is<T>(A.part[p].weight_dtype) && aligned16(A.part[p].weight);
    }
    return interleaved ? norm_of<T, true>(A, head_dim, dim, wide, s) : norm_of<T, false>(A, head_dim, dim, wide, s);
}
template <class T> dbs_status gradient(Gradient &A, int head_dim, int dim, bool interleaved, cudaStream_t s)
{
    constexpr int N = BACKWARD<T>;
    bool wide = whole_pieces<N>(head_dim, dim, interleaved, A.table);
    for (int p = 0; p < A.nparts; ++p) {
        const dbs_norm_gradient_heads &P = A.part[p];
        wide = wide && (P.heads == 0 || (on_pieces<T, N>(P.grad, P.grad_batch, P.grad_token, P.grad_head) &&
                                         on_pieces<T, N>(P.in, P.in_batch, P.in_token, P.in_head) &&
                                         on_pieces<T, N>(P.out, P.out_batch, P.out_token, P.out_head)));
        A.vectors[p] = P.weight && type_is<T>(P.weight_dtype) && aligned16(P.weight);
    }
    return interleaved ? gradient_of<T, true>(A, head_dim, dim, wide, s) : gradient_of<T, false>(A, head_dim, dim, wide, s);
}

// Sizes that both directions check.
bool sizes_ok(dbs_dtype dtype, int64_t batch, int64_t tokens, int32_t head_dim, int32_t dim, float eps, int64_t table_rows)
{
    if (!dtype_ok(dtype) || batch < 0 || tokens < 0 || head_dim < 1 || head_dim > 1024 || dim < 0 || dim > head_dim || (dim & 1) ||
        table_rows < 0 || !(eps >= 0) || !std::isfinite(eps))
        return false;
    if (batch == 0 || tokens == 0) return true;
    return batch <= (int64_t(1) << 31) && tokens <= (int64_t(1) << 31) && batch * tokens < (int64_t(1) << 31) &&
           batch * tokens * head_dim < (int64_t(1) << 32) - NT;
}
int64_t size_of(dbs_dtype dtype) { return dtype == DBS_F32 ? 4 : 2; }
// A negative stride among those of a group's heads.
bool backwards(int64_t batch, int64_t token, int64_t head) { return batch < 0 || token < 0 || head < 0; }

}  // namespace

extern "C" {

dbs_status dbs_norm_rotary(const dbs_norm_heads *parts, int32_t nparts, dbs_dtype dtype, int64_t batch, int64_t tokens,
                           int32_t head_dim, int32_t dim, float eps, const float *table, int64_t table_rows,
                           const int32_t *positions, const int32_t *slots, int64_t pages, int64_t page_size,
                           int32_t interleaved, void *stream)
{
    if (!parts || nparts < 1 || nparts > 3 || !sizes_ok(dtype, batch, tokens, head_dim, dim, eps, table_rows)) return DBS_ERR_INVALID_ARG;
    Norm A{};
    Places writes[3], reads[3];
    const bool work = batch > 0 && tokens > 0;
    for (int p = 0; p < nparts; ++p) {
        const dbs_rotary_heads &P = parts[p].heads;
        if (P.heads < 0 || P.heads > 16384) return DBS_ERR_INVALID_ARG;
        if (P.heads == 0) continue;
        if (P.rotate && parts[p].weight && !dtype_ok(parts[p].weight_dtype)) return DBS_ERR_INVALID_ARG;
        if (!work) continue;
        if (!P.in || (P.rotate && dim > 0 && (!table || !positions)) ||
            (P.to_slots && (!slots || pages < 0 || page_size < 1 || pages > (int64_t(1) << 31) / page_size)))
            return DBS_ERR_INVALID_ARG;
        if (P.to_slots && pages == 0) continue;                                // no slot is inside: nothing is written
        if (!P.out) return DBS_ERR_INVALID_ARG;
        const int64_t n_batch = P.to_slots ? pages : batch, n_token = P.to_slots ? page_size : tokens;
        const Places out(P.out, size_of(dtype), head_dim, {{n_batch, P.out_batch}, {n_token, P.out_token}, {P.heads, P.out_head}});
        if (backwards(P.in_batch, P.in_token, P.in_head) || !out.own || (P.to_slots && P.in == P.out)) return DBS_ERR_INVALID_ARG;
        // (of a cache only the slots are written, which the host does not know)
        if (!P.to_slots) writes[A.nparts] = out;
        reads[A.nparts] = {P.in, size_of(dtype), head_dim, {{batch, P.in_batch}, {tokens, P.in_token}, {P.heads, P.in_head}}};
        A.part[A.nparts++] = parts[p];
    }
    if (!work || A.nparts == 0) return DBS_OK;
    if (clash(writes, A.nparts, reads, A.nparts, true)) return DBS_ERR_INVALID_ARG;
    A.tokens = tokens;
    A.total = batch * tokens;
    A.eps = eps;
    A.table = table;
    A.table_rows = table_rows;
    A.positions = positions;
    A.slots = slots;
    A.page_size = page_size;
    A.slots_end = slots ? pages * page_size : 0;
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == DBS_F32   ? norm<float>(A, head_dim, dim, interleaved != 0, s)
           : dtype == DBS_F16 ? norm<__half>(A, head_dim, dim, interleaved != 0, s)
                              : norm<__nv_bfloat16>(A, head_dim, dim, interleaved != 0, s);
}

dbs_status dbs_norm_rotary_gradient_scratch(int32_t nparts, int32_t head_dim, int64_t *bytes)
{
    if (!bytes || nparts < 1 || nparts > 2 || head_dim < 1 || head_dim > 1024) return DBS_ERR_INVALID_ARG;
    const int sms = multiprocessors();
    if (sms == 0) return DBS_ERR_CUDA;
    *bytes = (int64_t)nparts * sms * BACKWARD_BLOCKS * head_dim * (int64_t)sizeof(float);
    return DBS_OK;
}

dbs_status dbs_norm_rotary_gradient(const dbs_norm_gradient_heads *parts, int32_t nparts, dbs_dtype dtype, int64_t batch,
                                    int64_t tokens, int32_t head_dim, int32_t dim, float eps, const float *table,
                                    int64_t table_rows, const int32_t *positions, int32_t interleaved, void *scratch,
                                    int64_t scratch_bytes, void *stream)
{
    if (!parts || nparts < 1 || nparts > 2 || !sizes_ok(dtype, batch, tokens, head_dim, dim, eps, table_rows)) return DBS_ERR_INVALID_ARG;
    Gradient A{};
    const bool work = batch > 0 && tokens > 0;
    bool sum = false, any = false;
    Places writes[4], grads[2], reads[2];              // x' and weight' of each group
    for (int p = 0; p < nparts; ++p) {
        dbs_norm_gradient_heads P = parts[p];
        if (P.heads < 0 || P.heads > 16384 || (P.weight && !dtype_ok(P.weight_dtype))) return DBS_ERR_INVALID_ARG;
        sum = sum || P.weight_grad;
        if (!work) P.heads = 0;
        if (P.heads) {
            if (!P.grad || !P.in || !P.out || (dim > 0 && (!table || !positions))) return DBS_ERR_INVALID_ARG;
            const Places out(P.out, size_of(dtype), head_dim, {{batch, P.out_batch}, {tokens, P.out_token}, {P.heads, P.out_head}});
            if (backwards(P.grad_batch, P.grad_token, P.grad_head) || backwards(P.in_batch, P.in_token, P.in_head) || !out.own)
                return DBS_ERR_INVALID_ARG;
            writes[p] = out;
            grads[p] = {P.grad, size_of(dtype), head_dim, {{batch, P.grad_batch}, {tokens, P.grad_token}, {P.heads, P.grad_head}}};
            reads[p] = {P.in, size_of(dtype), head_dim, {{batch, P.in_batch}, {tokens, P.in_token}, {P.heads, P.in_head}}};
            any = true;
        }
        if (P.weight_grad) writes[2 + p] = {P.weight_grad, 4, head_dim, {}};
        A.part[A.nparts++] = P;
    }
    if (clash(writes, 4, grads, 2, true) || clash(writes, 4, reads, 2, true)) return DBS_ERR_INVALID_ARG;
    if (!sum && !any) return DBS_OK;
    if (sum) {
        int64_t need = 0;
        const dbs_status st = dbs_norm_rotary_gradient_scratch(nparts, head_dim, &need);
        if (st != DBS_OK) return st;
        if (!scratch || !aligned16(scratch) || scratch_bytes < need) return DBS_ERR_INVALID_ARG;
    }
    A.tokens = work ? tokens : 1;
    A.total = work ? batch * tokens : 0;
    A.eps = eps;
    A.table = table;
    A.table_rows = table_rows;
    A.positions = positions;
    A.scratch = (float *)scratch;
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == DBS_F32   ? gradient<float>(A, head_dim, dim, interleaved != 0, s)
           : dtype == DBS_F16 ? gradient<__half>(A, head_dim, dim, interleaved != 0, s)
                              : gradient<__nv_bfloat16>(A, head_dim, dim, interleaved != 0, s);
}

}  // extern "C"
