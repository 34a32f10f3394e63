// Norms of queries and keys with their rotation in one pass (dbs_norm_rotary) and
// its gradient (dbs_norm_rotary_gradient, sm_103a).
#include <cmath>

#include "vec_dev.h"

using namespace dbs::ops;

namespace {

constexpr int NT = 256;

// A unit of a head is what one lane holds of it: two vectors of N values at `a` and
// `b`.  Of the turned entries they are the halves of N pairs, or, interleaved, N
// pairs one after another (the second vector is missing where the entries end); of
// the rest two vectors in a row.  A head is spread over L lanes of a warp (a power of
// two), K units each, so its sums need log2 L exchanges and no shared memory, and a
// head is read once.
struct Head {
    int head_dim, dim;
    int units, turned;                 // of a head; of its turned entries
    int lanes;                         // L
};

template <class T, bool INTERLEAVED, bool WIDE> struct Unit {
    static constexpr int N = Vec<T, WIDE>::n;
    static constexpr bool RUNS = INTERLEAVED && WIDE;      // pairs within a vector
    int a, b;
    bool some, both, turned;
    int pair;                                              // first of its N pairs
    __device__ __forceinline__ Unit(const Head &H, int c)
    {
        some = c < H.units;
        turned = c < H.turned;
        pair = c * N;
        const int r = H.dim + 2 * (c - H.turned) * N;
        a = !turned ? r : INTERLEAVED ? 2 * c * N : c * N;
        b = !turned || RUNS ? a + N : INTERLEAVED ? a + 1 : a + H.dim / 2;
        both = some && b < (turned ? H.dim : H.head_dim);
    }
};

template <class T, bool INTERLEAVED, bool WIDE> Head head_of(int head_dim, int dim)
{
    constexpr int N = Vec<T, WIDE>::n;
    Head H{head_dim, dim, 0, 0, 1};
    H.turned = (dim + 2 * N - 1) / (2 * N);
    H.units = H.turned + (head_dim - dim + 2 * N - 1) / (2 * N);
    while (H.lanes < 32 && H.lanes < H.units) H.lanes *= 2;
    return H;
}

template <class T, bool INTERLEAVED, bool WIDE, int K> struct Lane {
    using V = Vec<T, WIDE>;
    using VT = typename V::type;
    static constexpr int N = V::n, F = !WIDE ? 1 : N < 4 ? N : 4;
    using U = Unit<T, INTERLEAVED, WIDE>;

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
                const bool in = u.turned && u.pair + q < half;
                if (in && ok) {
                    const float *row = table + pos * H.dim + u.pair + q;
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
    static __device__ __forceinline__ void weights(const Head &H, int lane, const void *w, dbs_dtype type, float (&v)[K][2 * N])
    {
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
    static __device__ __forceinline__ void store(const Head &H, int lane, T *p, const VT (&x)[K][2])
    {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const U u(H, lane + k * H.lanes);
            if (u.some) *(VT *)(p + u.a) = x[k][0];
            if (u.both) *(VT *)(p + u.b) = x[k][1];
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
    static __device__ __forceinline__ void closed(const float (&v)[2 * N], VT (&x)[2])
    {
        float a[N], b[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            a[e] = v[e];
            b[e] = v[N + e];
        }
        shut<T>(a, x[0]);
        shut<T>(b, x[1]);
    }
    // (a, b) of every pair becomes (a cos - b sin, a sin + b cos)
    static __device__ __forceinline__ void turn(float (&v)[2 * N], const float (&cs)[N], const float (&sn)[N])
    {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float &a = U::RUNS ? v[2 * e] : v[e], &b = U::RUNS ? v[2 * e + 1] : v[N + e];
            const float a0 = a, b0 = b;
            a = a0 * cs[e] - b0 * sn[e];
            b = a0 * sn[e] + b0 * cs[e];
        }
    }
    // (every lane of the warp takes part; each head's lanes get their own sum)
    static __device__ __forceinline__ float sum(const Head &H, float v)
    {
        for (int d = H.lanes >> 1; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
        return v;
    }
};

// ---- forward ----

struct Norm {
    dbs_norm_heads part[3];
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
// `span` heads, HEADS of whose loads are issued together.  Bound by HBM: every entry is
// read and written once.
template <class T, bool INTERLEAVED, bool WIDE, int K>
__global__ void __launch_bounds__(NT) k_norm_rotary(Norm A, int span)
{
    using L = Lane<T, INTERLEAVED, WIDE, K>;
    constexpr int N = L::N, HEADS = K == 1 ? 4 : 1;
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
    float cs[K][N], sn[K][N], w[K][2 * N];
    if (norm) {
        L::angles(H, lane, A.table, A.table_rows, H.dim && in ? A.positions[tok] : 0, 1.f, cs, sn);
        L::weights(H, lane, A.part[p].weight, A.part[p].weight_dtype, w);
    }
    for (int h = 0; h < heads; h += HEADS) {
        typename L::VT x[HEADS][K][2];
#pragma unroll
        for (int k = 0; k < HEADS; ++k)
            if (h + k < heads) L::load(H, lane, src + k * P.in_head, x[k]);
#pragma unroll
        for (int k = 0; k < HEADS; ++k) {
            if (h + k >= heads) break;
            if (norm) {
                float v[K][2 * N], ss = 0.f;
#pragma unroll
                for (int c = 0; c < K; ++c) {
                    L::opened(x[k][c], v[c]);
#pragma unroll
                    for (int e = 0; e < 2 * N; ++e) ss = fmaf(v[c][e], v[c][e], ss);
                }
                const float r = 1.f / sqrtf(L::sum(H, ss) / (float)H.head_dim + A.eps);
#pragma unroll
                for (int c = 0; c < K; ++c) {
#pragma unroll
                    for (int e = 0; e < 2 * N; ++e) v[c][e] = v[c][e] * r * w[c][e];
                    L::turn(v[c], cs[c], sn[c]);
                    L::closed(v[c], x[k][c]);
                }
            }
            if (write) L::store(H, lane, dst + k * P.out_head, x[k]);
        }
        src += HEADS * P.in_head;
        dst += HEADS * P.out_head;
    }
}

template <class T, bool INTERLEAVED, bool WIDE, int K>
dbs_status launch_norm(Norm &A, int head_dim, int dim, cudaStream_t s)
{
    A.head = head_of<T, INTERLEAVED, WIDE>(head_dim, dim);
    A.copy = head_of<T, INTERLEAVED, WIDE>(head_dim, 0);
    const int lanes = A.head.lanes > A.copy.lanes ? A.head.lanes : A.copy.lanes;
    const int64_t room = (int64_t)multiprocessors() * 2048;
    if (room == 0) return DBS_ERR_CUDA;
    // Heads of a thread: eight, so that angles and weights are read once for all of them,
    // and fewer while that leaves some of the GPU's threads idle.
    int span = 8, chunks = 0;
    for (;; span /= 2) {
        chunks = 0;
        for (int p = 0; p < A.nparts; ++p) chunks += (A.part[p].heads.heads + span - 1) / span;
        if (span == 1 || A.total * lanes * chunks >= room || 2 * chunks > 65535) break;
    }
    k_norm_rotary<T, INTERLEAVED, WIDE, K><<<dim3((unsigned)((A.total * lanes + NT - 1) / NT), (unsigned)chunks), NT, 0, s>>>(A, span);
    return launched();
}

// ---- gradient ----

struct Gradient {
    dbs_norm_gradient_heads part[2];
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
// Bound by HBM: two entries are read and one is written.
template <class T, bool INTERLEAVED, bool WIDE, int K>
__global__ void __launch_bounds__(NT) k_norm_gradient(Gradient A, int span)
{
    using L = Lane<T, INTERLEAVED, WIDE, K>;
    constexpr int N = L::N, HEADS = K == 1 ? 2 : 1;
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
    float w[K][2 * N], dw[K][2 * N];
    L::weights(H, lane, P.weight, P.weight_dtype, w);
#pragma unroll
    for (int c = 0; c < K; ++c)
#pragma unroll
        for (int e = 0; e < 2 * N; ++e) dw[c][e] = 0.f;
    for (int64_t i0 = (int64_t)block * groups + first; i0 < items; i0 += step) {
        const int64_t i = i0 + (group - first);
        const bool in = i < items;
        const uint32_t tok = in ? (uint32_t)(i / chunks) : 0u, chunk = in ? (uint32_t)(i - (int64_t)tok * chunks) : 0u;
        const uint32_t b = tok / (uint32_t)A.tokens, t = tok - b * (uint32_t)A.tokens;
        const int h0 = (int)chunk * span, heads = P.heads - h0 < span ? P.heads - h0 : span;
        float cs[K][N], sn[K][N];
        L::angles(H, lane, A.table, A.table_rows, H.dim ? A.positions[tok] : 0, -1.f, cs, sn);
        const T *g = (const T *)P.grad + b * P.grad_batch + t * P.grad_token + h0 * P.grad_head;
        const T *x = (const T *)P.in + b * P.in_batch + t * P.in_token + h0 * P.in_head;
        T *out = (T *)P.out + b * P.out_batch + t * P.out_token + h0 * P.out_head;
        for (int h = 0; h < span; h += HEADS) {
            typename L::VT gv[HEADS][K][2], xv[HEADS][K][2];
#pragma unroll
            for (int k = 0; k < HEADS; ++k)
                if (in && h + k < heads) {
                    L::load(H, lane, g + k * P.grad_head, gv[k]);
                    L::load(H, lane, x + k * P.in_head, xv[k]);
                }
#pragma unroll
            for (int k = 0; k < HEADS; ++k) {
                const bool live = in && h + k < heads;
                float gf[K][2 * N], xf[K][2 * N], ss = 0.f, dot = 0.f;
#pragma unroll
                for (int c = 0; c < K; ++c) {
                    L::opened(gv[k][c], gf[c]);
                    L::opened(xv[k][c], xf[c]);
                    L::turn(gf[c], cs[c], sn[c]);
#pragma unroll
                    for (int e = 0; e < 2 * N; ++e) {
                        ss = fmaf(xf[c][e], xf[c][e], ss);
                        dot = fmaf(w[c][e] * gf[c][e], xf[c][e], dot);
                    }
                }
                ss = L::sum(H, ss);
                dot = L::sum(H, dot);
                const float r = 1.f / sqrtf(ss / (float)H.head_dim + A.eps), f = dot * r * r / (float)H.head_dim;
                if (!live) continue;
#pragma unroll
                for (int c = 0; c < K; ++c) {
#pragma unroll
                    for (int e = 0; e < 2 * N; ++e) {
                        dw[c][e] = fmaf(gf[c][e], xf[c][e] * r, dw[c][e]);
                        gf[c][e] = r * (w[c][e] * gf[c][e] - xf[c][e] * f);
                    }
                    L::closed(gf[c], gv[k][c]);
                }
                L::store(H, lane, out + k * P.out_head, gv[k]);
            }
            g += HEADS * P.grad_head;
            x += HEADS * P.in_head;
            out += HEADS * P.out_head;
        }
    }
    if (!P.weight_grad) return;
#pragma unroll
    for (int c = 0; c < K; ++c) {
        const typename L::U u(H, lane + c * H.lanes);
#pragma unroll
        for (int e = 0; e < 2 * N; ++e)
            if (e < N ? u.some : u.both) sums[group * H.head_dim + (e < N ? u.a + e : u.b + e - N)] = dw[c][e];
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
#pragma unroll 4
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

constexpr int GRADIENT_BLOCKS = 4;     // of a multiprocessor, at most

template <class T, bool INTERLEAVED, bool WIDE, int K>
dbs_status launch_gradient(Gradient &A, int head_dim, int dim, cudaStream_t s)
{
    A.head = head_of<T, INTERLEAVED, WIDE>(head_dim, dim);
    const int sms = multiprocessors(), groups = NT / A.head.lanes;
    if (sms == 0) return DBS_ERR_CUDA;
    A.room = sms * GRADIENT_BLOCKS;
    // Heads of a turn: as for the forward pass
    int span = 8;
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
        int64_t share = heads ? ((int64_t)A.room * A.part[p].heads + heads - 1) / heads : 0;
        share = share < A.room ? share : A.room;
        A.blocks[p] = (int)(most < share ? most : share);
        blocks += A.blocks[p];
        sum = sum || A.part[p].weight_grad;
    }
    if (blocks) {
        const int smem = groups * head_dim * (int)sizeof(float);
        k_norm_gradient<T, INTERLEAVED, WIDE, K><<<blocks, NT, smem, s>>>(A, span);
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

// 16-byte accesses: every head on such a boundary, and whole vectors in each part of a head.
template <class T> bool whole_vectors(int head_dim, int dim, bool interleaved, const float *table)
{
    constexpr int N = 16 / (int)sizeof(T);
    return dim % (interleaved ? N : 2 * N) == 0 && head_dim % N == 0 && aligned16(table);
}
template <class T> bool on_vectors(const void *p, int64_t b, int64_t t, int64_t h)
{
    constexpr int N = 16 / (int)sizeof(T);
    return aligned16(p) && ((b | t | h) & (N - 1)) == 0;
}

// The kernel for a head's size: units of a lane.
template <class T, bool INTERLEAVED, class A>
dbs_status choose(A &a, int head_dim, int dim, bool wide, cudaStream_t s, dbs_status (*const (&launch)[4])(A &, int, int, cudaStream_t))
{
    const int units = wide ? head_of<T, INTERLEAVED, true>(head_dim, dim).units : head_of<T, INTERLEAVED, false>(head_dim, dim).units;
    if (wide) return launch[units <= 32 ? 0 : 1](a, head_dim, dim, s);
    return launch[units <= 128 ? 2 : 3](a, head_dim, dim, s);
}
template <class T, bool INTERLEAVED> dbs_status norm_of(Norm &A, int head_dim, int dim, bool wide, cudaStream_t s)
{
    constexpr int MANY = sizeof(T) == 4 ? 5 : 3;           // (of 1024 entries at most, up to two vectors of which are short)
    static constexpr dbs_status (*launch[4])(Norm &, int, int, cudaStream_t) = {
        launch_norm<T, INTERLEAVED, true, 1>, launch_norm<T, INTERLEAVED, true, MANY>, launch_norm<T, INTERLEAVED, false, 4>,
        launch_norm<T, INTERLEAVED, false, 16>};
    return choose<T, INTERLEAVED, Norm>(A, head_dim, dim, wide, s, launch);
}
template <class T, bool INTERLEAVED> dbs_status gradient_of(Gradient &A, int head_dim, int dim, bool wide, cudaStream_t s)
{
    constexpr int MANY = sizeof(T) == 4 ? 5 : 3;
    static constexpr dbs_status (*launch[4])(Gradient &, int, int, cudaStream_t) = {
        launch_gradient<T, INTERLEAVED, true, 1>, launch_gradient<T, INTERLEAVED, true, MANY>, launch_gradient<T, INTERLEAVED, false, 4>,
        launch_gradient<T, INTERLEAVED, false, 16>};
    return choose<T, INTERLEAVED, Gradient>(A, head_dim, dim, wide, s, launch);
}

template <class T> dbs_status norm(Norm &A, int head_dim, int dim, bool interleaved, cudaStream_t s)
{
    bool wide = whole_vectors<T>(head_dim, dim, interleaved, A.table);
    for (int p = 0; p < A.nparts; ++p) {
        const dbs_rotary_heads &P = A.part[p].heads;
        wide = wide && on_vectors<T>(P.in, P.in_batch, P.in_token, P.in_head) && on_vectors<T>(P.out, P.out_batch, P.out_token, P.out_head);
    }
    return interleaved ? norm_of<T, true>(A, head_dim, dim, wide, s) : norm_of<T, false>(A, head_dim, dim, wide, s);
}
template <class T> dbs_status gradient(Gradient &A, int head_dim, int dim, bool interleaved, cudaStream_t s)
{
    bool wide = whole_vectors<T>(head_dim, dim, interleaved, A.table);
    for (int p = 0; p < A.nparts; ++p) {
        const dbs_norm_gradient_heads &P = A.part[p];
        wide = wide && (P.heads == 0 || (on_vectors<T>(P.grad, P.grad_batch, P.grad_token, P.grad_head) &&
                                         on_vectors<T>(P.in, P.in_batch, P.in_token, P.in_head) &&
                                         on_vectors<T>(P.out, P.out_batch, P.out_token, P.out_head)));
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
bool places_apart(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t size)
{
    return (n0 <= 1 || s0 >= size) && (n1 <= 1 || s1 >= size) && (n2 <= 1 || s2 >= size);
}

}  // namespace

extern "C" {

dbs_status dbs_norm_rotary(const dbs_norm_heads *parts, int32_t nparts, dbs_dtype dtype, int64_t batch, int64_t tokens,
                           int32_t head_dim, int32_t dim, float eps, const float *table, int64_t table_rows,
                           const int32_t *positions, const int32_t *slots, int64_t pages, int64_t page_size,
                           int32_t interleaved, void *stream)
{
    if (!parts || nparts < 1 || nparts > 3 || !sizes_ok(dtype, batch, tokens, head_dim, dim, eps, table_rows)) return DBS_ERR_INVALID_ARG;
    Norm A{};
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
        const bool apart = places_apart(P.heads, P.out_head, n_token, P.out_token, n_batch, P.out_batch, head_dim);
        const bool placed = P.in != P.out || (!P.to_slots && (P.heads == 1 || P.in_head == P.out_head) &&
                                              (tokens == 1 || P.in_token == P.out_token) && (batch == 1 || P.in_batch == P.out_batch));
        if (P.in_head < 0 || P.in_token < 0 || P.in_batch < 0 || !apart || !placed) return DBS_ERR_INVALID_ARG;
        A.part[A.nparts++] = parts[p];
    }
    if (!work || A.nparts == 0) return DBS_OK;
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
    *bytes = (int64_t)nparts * sms * GRADIENT_BLOCKS * head_dim * (int64_t)sizeof(float);
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
    for (int p = 0; p < nparts; ++p) {
        dbs_norm_gradient_heads P = parts[p];
        if (P.heads < 0 || P.heads > 16384 || (P.weight && !dtype_ok(P.weight_dtype))) return DBS_ERR_INVALID_ARG;
        sum = sum || P.weight_grad;
        if (!work) P.heads = 0;
        if (P.heads) {
            if (!P.grad || !P.in || !P.out || (dim > 0 && (!table || !positions))) return DBS_ERR_INVALID_ARG;
            for (int64_t stride : {P.grad_batch, P.grad_token, P.grad_head, P.in_batch, P.in_token, P.in_head})
                if (stride < 0) return DBS_ERR_INVALID_ARG;
            if (!places_apart(P.heads, P.out_head, tokens, P.out_token, batch, P.out_batch, head_dim)) return DBS_ERR_INVALID_ARG;
            auto same = [&](int64_t b, int64_t t, int64_t h) {
                return (batch == 1 || b == P.out_batch) && (tokens == 1 || t == P.out_token) && (P.heads == 1 || h == P.out_head);
            };
            if ((P.out == P.grad && !same(P.grad_batch, P.grad_token, P.grad_head)) || (P.out == P.in && !same(P.in_batch, P.in_token, P.in_head)))
                return DBS_ERR_INVALID_ARG;
            any = true;
        }
        A.part[A.nparts++] = P;
    }
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
