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

bool aligned8(int64_t v) { return (v & 7) == 0; }

template <class T>
dbs_status launch(const Win &A, cudaStream_t s)
{
    k_window_rows<T><<<(unsigned)(A.a.batch * A.a.tokens * A.a.q_heads), ROW_NT, 0, s>>>(A);
    return launched();
}

}  // namespace

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
