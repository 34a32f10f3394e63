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
    int64_t kv, first;         // entries; index of the first drafted one (may be < 0)
    int tree;                  // drafted tokens
};

__device__ __forceinline__ Seq sequence(const Attn &A, int64_t b)
{
    const dbs_attention_args &a = A.a;
    Seq s;
    const int64_t room = a.max_pages * a.page_size;
    int64_t kv = a.kv_lens[b], t = a.tree_lens ? a.tree_lens[b] : a.tokens;
    s.kv = kv < 0 ? 0 : kv > room ? room : kv;
    s.tree = (int)(t < 0 ? 0 : t > a.tokens ? a.tokens : t);
    s.first = s.kv - s.tree;
    return s;
}

__device__ __forceinline__ int64_t page_of(const dbs_attention_args &a, int64_t b, int64_t j)
{
    if (!a.page_table) return b;
    const int64_t p = a.page_table[b * a.page_row + j / a.page_size];
    return p < 0 ? 0 : p >= a.pages ? a.pages - 1 : p;
}

// Whether token t of sequence b sees drafted entry i (0 <= i < tree).
__device__ __forceinline__ bool sees(const Attn &A, int64_t b, int t, int i)
{
    if (!A.a.tree) return i <= t;
    return (uint64_t)A.a.tree[(b * A.a.tokens + t) * A.words + (i >> 6)] >> (i & 63) & 1u;
}

constexpr int ROW_NT = 128;

// Any head size and alignment: one block per query row; its warps take every
// fourth entry, a lane holds head_dim / 32 of the row.
template <class T>
__global__ void __launch_bounds__(ROW_NT) k_attn_rows(Attn A)
{
    const dbs_attention_args &a = A.a;
    constexpr int W = ROW_NT / 32, E = 8;       // 8 entries of a head per lane cover 256
    __shared__ float s_m[W], s_l[W], s_o[W][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t rows = a.batch * a.tokens * a.q_heads;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int h = (int)(r % a.q_heads);
        const int64_t bt = r / a.q_heads, b = bt / a.tokens;
        const int t = (int)(bt % a.tokens), hk = h / (a.q_heads / a.kv_heads);
        const Seq s = sequence(A, b);
        const T *q = (const T *)a.q + b * a.q_batch + t * a.q_token + h * a.q_head;
        float qr[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = lane + 32 * e;
            qr[e] = c < a.head_dim ? to_f32(q[c]) : 0.f;
            o[e] = 0.f;
        }
        if (t < s.tree)
            for (int64_t j = warp; j < s.kv; j += W) {
                if (j >= s.first && !sees(A, b, t, (int)(j - s.first))) continue;
                const int64_t p = page_of(a, b, j), in = a.page_table ? j % a.page_size : j;
                const T *k = (const T *)a.k + p * a.k_page + in * a.k_entry + hk * a.k_head;
                const T *v = (const T *)a.v + p * a.v_page + in * a.v_entry + hk * a.v_head;
                float x = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e)
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
                for (int e = 0; e < E; ++e)
                    if (lane + 32 * e < a.head_dim) o[e] = fmaf(pr, to_f32(v[lane + 32 * e]), o[e] * keep);
            }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) s_o[warp][lane + 32 * e] = o[e];
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
        __syncthreads();
        float top = -INFINITY, sum = 0.f, f[W];
        for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w]);
        for (int w = 0; w < W; ++w) {
            f[w] = s_m[w] == -INFINITY ? (s_l[w] != s_l[w] ? s_l[w] : 0.f) : exp2f(s_m[w] - top);
            sum += f[w] * s_l[w];
        }
        T *out = (T *)a.out + b * a.o_batch + t * a.o_token + h * a.o_head;
        for (int c = threadIdx.x; c < a.head_dim; c += ROW_NT) {
            float v = 0.f;
            for (int w = 0; w < W; ++w) v += f[w] * s_o[w][c];
            out[c] = from_f32<T>(sum == 0.f ? 0.f : v / sum);
        }
        if (a.lse && threadIdx.x == 0)
            a.lse[(b * a.tokens + t) * a.q_heads + h] = sum == 0.f ? -INFINITY : top * 0.6931471805599453f + logf(sum);
    }
}

template <class T>
void launch(const Attn &A, cudaStream_t s)
{
    const int64_t rows = A.a.batch * A.a.tokens * A.a.q_heads;
    k_attn_rows<T><<<(unsigned)(rows < (1 << 30) ? rows : (1 << 30)), ROW_NT, 0, s>>>(A);
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
    return DBS_OK;
}

dbs_status dbs_tree_attention(const dbs_attention_args *a, void *stream)
{
    if (!args_ok(a)) return DBS_ERR_INVALID_ARG;
    if (a->batch == 0 || a->tokens == 0) return DBS_OK;
    const Attn A{*a, a->scale * 1.4426950408889634f, (int)((a->tokens + 63) / 64)};
    if (a->dtype == DBS_F16) launch<__half>(A, (cudaStream_t)stream);
    else launch<__nv_bfloat16>(A, (cudaStream_t)stream);
    return launched();
}

}  // extern "C"
