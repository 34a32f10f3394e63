// What the attentions over a cache (attention.cu, window.cu) have in common: where entries
// lie, a row taken entry by entry, copies and matrix instructions of 16 rows, tensor maps
// of the caches, outputs.  A is dbs_attention_args or dbs_window_args.
#pragma once
#include <cmath>

#include "ops_dev.h"

namespace dbs::ops {

// Where entry j of sequence b lies: its page, and its place in it.
struct Place {
    int64_t page;
    uint32_t in;
};
template <class A> __device__ __forceinline__ Place place_of(const A &a, int64_t b, int j)
{
    if (!a.page_table) return {b, (uint32_t)j};
    const uint32_t size = (uint32_t)a.page_size, n = (uint32_t)j / size;
    const int64_t p = a.page_table[b * a.page_row + n];
    return {p < 0 ? 0 : p >= a.pages ? a.pages - 1 : p, (uint32_t)j - n * size};
}

// ---- one row by one warp, a lane every 32nd value ----

// A row's query; no maximum, sum and output yet.
template <class T, class A>
__device__ __forceinline__ void begin_row(const A &a, int64_t b, int t, int h, float (&q)[8], float &m, float &l, float (&o)[8])
{
    const int lane = threadIdx.x & 31;
    const T *from = (const T *)a.q + b * a.q_batch + t * a.q_token + h * a.q_head;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        q[e] = lane + 32 * e < a.head_dim ? to_f32(from[lane + 32 * e]) : 0.f;
        o[e] = 0.f;
    }
}
// One entry more.
template <class T, class A>
__device__ __forceinline__ void take_entry(const A &a, const Place &at, int hk, float scale_log2, const float (&q)[8], float &m, float &l, float (&o)[8])
{
    const int lane = threadIdx.x & 31;
    const T *k = (const T *)a.k + at.page * a.k_page + at.in * a.k_entry + hk * a.k_head;
    const T *v = (const T *)a.v + at.page * a.v_page + at.in * a.v_entry + hk * a.v_head;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (lane + 32 * e < a.head_dim) x = fmaf(q[e], to_f32(k[lane + 32 * e]), x);
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    x *= scale_log2;
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
// A row's output and lse from its sums: out = o / l, lse = (m + log2 l) ln 2.
template <class T, class A> __device__ __forceinline__ void store_out(const A &a, int64_t b, int t, int h, float l, const float (&o)[8])
{
    const int lane = threadIdx.x & 31;
    T *out = (T *)a.out + b * a.o_batch + t * a.o_token + h * a.o_head;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (lane + 32 * e < a.head_dim) out[lane + 32 * e] = from_f32<T>(l == 0.f ? 0.f : o[e] / l);
}
template <class A> __device__ __forceinline__ void store_lse(const A &a, int64_t b, int t, int h, float m, float l)
{
    a.lse[(b * a.tokens + t) * a.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}
template <class T, class A>
__device__ __forceinline__ void store_row(const A &a, int64_t b, int t, int h, float m, float l, const float (&o)[8])
{
    store_out<T>(a, b, t, h, l, o);
    if (a.lse && (threadIdx.x & 31) == 0) store_lse(a, b, t, h, m, l);
}

// What a part of a softmax's row counts in the row, whose maximum (in powers of two) is `top`: its sum and its outputs
// times that.  A part without a maximum has nothing, or a NaN that has to stay.  The product is taken even where the
// weight is 0: a NaN in a part is one in the row, however little it weighs.
__device__ __forceinline__ float weight_of(float m, float l, float top) { return m == -INFINITY ? (l != l ? 1.f : 0.f) : exp2f(m - top); }
// Its sum times that, rounded by itself: the lanes add theirs in pairs, and both of a pair have to come to the same.
__device__ __forceinline__ float weighed(float f, float l) { return __fmul_rn(f, l); }

// ---- 16 rows: asynchronous copies, fragments, matrix instructions ----

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

constexpr int FEW_NT = 128, FEW_W = FEW_NT / 32;
constexpr int FEW_ROWS = 16;               // one matrix instruction's rows
constexpr int FEW_STEP = 16;               // entries of a stage of a warp
constexpr int FEW_KEYS = FEW_W * FEW_STEP;
constexpr int FEW_SPLIT = 16;              // blocks of a cluster, at most

// Another block's value, by its address in this one.
__device__ __forceinline__ float remote(const void *p, int block)
{
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(block));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() { asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory"); }

// ---- 128 rows ----

// (to 2 units of the last place, and 0 below 2^-126: far below the 16 bits that P keeps)
__device__ __forceinline__ float pow2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 32 bytes, a whole sector, at once.
__device__ __forceinline__ void store32(float *p, float a, float b, float c, float d, float e, float f, float g, float h)
{
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d), "f"(e), "f"(f), "f"(g), "f"(h) : "memory");
}

// ---- tensor maps of K and V: [pages, entries, heads, head_dim], boxes of 64 columns of one head of `box` entries ----

struct Maps {
    CUtensorMap k, v;
    int box;
};

__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap *map, int d, int head, int entry, int page, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
                 "l"(map), "r"(bar), "r"(d), "r"(head), "r"(entry), "r"(page) : "memory");
}

inline bool aligned8(int64_t v) { return (v & 7) == 0; }
// Whether 16-byte copies of heads may be made: every head starts on such a boundary.
template <class A> bool on_vectors(const A &a)
{
    return a.head_dim % 8 == 0 && aligned16(a.q) && aligned16(a.k) && aligned16(a.v) && aligned8(a.q_batch) && aligned8(a.q_token) &&
           aligned8(a.q_head) && aligned8(a.k_page) && aligned8(a.k_entry) && aligned8(a.k_head) && aligned8(a.v_page) &&
           aligned8(a.v_entry) && aligned8(a.v_head);
}
inline bool wide_out(const void *out, int64_t batch, int64_t token, int64_t head)
{
    return aligned16(out) && aligned8(batch) && aligned8(token) && aligned8(head);
}

// A map of heads on vectors, `by` their strides; boxes of 64 columns.  (A dimension of one has any stride.)
inline bool map_of(CUtensorMap &map, dbs_dtype dtype, const void *p, const cuuint64_t (&dims)[4], const int64_t (&by)[3], const cuuint32_t (&box)[4])
{
    const encode_tiled_fn encode = encode_tiled();
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    cuuint64_t strides[3];
    for (int d = 0; d < 3; ++d) {
        const int64_t bytes = dims[d + 1] == 1 ? 16 * (int64_t)dims[0] : by[d] * 2;
        if (bytes <= 0 || bytes >= int64_t(1) << 40 || dims[d + 1] >= cuuint64_t(1) << 31) return false;
        strides[d] = (cuuint64_t)bytes;
    }
    return encode && encode(&map, dtype == DBS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims,
                            strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Boxes of the caches, of `most` entries (a power of two) or as many as divide a page, eight at least; false where pages or
// strides do not allow them.
template <class A> bool make_maps(const A &a, int most, Maps &M)
{
    if (a.page_size < 1 || a.pages < 1 || a.max_pages < 1) return false;
    // a sequence's own page is one run of entries; pages of a table split into boxes
    M.box = most;
    if (a.page_table)
        while (M.box >= 8 && a.page_size % M.box) M.box /= 2;
    if (M.box < 8) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.kv_heads, (cuuint64_t)a.page_size, (cuuint64_t)a.pages};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)M.box, 1};
    return map_of(M.k, a.dtype, a.k, dims, {a.k_head, a.k_entry, a.k_page}, box) && map_of(M.v, a.dtype, a.v, dims, {a.v_head, a.v_entry, a.v_page}, box);
}

}  // namespace dbs::ops
