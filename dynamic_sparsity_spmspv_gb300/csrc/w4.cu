// Linear layer with 4-bit weights and group scales for one or a few tokens
// (dbs_w4_linear, sm_103a):
//     y[t, i] = sum_g s[i, g] * sum_{j in g} x[t, j] (q[i, j] - z[i, g]).
#include "ops_dev.h"
#include "tc_dev.h"
#include <type_traits>

using namespace dbs::ops;

namespace {

struct W4 {
    const void *x;
    const uint8_t *q;
    const void *scales;
    const uint8_t *zeros;
    void *y;
    int64_t tokens, x_stride, q_stride, scale_stride, zero_stride, m, n, y_stride;
    int32_t group;
    Waits waits;
};

// 16-byte loads of x: every token's row on such a boundary.
template <class T>
__device__ __forceinline__ bool aligned_x(const T *x, int64_t stride)
{
    return (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (stride * sizeof(T) & 15u) == 0;
}

constexpr int ROWS_NT = 128;     // four warps, one row each
constexpr int ROWS_TOK = 4;      // tokens a warp carries at a time

// Any alignment: one warp per row and ROWS_TOK tokens, two columns per byte.  Bound
// by its instructions (1 token, 4096 x 11008, fp32: 73 us, k_w4_mma 12).
template <class T, class S>
__global__ void __launch_bounds__(ROWS_NT) k_w4_rows(W4 A)
{
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * (ROWS_NT / 32) + (threadIdx.x >> 5);
    if (i >= A.m) return;
    const uint8_t *q = A.q + i * A.q_stride;
    const uint8_t *z = A.zeros ? A.zeros + i * A.zero_stride : nullptr;
    const int64_t bytes = (A.n + 1) >> 1;
    for (int64_t t0 = (int64_t)blockIdx.y * ROWS_TOK; t0 < A.tokens; t0 += (int64_t)gridDim.y * ROWS_TOK) {
        float acc[ROWS_TOK] = {};
        for (int64_t c = lane; c < bytes; c += 32) {
            const int64_t j = 2 * c, g = j / A.group;
            const float sc = to_f32(((const S *)A.scales)[i * A.scale_stride + g]), zp = z ? (float)(z[g] & 127) : 8.f;
            const unsigned b = q[c];
            const float w0 = ((float)(b & 15u) - zp) * sc, w1 = ((float)(b >> 4) - zp) * sc;
#pragma unroll
            for (int k = 0; k < ROWS_TOK; ++k) {
                if (t0 + k >= A.tokens) break;
                const T *x = (const T *)A.x + (t0 + k) * A.x_stride;
                acc[k] = fmaf(w0, to_f32(x[j]), acc[k]);
                if (j + 1 < A.n) acc[k] = fmaf(w1, to_f32(x[j + 1]), acc[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < ROWS_TOK; ++k) {
#pragma unroll
            for (int o = 16; o; o >>= 1) acc[k] += __shfl_xor_sync(~0u, acc[k], o);
            if (lane == 0 && t0 + k < A.tokens) ((T *)A.y)[(t0 + k) * A.y_stride + i] = from_f32<T>(acc[k]);
        }
    }
}

// ---- rows on 16-byte boundaries: tensor cores ----
//
// A matrix instruction takes 16 rows of codes (A, 16 x 16) and 8 columns of x
// (B, 16 x 8): the columns are tokens, or, for fp32 x, the three 8-bit pieces
// hi + mid + lo whose sum is x exactly (truncated splits of its 24 bits), so
// fp32 costs three columns a token and loses nothing.  Codes become numbers in
// registers: with a nibble in the low mantissa bits, (128 + q) / 256 in bf16 (1024
// + q in fp16) is one AND-OR of a word's nibble pair, and subtracting the same
// of z gives q - z (by the unit 1/256) exactly.  Which column of x a fragment's slot
// stands for is free as long as A and B agree: a lane's word holds 8 neighbouring columns, paired (0, 4),
// (1, 5), (2, 6), (3, 7) as they lie in the word, and x is laid out to match.
// Groups' sums are fp32 accumulators, multiplied by the scale in fp32.
template <class T> struct Half2;
template <> struct Half2<__half> {
    static constexpr uint32_t magic = 0x64006400u, one = 0x00010001u;   // 1024 + q
    static constexpr float unit = 1.f;
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Half2<__nv_bfloat16> {
    // (128 + q) / 256: sums stay below the largest fp32 for the largest x
    static constexpr uint32_t magic = 0x3f003f00u, one = 0x00010001u;
    static constexpr float unit = 256.f;
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// The matrix type of x's type, and its columns per token.
template <class T> struct Piece { using type = T; static constexpr int parts = 1; };
template <> struct Piece<float> { using type = __nv_bfloat16; static constexpr int parts = 3; };

constexpr int MMA_NT = 512, MMA_W = MMA_NT / 32;   // one block an SM
constexpr int STAGES = 3, STAGE = 2048;           // of a warp's ring; bytes
// A stage is RT tiles of 16 rows: 256 columns of one, or 128 of two.
template <int RT> constexpr int STEP_V = RT == 1 ? 256 : 128;

// How a call is cut up.
struct Cut {
    int wk;                    // warps of a block that share a row tile and take turns of its stages
    int steps, phase;          // stages of a row; stages whose x is in shared memory at a time
    int shift;                 // log2 of the group
    int64_t groups;            // of rows: a block's rows at a time
    bool bf16_scales;          // of 16-bit ones
    uint32_t magic;            // of the codes' numbers
};

__device__ __forceinline__ void stage_load(uint32_t dst, const CUtensorMap *map, int byte, int row, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(map),
                 "r"(bar), "r"(byte), "r"(row) : "memory");
}

// Eight neighbouring values of x, zeros behind the row's end, and the same as the
// pairs (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __noinline__ uint4 eight_by_one(const uint16_t *x, int64_t j, int64_t n)
{
    uint16_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = j + e < n ? x[j + e] : (uint16_t)0;
    return make_uint4(v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16, v[4] | (uint32_t)v[5] << 16, v[6] | (uint32_t)v[7] << 16);
}
template <class T>
__device__ __forceinline__ uint4 eight(const T *x, int64_t j, int64_t n, bool wide)
{
    return wide && j + 8 <= n ? *(const uint4 *)(x + j) : eight_by_one((const uint16_t *)x, j, n);
}
__device__ __forceinline__ uint4 paired(uint4 u)
{
    return make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410), __byte_perm(u.y, u.w, 0x7632));
}
template <class T>
__device__ __forceinline__ void lay_out(const T *x, int64_t j, int64_t n, bool wide, uint4 (&out)[1])
{
    out[0] = paired(eight(x, j, n, wide));
}

// The same of fp32: the upper 8 bits of each value, the next 8, the last 8, each
// a bf16.  What is not finite goes into the first piece alone.
__device__ __forceinline__ void lay_out(const float *x, int64_t j, int64_t n, bool wide, uint4 (&out)[3])
{
    float v[8];
    if (wide && j + 8 <= n) {
        *(float4 *)v = *(const float4 *)(x + j);
        *(float4 *)(v + 4) = *(const float4 *)(x + j + 4);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = j + e < n ? x[j + e] : 0.f;
    }
    uint32_t w[3][4];
    float odd = 0.f;                     // NaN if a value is not finite
#pragma unroll
    for (int e = 0; e < 8; ++e) odd = fmaf(v[e], 0.f, odd);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float r[2], q[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float f = v[e + 4 * k];
            r[k] = f - __uint_as_float(__float_as_uint(f) & 0xffff0000u);
            q[k] = r[k] - __uint_as_float(__float_as_uint(r[k]) & 0xffff0000u);
        }
        // the upper halves of two words
        w[0][e] = __byte_perm(__float_as_uint(v[e]), __float_as_uint(v[e + 4]), 0x7632);
        w[1][e] = __byte_perm(__float_as_uint(r[0]), __float_as_uint(r[1]), 0x7632);
        w[2][e] = __byte_perm(__float_as_uint(q[0]), __float_as_uint(q[1]), 0x7632);
    }
    if (odd != odd) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t mask = e < 4 ? 0xffff0000u : 0x0000ffffu;         // of the other value of the word
            if (v[e] != v[e]) w[0][e & 3] = (w[0][e & 3] & mask) | (0x7fc07fc0u & ~mask);   // a NaN stays one
            if (!isfinite(v[e])) {
                w[1][e & 3] &= mask;
                w[2][e & 3] &= mask;
            }
        }
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) out[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

// (v & 0x000f000f) | magic as one instruction: as an expression it is two.
__device__ __forceinline__ uint32_t nibbles(uint32_t v, uint32_t magic)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(v), "n"(0x000f000f), "r"(magic));
    return r;
}
__device__ __forceinline__ uint4 ld16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld4(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// After a wait ran out: the copies of a warp's ring that are under way have ended, from the stage in use on.
// (A call, so that the loop that it is left from keeps its registers.)
__device__ __noinline__ void land(uint32_t bar, int use, uint32_t parity, uint32_t limit)
{
    ran_out = 1;
    for (int i = 0; i < STAGES; ++i) {
        int last = 0;
        bar_wait(bar + 8 * use, parity, &last, limit);
        if (++use == STAGES) {
            use = 0;
            parity ^= 1;
        }
    }
    __syncwarp();
}

// One block takes groups of rows in turn; each warp streams stages of weights
// through its own ring of shared memory, a tiled copy (TMA) a stage, with no
// block-wide wait, against x in shared memory: all of it, laid out once, or,
// where it does not fit, a phase at a time.  S16: scales of 16 bits; FINE: groups
// of 32 or 64 columns.  A warp whose wait runs out fetches no more and leaves NaN.
// One token, 4096 x 11008, fp32: 12.3 us for 24 MB, whose copies alone would take 3.5.
// Bound by the warps' instructions, half of which turn codes into numbers, and, with a
// start and a join of 4 us, by latency.  (bf16 x, a column of the instruction instead of
// three of the same eight, takes 12.6.)
template <class T, bool S16, int NT, int RT, bool FINE>
__global__ void __launch_bounds__(MMA_NT, 1) k_w4_mma(W4 A, Cut C, const __grid_constant__ CUtensorMap map)
{
    using P = Piece<T>;
    using H = Half2<typename P::type>;
    constexpr int STEP = STEP_V<RT>, ROWB = STEP / 2, WORDS = STEP / 32;
    constexpr int RED = RT * 16 * NT * 8;                                    // floats of a warp's sums
    extern __shared__ unsigned char raw[];
    unsigned char *const sm = raw + (-smem_addr(raw) & 1023u);               // (the swizzle counts from 1024-byte boundaries)
    __shared__ __align__(8) uint64_t bars[MMA_W * STAGES];
    __shared__ int stop;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int wk = warp & (C.wk - 1), wr = warp / C.wk, wrs = MMA_W / C.wk;
    const uint32_t ring = smem_addr(sm + warp * STAGES * STAGE), bar = smem_addr(bars + warp * STAGES);
    uint4 *const none = (uint4 *)(sm + MMA_W * STAGES * STAGE);              // 16 bytes of zeros
    float *const red = (float *)(none + 8);                                  // (128 bytes on)
    uint4 *const xs = (uint4 *)(red + (C.wk > 1 || P::parts > 1 ? MMA_W * RED : 0));
    const int64_t t0 = (int64_t)blockIdx.y * (NT * 8 / P::parts);            // the pass's first token
    const int64_t left = A.tokens - t0;
    const int tokens = (int)(left < NT * 8 / P::parts ? left : NT * 8 / P::parts), cols = tokens * P::parts;
    const T *x = (const T *)A.x + t0 * A.x_stride;
    const bool wide = aligned_x(x, A.x_stride);
    const int last_group = (int)((A.n - 1) >> C.shift);
    const uint32_t magic = C.magic;                                          // H::magic, from a register
    const uint32_t per = FINE ? (1u << C.shift) / 32u : 4u;                  // words of a group (or of half of one)

    if (threadIdx.x == 0) {
        for (int i = 0; i < MMA_W * STAGES; ++i) bar_init(smem_addr(bars + i), 1);
        stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x < 8) none[threadIdx.x] = make_uint4(0, 0, 0, 0);
    __syncthreads();

    // The stages to fetch run ahead of the stages in use, across groups of rows.
    int64_t fg = wk < C.steps ? blockIdx.x : C.groups;
    int fs = wk, slot = 0;
    auto fetch = [&]() {
        if (fg < C.groups) {
            if (elected()) {
                bar_expect(bar + 8 * slot, STAGE + vain_bytes(A.waits));
                stage_load(ring + slot * STAGE, &map, fs * ROWB, (int)((fg * wrs + wr) * (16 * RT)), bar + 8 * slot);
            }
            fs += C.wk;
            if (fs >= C.steps) {
                fs = wk;
                fg += gridDim.x;
            }
        }
        slot = slot + 1 == STAGES ? 0 : slot + 1;
    };
    // Scales and zero points, of rows g and g + 8 of a row tile, lie in the four
    // lanes that share those rows and two sets of registers.
    //   FINE: of one stage; word j in lane j % 4, set j / 4 (RT = 1) or of row
    //   tile `set` (RT = 2);
    //   else a stage has one group (RT = 2) or two (RT = 1, its halves), and they
    //   are read for four of the warp's stages at once: stage k in lane k, set =
    //   row tile; or in lane 2 (k % 2) + half, set k / 2.
    // (Offsets fit 32 bits: the launch sees to it.)
    constexpr int ROUND = FINE ? 1 : 4;
    float sn[2][2];
    uint32_t zn[2][2], so[2][2], zo[2][2];
    auto constants_from = [&](int64_t grp) {
        const int64_t row0 = (grp * wrs + wr) * (16 * RT) + g;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int64_t row = row0 + (RT == 1 ? 0 : 16 * i) + 8 * h;
                row = row < A.m ? row : A.m - 1;
                so[i][h] = (uint32_t)(row * A.scale_stride);
                zo[i][h] = (uint32_t)(row * A.zero_stride);
            }
    };
    auto constants = [&](int st) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int col = FINE      ? st * STEP + 32 * (t4 + (RT == 1 ? 4 * i : 0))
                            : RT == 2 ? (st + t4 * C.wk) * STEP
                                      : (st + (2 * i + (t4 >> 1)) * C.wk) * STEP + 128 * (t4 & 1);
            int gi = col >> C.shift;
            gi = gi < last_group ? gi : last_group;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (S16) {
                    const uint16_t u = ((const uint16_t *)A.scales)[so[i][h] + (uint32_t)gi];
                    sn[i][h] = __uint_as_float(u);
                } else {
                    sn[i][h] = ((const float *)A.scales)[so[i][h] + (uint32_t)gi];
                }
                zn[i][h] = A.zeros ? A.zeros[zo[i][h] + (uint32_t)gi] : 8u;
            }
        }
    };
    // x of a phase: piece (32-column block, column of B, quarter) at
    // [block][column][quarter], 16 bytes each
    auto stage_x = [&](int p0, int p1) {
        const int quarters = (p1 - p0) * (STEP / 8);
        for (int k = threadIdx.x; k < quarters; k += MMA_NT) {
            uint4 *to = xs + (k >> 2) * cols * 4 + (k & 3);
            const T *from = x;
            for (int tok = 0; tok < tokens; tok += 2) {
                uint4 v[2][P::parts];
                lay_out(from, (int64_t)p0 * STEP + 8 * k, A.n, wide, v[0]);
                if (tok + 1 < tokens) lay_out(from + A.x_stride, (int64_t)p0 * STEP + 8 * k, A.n, wide, v[1]);
                from += 2 * A.x_stride;
#pragma unroll
                for (int p = 0; p < P::parts; ++p) {
                    to[4 * p] = v[0][p];
                    if (tok + 1 < tokens) to[4 * (P::parts + p)] = v[1][p];
                }
                to += 8 * P::parts;
            }
        }
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch();
    if (wk < C.steps && blockIdx.x < C.groups) {
        constants_from(blockIdx.x);
        constants(wk);
    }

    // this lane's pieces of B: column 8 c + g of each block, or zeros
    uint32_t step_b[NT], from[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const bool in = 8 * c + g < cols;
        from[c] = (uint32_t)__cvta_generic_to_shared(in ? xs + (8 * c + g) * 4 + t4 : none);
        step_b[c] = in ? cols * 64 : 0;
    }

    uint32_t at_word[WORDS];                                                 // of this lane's word of each 32 columns in a stage
#pragma unroll
    for (int j = 0; j < WORDS; ++j) at_word[j] = g * ROWB + 4 * t4 + ((j ^ (RT == 1 ? g : g >> 1 & 3)) << 4);
    int use = 0;
    uint32_t parity = 0;
    bool have = false, ok = true;
    for (int64_t grp = blockIdx.x; grp < C.groups; grp += gridDim.x) {
        float tot[RT][NT][4] = {}, sc[2][2];
        uint32_t zc[2][2];
        int turn = 0;
        for (int p0 = 0; p0 < C.steps; p0 += C.phase) {
            const int p1 = p0 + C.phase < C.steps ? p0 + C.phase : C.steps;
            if (!have || C.phase < C.steps) {
                if (have) __syncthreads();
                stage_x(p0, p1);
                __syncthreads();
                have = true;
            }
            // phases are whole turns of the warps, so turns go on across them
            for (int st = p0 + wk; st < p1; st += C.wk) {
                if (FINE || (turn & 3) == 0) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t u = __float_as_uint(sn[i][h]);
                            sc[i][h] = !S16 ? sn[i][h] : C.bf16_scales ? __uint_as_float(u << 16) : __half2float(__ushort_as_half((uint16_t)u));
                            zc[i][h] = H::magic + (zn[i][h] & 127u) * H::one;
                        }
                    if (st + ROUND * C.wk < C.steps) {
                        constants(st + ROUND * C.wk);
                    } else if (grp + gridDim.x < C.groups) {
                        constants_from(grp + gridDim.x);
                        constants(wk);
                    }
                }
                const int k4 = turn++ & 3;
                fetch();
                if (ok && !__all_sync(~0u, bar_wait(bar + 8 * use, parity, &stop, A.waits.limit))) {
                    ok = false;
                    fg = C.groups;                       // nothing more is fetched
                    land(bar, use, parity, A.waits.limit);
                }
                const uint32_t w = ring + use * STAGE;
                if (++use == STAGES) {
                    use = 0;
                    parity ^= 1;
                }
                uint32_t bx[NT];
#pragma unroll
                for (int c = 0; c < NT; ++c) bx[c] = from[c] + (st - p0) * WORDS * step_b[c];
                float part[RT][NT][4] = {};
                uint32_t za[RT] = {}, zb[RT] = {};
#pragma unroll
                for (int j = 0; j < WORDS; ++j) {
                    const int src = (lane & ~3) | (FINE ? j & 3 : RT == 2 ? k4 : 2 * (k4 & 1) + (j >> 2));
                    uint4 b[NT];
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        b[c] = ld16(bx[c]);
                        bx[c] += step_b[c];
                    }
                    const bool begins = FINE ? (j & (per - 1)) == 0 : (j & 3) == 0, ends = FINE ? ((j + 1) & (per - 1)) == 0 : (j & 3) == 3;
                    if (begins) {
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const bool second = FINE ? j >> 2 : RT == 1 ? k4 >> 1 : false;
                            za[r] = __shfl_sync(~0u, RT == 2 ? zc[r][0] : second ? zc[1][0] : zc[0][0], src);
                            zb[r] = __shfl_sync(~0u, RT == 2 ? zc[r][1] : second ? zc[1][1] : zc[0][1], src);
#pragma unroll
                            for (int c = 0; c < NT; ++c)
#pragma unroll
                                for (int e = 0; e < 4; ++e) part[r][c][e] = 0.f;
                        }
                    }
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const uint32_t wa = ld4(w + at_word[j] + r * 16 * ROWB), wb = ld4(w + at_word[j] + (r * 16 + 8) * ROWB);
                        uint32_t a[4];
                        a[0] = H::sub(nibbles(wa, magic), za[r]);
                        a[1] = H::sub(nibbles(wb, magic), zb[r]);
                        a[2] = H::sub(nibbles(wa >> 4, magic), za[r]);
                        a[3] = H::sub(nibbles(wb >> 4, magic), zb[r]);
#pragma unroll
                        for (int c = 0; c < NT; ++c) H::mma(part[r][c], a, b[c].x, b[c].y);
                        a[0] = H::sub(nibbles(wa >> 8, magic), za[r]);
                        a[1] = H::sub(nibbles(wb >> 8, magic), zb[r]);
                        a[2] = H::sub(nibbles(wa >> 12, magic), za[r]);
                        a[3] = H::sub(nibbles(wb >> 12, magic), zb[r]);
#pragma unroll
                        for (int c = 0; c < NT; ++c) H::mma(part[r][c], a, b[c].z, b[c].w);
                    }
                    if (ends) {
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const bool second = FINE ? j >> 2 : RT == 1 ? k4 >> 1 : false;
                            const float sa = __shfl_sync(~0u, RT == 2 ? sc[r][0] : second ? sc[1][0] : sc[0][0], src);
                            const float sb = __shfl_sync(~0u, RT == 2 ? sc[r][1] : second ? sc[1][1] : sc[0][1], src);
#pragma unroll
                            for (int c = 0; c < NT; ++c) {
                                tot[r][c][0] = fmaf(sa, part[r][c][0], tot[r][c][0]);
                                tot[r][c][1] = fmaf(sa, part[r][c][1], tot[r][c][1]);
                                tot[r][c][2] = fmaf(sb, part[r][c][2], tot[r][c][2]);
                                tot[r][c][3] = fmaf(sb, part[r][c][3], tot[r][c][3]);
                            }
                        }
                    }
                }
                __syncwarp();
            }
        }
        if (!ok)
#pragma unroll
            for (int e = 0; e < RT * NT * 4; ++e) (&tot[0][0][0])[e] = nanf("");
        if (C.wk == 1 && P::parts == 1) {
            // the warp has its rows' whole sums
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int64_t row = (grp * wrs + wr) * (16 * RT) + 16 * r + g + (e >> 1) * 8;
                        const int tok = 8 * c + 2 * t4 + (e & 1);
                        if (tok < tokens && row < A.m) ((T *)A.y)[(t0 + tok) * A.y_stride + row] = from_f32<T>(tot[r][c][e] * H::unit);
                    }
            continue;
        }
        // sums of the warps of a row tile and of the pieces of a token, in order
        float *mine = red + warp * RED;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                // [column][row]
                float *d = mine + (8 * c + 2 * t4) * (RT * 16) + 16 * r + g;
                d[0] = tot[r][c][0];
                d[RT * 16] = tot[r][c][1];
                d[8] = tot[r][c][2];
                d[RT * 16 + 8] = tot[r][c][3];
            }
        __syncthreads();
        const int rows = wrs * RT * 16;
        for (int i = threadIdx.x; i < rows * tokens; i += MMA_NT) {
            const int tok = i / rows, rr = i - tok * rows, wr2 = rr / (RT * 16), r = rr % (RT * 16);
            const int64_t row = grp * rows + rr;
            const float *f = red + wr2 * C.wk * RED + tok * P::parts * (RT * 16) + r;
            float v = 0.f;
#pragma unroll 4
            for (int k = 0; k < C.wk; ++k)
#pragma unroll
                for (int p = 0; p < P::parts; ++p) v += f[k * RED + p * (RT * 16)];
            if (row < A.m) ((T *)A.y)[(t0 + tok) * A.y_stride + row] = from_f32<T>(v * H::unit);
        }
        __syncthreads();
    }
}

constexpr int SMEM_MAX = 226 * 1024;      // (and the barriers)

template <class T, bool S16, int NT, int RT, bool FINE>
dbs_status launch_mma(const W4 &A, dbs_dtype sd, const CUtensorMap &map, cudaStream_t s)
{
    constexpr int parts = Piece<T>::parts, pass = NT * 8 / parts, STEP = STEP_V<RT>;
    constexpr int ring = MMA_W * STAGES * STAGE + 128, red = MMA_W * RT * 16 * NT * 8 * 4;
    static Once once;
    const int sms = multiprocessors();
    if (sms == 0 || !room_for(once, k_w4_mma<T, S16, NT, RT, FINE>, SMEM_MAX)) return DBS_ERR_CUDA;
    Cut C{};
    C.steps = (int)((A.n + STEP - 1) / STEP);
    C.bf16_scales = sd == DBS_BF16;
    C.magic = Half2<typename Piece<T>::type>::magic;
    while (1 << C.shift < A.group) ++C.shift;
    const int step_bytes = STEP * (int)((A.tokens < pass ? A.tokens : pass) * parts) * 2;
    // Warps per row tile: the time of a block, counted in instructions of a
    // warp: rounds of (its stages, about 300 + 64 NT for each row tile; the join
    // of the warps' sums; laying out x again, if it does not fit at once, about
    // 30 for 16 bytes of a piece).
    double best = 0;
    int smem = 0;
    for (int wk = 1; wk <= MMA_W; wk *= 2) {
        const int room = SMEM_MAX - 1024 - ring - (wk > 1 || parts > 1 ? red : 0);
        int phase = room / step_bytes;
        if (phase >= C.steps) phase = C.steps;
        else phase = phase / wk * wk;
        if (phase < 1) continue;
        const int rows = MMA_W / wk * RT * 16;
        const int64_t groups = (A.m + rows - 1) / rows, rounds = (groups + sms - 1) / sms;
        const double stages = (C.steps + wk - 1) / wk * (300. + 64 * NT) , join = wk > 1 ? 100. + 10 * NT * RT * wk : 60.;
        const double lay = (double)C.steps * step_bytes / 16 / parts / MMA_NT * 30;
        const double cost = rounds * (stages + join + (phase < C.steps ? lay + 1000. * ((C.steps + phase - 1) / phase) : 0.)) + lay;
        if (smem == 0 || cost < best) {
            best = cost;
            C.wk = wk;
            C.phase = phase;
            C.groups = groups;
            smem = 1024 + ring + (wk > 1 || parts > 1 ? red : 0) + phase * step_bytes;
        }
    }
    const int64_t grid = C.groups < sms ? C.groups : sms;
    const int64_t passes = (A.tokens + pass - 1) / pass;
    W4 B = A;
    for (int64_t p = 0; p < passes; p += 32768) {
        const int64_t now = passes - p < 32768 ? passes - p : 32768;
        B.x = (const T *)A.x + p * pass * A.x_stride;
        B.y = (T *)A.y + p * pass * A.y_stride;
        B.tokens = A.tokens - p * pass;
        k_w4_mma<T, S16, NT, RT, FINE><<<dim3((unsigned)grid, (unsigned)now), MMA_NT, smem, s>>>(B, C, map);
    }
    return launched();
}

// ---- many rows and several tokens: tcgen05 ----
//
// 128 rows of codes and N columns of x (tokens) on the fifth-generation tensor
// cores: the codes' numbers, made as above, go from registers into tensor memory (a
// row a lane, two numbers a column), x into shared memory in the 128-byte swizzle,
// and the sums of each group, in tensor memory, come back to be scaled in fp32.
// Warps have roles: two or three fours make numbers, half a chunk of 256 columns at
// a time; four scale (a thread a row); four bring x's columns into the order of the
// numbers, in place; one fetches codes and one x, by tiled copies; one issues the
// products.  Fours of warps that need few registers leave theirs to those that scale.
//
// 24 tokens, 128000 x 4096: 92.5 us, against 150 with k_w4_mma, whose warps spend their
// instructions on fragments of x.  A block's chunk takes 0.8 us, of which memory
// would take 0.4: the chain of the products' issue and the scaling of their sums
// bounds it (two thirds of the issue slots are used).
template <int N> struct Many {
    static constexpr int MG = N == 32 ? 3 : 2;                               // fours of warps that make numbers
    static constexpr int XS = MG, RA = 2 * MG, WS = 6;                // stages: of x, of numbers (half a chunk), of codes
    static constexpr int CODES = 128 * 128, X = N * 512;                     // bytes of a stage
    static constexpr int SCALE = 4 * MG, LAY = SCALE + 4, FETCH = LAY + 4, ISSUE = FETCH + 2, NT = 32 * (FETCH + 4);
    // registers of a thread: at launch, and after the fours of warps have shared them out
    static constexpr int REGS = MG == 3 ? 80 : 96, FEW = 56, SOME = 64, MANY = REGS + (REGS - FEW) + (REGS - SOME);
    static constexpr int SUMS = 0, NUMBERS = 4 * N;                          // columns of tensor memory
    static constexpr int SMEM = 1024 + WS * CODES + XS * X;
};
static_assert(Many<32>::NUMBERS + Many<32>::RA * 64 <= 512 && Many<64>::NUMBERS + Many<64>::RA * 64 <= 512, "tensor memory");

struct Walk {
    int steps, shift;          // chunks of a row; log2 of the group
    int passes;                // of N tokens
    int units;                 // of 128 rows and N tokens; a block takes every gridDim.x-th, or
    int split;                 // so many blocks, a cluster, one, a part of its columns each
    int scales;                // their type
};

template <class T, int N>
__global__ void __launch_bounds__(Many<N>::NT, 1) k_w4_many(W4 A, Walk C, const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap xmap)
{
    using M = Many<N>;
    using H = Half2<T>;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bars[2 * M::WS + 3 * M::XS + 2 * M::RA + 5];
    __shared__ uint32_t tmem_at;
    __shared__ int stop;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t codes = smem_addr(raw) + (-smem_addr(raw) & 1023u), xs = codes + M::WS * M::CODES;
    const uint32_t w_full = smem_addr(bars), w_empty = w_full + 8 * M::WS, x_full = w_empty + 8 * M::WS, x_empty = x_full + 8 * M::XS;
    const uint32_t a_full = x_empty + 8 * M::XS, a_empty = a_full + 8 * M::RA, d_full = a_empty + 8 * M::RA, d_empty = d_full + 16;
    const uint32_t x_here = d_empty + 16, last_bar = x_here + 8 * M::XS;
    if (threadIdx.x == 0) {
        for (int i = 0; i < M::WS; ++i) {
            bar_init(w_full + 8 * i, 1);
            bar_init(w_empty + 8 * i, 8);
        }
        for (int i = 0; i < M::XS; ++i) {
            bar_init(x_full + 8 * i, 128);
            bar_init(x_empty + 8 * i, 1);
            bar_init(x_here + 8 * i, 1);
        }
        for (int i = 0; i < M::RA; ++i) {
            bar_init(a_full + 8 * i, 4);
            bar_init(a_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(d_full + 8 * i, 1);
            bar_init(d_empty + 8 * i, 4);
        }
        bar_init(last_bar, 1);
        stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == M::ISSUE) tc_alloc(smem_addr(&tmem_at));
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tmem_at;
    const int last_group = (int)((A.n - 1) >> C.shift);
    const int rank = (int)blockIdx.x % C.split, first = (int)blockIdx.x / C.split;
    const int c0 = C.steps * rank / C.split;                                 // of the first unit; the launch sees that all chunks fit an int
    const int chunks = C.split > 1 ? C.steps * (rank + 1) / C.split - c0 : (C.units - first + (int)gridDim.x - 1) / (int)gridDim.x * C.steps;

    // The unit and chunk (or group) that a role is at; a unit's row tile and pass.
    struct At {
        int unit, tile, pass, at;
    };
    auto begin = [&](int each) { return At{first, first / C.passes, first % C.passes, c0 * each}; };        // each: a chunk's share of `at`
    auto step = [&](At &p, int of) {
        if (++p.at < of) return;
        p.at = 0;
        p.unit += gridDim.x;
        p.tile = p.unit / C.passes;
        p.pass = p.unit - p.tile * C.passes;
    };

    // All threads of the cluster.
    auto meet = [&] {
        asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
    };

    if (warp < M::SCALE) {
        // ---- numbers: a thread has a row's 128 codes of half a chunk, the halves in turns ----
        const int r = threadIdx.x & 127;
        const int parts = C.shift == 5 ? 4 : C.shift == 6 ? 2 : 1;           // groups among them
        At ahead = begin(2);                                                 // (in halves)
        auto skip = [&](int by) {
            ahead.at += by;
            while (ahead.at >= 2 * C.steps) {
                ahead.at -= 2 * C.steps;
                ahead.unit += gridDim.x;
                ahead.tile = ahead.unit / C.passes;
            }
        };
        uint32_t zn[4] = {8, 8, 8, 8};                                       // zero points of the next half
        auto zero_points = [&] {
            if (A.zeros && ahead.unit < C.units) {
                const int64_t row = (int64_t)ahead.tile * 128 + r;
                const uint8_t *from = A.zeros + (row < A.m ? row : A.m - 1) * A.zero_stride;
                const int g = ahead.at * 128 >> C.shift;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < parts) zn[i] = from[g + i < last_group ? g + i : last_group];
            }
            skip(M::MG);
        };
        skip(warp >> 2);
        zero_points();
        const uint32_t to = tmem + ((uint32_t)(warp & 3) << 21) + M::NUMBERS;
        int ws = warp >> 3, as = warp >> 2;
        uint32_t wp = 0, ap = 1;
        bool ok = true;
#pragma unroll 1
        for (int u = warp >> 2; u < 2 * chunks && ok; u += M::MG) {
            uint32_t z[4];                                                   // as numbers, of 32 codes each
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = H::magic + ((parts == 4 ? zn[i] : parts == 2 ? zn[i >> 1] : zn[0]) & 127u) * H::one;
            zero_points();
            ok = __all_sync(~0u, bar_wait(w_full + 8 * ws, wp, &stop, A.waits.limit));
            if (!ok) break;                              // (codes that have not come are not given back)
            const int half = u & 1;
            uint4 q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = ld16(codes + ws * M::CODES + r * 128 + (((half * 4 + i) ^ (r & 7)) << 4));
            __syncwarp();
            if (lane == 0) bar_arrive(w_empty + 8 * ws);
            ws += ((u + M::MG) >> 1) - (u >> 1);
            if (ws >= M::WS) {
                ws -= M::WS;
                wp ^= 1;
            }
            ok = __all_sync(~0u, bar_wait(a_empty + 8 * as, ap, &stop, A.waits.limit));
            if (!ok) break;
            tc_after();
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint32_t out[32];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w[4] = {q[2 * p + i].x, q[2 * p + i].y, q[2 * p + i].z, q[2 * p + i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int b = 0; b < 4; ++b) out[16 * i + 4 * e + b] = H::sub(nibbles(w[e] >> 4 * b, H::magic), z[2 * p + i]);
                }
                tc_st(to + as * 64 + 32 * p, out);
            }
            tc_wait_st();
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(a_full + 8 * as);
            if ((as += M::MG) >= M::RA) {
                as -= M::RA;
                ap ^= 1;
            }
        }
    } else if (warp < M::LAY) {
        // ---- groups' sums, scaled: a thread has a row ----
        more_registers<M::MANY>();
        // (a set of sums: two neighbouring groups, or one of 256 columns)
        const int r = threadIdx.x & 127, two = C.shift < 8 ? 2 : 1, of = C.steps * (256 >> C.shift) / two;
        At ahead = begin(of / C.steps), now = ahead;
        auto row_of = [&](const At &p) {
            const int64_t row = (int64_t)p.tile * 128 + r;
            return row < A.m ? row : A.m - 1;
        };
        int64_t from = row_of(ahead) * A.scale_stride;
        uint32_t sn[2] = {};                                                 // scales of the next set
        auto scales = [&] {
            if (ahead.unit < C.units) {
                if (ahead.at == 0) from = row_of(ahead) * A.scale_stride;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int g = ahead.at * two + i;
                    if (i < two && g <= last_group) sn[i] = C.scales == DBS_F32 ? ((const uint32_t *)A.scales)[from + g] : ((const uint16_t *)A.scales)[from + g];
                    else sn[i] = 0;                                          // (behind the row's end, where the sums are 0)
                }
            }
            step(ahead, of);
        };
        scales();
        float acc[N] = {};
        bool ok = true;
        const int all = chunks * (of / C.steps);
        auto store = [&](const At &p) {
            const int64_t row = (int64_t)p.tile * 128 + r, t0 = (int64_t)p.pass * N;
            T *y = (T *)A.y + t0 * A.y_stride + row;
#pragma unroll
            for (int t = 0; t < N; ++t) {
                if (t0 + t < A.tokens && row < A.m) *y = from_f32<T>(ok ? acc[t] * H::unit : nanf(""));
                y += A.y_stride;
            }
        };
#pragma unroll 1
        for (int g = 0; g < all; ++g) {
            ok = ok && __all_sync(~0u, bar_wait(d_full + 8 * (g & 1), g >> 1 & 1, &stop, A.waits.limit));
            if (ok) {
                tc_after();
                const uint32_t sums = tmem + ((uint32_t)(warp & 3) << 21) + M::SUMS + (g & 1) * (2 * N);
                uint32_t part[32];
                tc_ld_begin(part, sums);
                float f[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) f[i] = C.scales == DBS_F32 ? __uint_as_float(sn[i]) : C.scales == DBS_BF16 ? __uint_as_float(sn[i] << 16) : __half2float(__ushort_as_half((uint16_t)sn[i]));
                scales();
#pragma unroll
                for (int t = 0; t < 2 * N; t += 32) {
                    if (t == N && two == 1) break;
                    tc_ld_end(part);
#pragma unroll
                    for (int e = 0; e < 32; ++e) acc[t % N + e] = fmaf(f[t / N], __uint_as_float(part[e]), acc[t % N + e]);
                    if (t + 32 < 2 * N && (two == 2 || t + 32 < N)) tc_ld_begin(part, sums + t + 32);
                }
                tc_before();
                __syncwarp();
                if (lane == 0) bar_arrive(d_empty + 8 * (g & 1));
            }
            if (C.split == 1 && now.at == of - 1) {
                store(now);
#pragma unroll
                for (int t = 0; t < N; ++t) acc[t] = 0.f;
            }
            step(now, of);
        }
        if (C.split > 1) {
            // the parts of the columns, in order, in the first block's shared memory
            meet();
            const uint32_t at = codes + r * 16;
            if (!ok)
#pragma unroll
                for (int t = 0; t < N; ++t) acc[t] = nanf("");
            if (rank > 0) {
                uint32_t to;
                asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(at + (rank - 1) * (N * 512)));
#pragma unroll
                for (int t = 0; t < N; t += 4)
                    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(to + t * 512), "f"(acc[t]), "f"(acc[t + 1]), "f"(acc[t + 2]),
                                 "f"(acc[t + 3]) : "memory");
            }
            meet();
            if (rank == 0) {
                for (int i = 0; i < C.split - 1; ++i)
#pragma unroll
                    for (int t = 0; t < N; t += 4) {
                        const uint4 v = ld16(at + i * (N * 512) + t * 512);
                        acc[t] += __uint_as_float(v.x);
                        acc[t + 1] += __uint_as_float(v.y);
                        acc[t + 2] += __uint_as_float(v.z);
                        acc[t + 3] += __uint_as_float(v.w);
                    }
                store(begin(0));
            }
        }
    } else if (warp < M::FETCH) {
        // ---- x: pairs of its columns in their places ----
        fewer_registers<M::SOME>();
        int st = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (int n = 0; n < chunks && ok; ++n) {
            ok = __all_sync(~0u, bar_wait(x_here + 8 * st, parity, &stop, A.waits.limit));
            if (!ok) break;
            const uint32_t at = xs + st * M::X + (threadIdx.x & 127) * 16;
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < N / 4; i += 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = ld16(at + (i + e) * 2048);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint4 u = paired(v[e]);
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + (i + e) * 2048), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w) : "memory");
                }
            }
            async_fence();
            bar_arrive(x_full + 8 * st);
            if (++st == M::XS) {
                st = 0;
                parity ^= 1;
            }
        }
    } else if (fewer_registers<M::FEW>(), warp < M::ISSUE) {
        // ---- fetch: one warp codes, one x; tiled copies a chunk ----
        const bool is_x = warp > M::FETCH;
        const int stages = is_x ? M::XS : M::WS, bytes = is_x ? M::X : M::CODES;
        const uint32_t full = is_x ? x_here : w_full, empty = is_x ? x_empty : w_empty, store = is_x ? xs : codes;
        At p = begin(1);
        int st = 0, fetched = 0;
        uint32_t parity = 1;
        for (int n = 0; n < chunks; ++n) {
            if (!__all_sync(~0u, bar_wait(empty + 8 * st, parity, &stop, A.waits.limit))) break;
            if (elected()) {
                bar_expect(full + 8 * st, bytes + vain_bytes(A.waits));
                if (is_x) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) stage_load(store + st * bytes + i * (N * 128), &xmap, p.at * 256 + 64 * i, p.pass * N, full + 8 * st);
                } else {
                    stage_load(store + st * bytes, &map, p.at * 128, p.tile * 128, full + 8 * st);
                }
            }
            __syncwarp();
            step(p, C.steps);
            if (++st == stages) {
                st = 0;
                parity ^= 1;
            }
            fetched = n + 1;
        }
        // copies under way end before their memory is given back, or taken for sums of other blocks
        for (int n = fetched > stages ? fetched - stages : 0; n < fetched; ++n) {
            int last = 0;
            bar_wait(full + 8 * (n % stages), n / stages & 1, &last, A.waits.limit);
        }
    } else if (warp == M::ISSUE) {
        // ---- products ----
        constexpr uint32_t FMT = __is_same(T, __nv_bfloat16) ? 1u : 0u;
        constexpr uint32_t DESC = 1u << 4 | FMT << 7 | FMT << 10 | (uint32_t)(N >> 3) << 17 | (128u >> 4) << 24;
        int q = 0;
        bool ok = true;
        // LEN: instructions of a group, at most those of half a chunk.  A turn goes
        // once through all stages of x and of numbers, so that the descriptors are
        // sums of constants.  (Tensor memory begins at 0: the block has all of it.)
        auto issue = [&](auto length) {
            constexpr int LEN = decltype(length)::value;
            uint32_t turn = 0;
            for (int n0 = 0; n0 < chunks && ok; n0 += M::XS, turn ^= 1) {
#pragma unroll
                for (int u = 0; u < 2 * M::XS; ++u) {
                    const int half = u & 1;
                    if (n0 + u / 2 >= chunks) break;
                    if (half == 0) ok = ok && __all_sync(~0u, bar_wait(x_full + 8 * (u / 2), turn, &stop, A.waits.limit));
                    ok = ok && __all_sync(~0u, bar_wait(a_full + 8 * u, turn, &stop, A.waits.limit));
                    const uint32_t lo = (xs + u / 2 * M::X + half * (2 * N * 128)) >> 4 | 1u << 16, a = M::NUMBERS + u * 64;
                    uint64_t b[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) b[k] = desc_of(lo + ((k >> 2) * (N * 128) + (k & 3) * 32) / 16);
#pragma unroll
                    for (int k0 = 0; k0 < 8; k0 += LEN) {
                        // the group's place in its set, and whether the set begins or ends here
                        const bool second = LEN == 8 ? half == 1 && C.shift < 8 : k0 / LEN & 1;
                        const bool begins = LEN == 8 ? half == 0 : !second, ends = LEN == 8 ? half == 1 : second;
                        if (begins) ok = ok && __all_sync(~0u, bar_wait(d_empty + 8 * (q & 1), (q >> 1 & 1) ^ 1, &stop, A.waits.limit));
                        if (!ok) break;
                        tc_after();
                        const uint32_t d = M::SUMS + (q & 1) * (2 * N) + (second ? N : 0), full = d_full + 8 * (q & 1);
                        const bool more = LEN == 8 && half == 1 && !second;  // (a group of 256 goes on)
                        if (elected()) {
#pragma unroll
                            for (int k = k0; k < k0 + LEN; ++k) tc_mma_ts(d, a + 8 * k, b[k], DESC, k > k0 || more);
                            if (ends) tc_commit(full);
                            if (k0 + LEN == 8) {
                                tc_commit(a_empty + 8 * u);
                                if (half == 1) tc_commit(x_empty + 8 * (u / 2));
                            }
                        }
                        if (ends) ++q;
                        __syncwarp();
                    }
                }
            }
        };
        if (C.shift >= 7) issue(std::integral_constant<int, 8>());
        else if (C.shift == 6) issue(std::integral_constant<int, 4>());
        else issue(std::integral_constant<int, 2>());
        // the instructions under way, before tensor memory is given back
        if (elected()) tc_commit(last_bar);
        __syncwarp();
        int last = 0;
        bar_wait(last_bar, 0, &last, A.waits.limit);
    }
    if (C.split > 1 && (warp < M::SCALE || warp >= M::LAY)) {
        __syncwarp();
        meet();
        meet();
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    if (warp == M::ISSUE) {
        tc_after();
        tc_free(tmem);
    }
    if (threadIdx.x == 0 && stop) ran_out = 1;
}

// The weights as rows of bytes, in stages of `columns` bytes of `rows` rows.
bool make_map(const W4 &A, int columns, int rows, CUtensorMap &map)
{
    const encode_tiled_fn encode = encode_tiled();
    const int64_t bytes = (A.n + 1) / 2, stride = A.m == 1 ? (bytes + 15) / 16 * 16 : A.q_stride;
    if (!encode || stride < bytes || stride >= int64_t(1) << 40) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)A.m}, strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {(cuuint32_t)columns, (cuuint32_t)rows}, ones[2] = {1, 1};
    return encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(A.q), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  columns == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// x (of 16 bits) in boxes of 64 columns of `rows` tokens.
bool make_x_map(const W4 &A, int rows, CUtensorMap &map)
{
    const encode_tiled_fn encode = encode_tiled();
    const int64_t stride = A.tokens == 1 ? (2 * A.n + 15) / 16 * 16 : 2 * A.x_stride;
    if (!encode || !aligned16(A.x) || (stride & 15) != 0 || stride < 2 * A.n || stride >= int64_t(1) << 40) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)A.n, (cuuint64_t)A.tokens}, strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {64, (cuuint32_t)rows}, ones[2] = {1, 1};
    return encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(A.x), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// From 13 tokens of 16-bit x on, where x's rows are on 16-byte boundaries: k_w4_mma takes
// a matrix instruction for each eight tokens, this one the same time up to 32.  k_w4_mma
// and this one, us, bf16, groups of 128, zeros:
//                   8 tokens       12          13          16          24
//    4096 x 11008  20.8  18.6   24.5  18.6   35.1  18.7   37.3  18.7   98   18.7
//   11008 x  4096  16.6  18.8   18.7  18.8   23.0  18.8   24.8  18.7   41   18.7
//   32000 x  4096  25.2  33.3   30.0  33.3   34.7  33.3   35.7  33.3   58   33.3
//  128000 x  4096  74.8  93.9   87.9  94.1   89.1  93.6   90.2  93.7  150   93.8
// So the right place is between 5 tokens and 16, later for more rows; 13 costs at most 32%
// (4096 rows, 12 tokens) and 5% (128000 rows, 13).
constexpr int64_t MANY_TOKENS = 12;

struct Tall {
    CUtensorMap codes, x;
    Walk walk;
};
// How such a call is cut up; false if it does not fit.
template <int N>
bool plan_many(const W4 &A, dbs_dtype sd, int sms, Tall &t)
{
    const int64_t passes = (A.tokens + N - 1) / N, units = (A.m + 127) / 128 * passes, steps = (A.n + 255) / 256;
    // (counts of groups of 32 columns of a block, and of columns, are ints)
    if (passes >= int64_t(1) << 31 || units >= int64_t(1) << 31 || (units / sms + 1) * steps >= int64_t(1) << 27) return false;
    if (!make_map(A, 128, 128, t.codes) || !make_x_map(A, N, t.x)) return false;
    t.walk = {(int)steps, 0, (int)passes, (int)units, 1, sd};
    while (1 << t.walk.shift < A.group) ++t.walk.shift;
    // few units: blocks of a cluster share one's columns (4096 x 11008, 24 tokens: 18.7
    // us with four, 39.1 with one)
    while (t.walk.split < (N == 32 ? 8 : 4) && units * 2 * t.walk.split <= sms && steps >= 4 * t.walk.split) t.walk.split *= 2;
    return true;
}
template <class T, int N>
dbs_status launch_many(const W4 &A, const Tall &t, int sms, cudaStream_t s)
{
    static Once once;
    if (!room_for(once, k_w4_many<T, N>, Many<N>::SMEM, false, Many<N>::REGS)) return DBS_ERR_CUDA;
    const Walk &w = t.walk;
    cudaLaunchConfig_t how{};
    how.gridDim = dim3((unsigned)(w.split > 1 ? w.units * w.split : w.units < sms ? w.units : sms));
    how.blockDim = dim3(Many<N>::NT);
    how.dynamicSmemBytes = Many<N>::SMEM;
    how.stream = s;
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = (unsigned)w.split;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    how.attrs = &cluster;
    how.numAttrs = 1;
    cudaLaunchKernelEx(&how, k_w4_many<T, N>, A, w, t.codes, t.x);
    return launched();
}

template <class T, bool S16, int NT, int RT>
dbs_status launch_tiles(const W4 &A, dbs_dtype sd, const CUtensorMap &map, cudaStream_t s)
{
    return A.group < 128 ? launch_mma<T, S16, NT, RT, true>(A, sd, map, s) : launch_mma<T, S16, NT, RT, false>(A, sd, map, s);
}

template <class T, bool S16>
dbs_status launch_cols(const W4 &A, dbs_dtype sd, const CUtensorMap &map, cudaStream_t s)
{
    const int64_t cols = A.tokens * Piece<T>::parts;             // of B, in eights
    return cols <= 8 ? launch_tiles<T, S16, 1, 1>(A, sd, map, s) : cols <= 16 ? launch_tiles<T, S16, 2, 2>(A, sd, map, s)
           : cols <= 24 ? launch_tiles<T, S16, 3, 2>(A, sd, map, s) : launch_tiles<T, S16, 4, 2>(A, sd, map, s);
}

template <class T, class S>
dbs_status launch(const W4 &A, dbs_dtype sd, cudaStream_t s)
{
    constexpr int64_t LIMIT = int64_t(1) << 32;
    const bool rows16 = A.n > 0 && aligned16(A.q) && (A.q_stride & 15) == 0;
    if constexpr (sizeof(T) == 2)
        if (rows16 && A.tokens > MANY_TOKENS) {
            Tall t;
            const int sms = multiprocessors();
            if (sms == 0) return DBS_ERR_CUDA;
            if (A.tokens <= 32 && plan_many<32>(A, sd, sms, t)) return launch_many<T, 32>(A, t, sms, s);
            if (A.tokens > 32 && plan_many<64>(A, sd, sms, t)) return launch_many<T, 64>(A, t, sms, s);
        }
    CUtensorMap map;
    const bool one = A.tokens * Piece<T>::parts <= 8;
    if (rows16 && (A.m + 1) * A.scale_stride < LIMIT && (A.m + 1) * A.zero_stride < LIMIT &&
        make_map(A, one ? 128 : 64, one ? 16 : 32, map))
        return launch_cols<T, sizeof(S) == 2>(A, sd, map, s);
    const int64_t chunks = (A.tokens + ROWS_TOK - 1) / ROWS_TOK;
    const dim3 grid((unsigned)((A.m + ROWS_NT / 32 - 1) / (ROWS_NT / 32)), (unsigned)(chunks < 65535 ? chunks : 65535));
    k_w4_rows<T, S><<<grid, ROWS_NT, 0, s>>>(A);
    return launched();
}

template <class T>
dbs_status launch_scales(const W4 &A, dbs_dtype sd, cudaStream_t s)
{
    return sd == DBS_F32 ? launch<T, float>(A, sd, s) : sd == DBS_F16 ? launch<T, __half>(A, sd, s) : launch<T, __nv_bfloat16>(A, sd, s);
}

}  // namespace

dbs_status dbs::ops::w4_waits_since(cudaStream_t s) { return waits_since(s); }

extern "C" dbs_status dbs_w4_linear(const void *x, dbs_dtype dtype, int64_t tokens, int64_t x_stride, const uint8_t *q,
                                    int64_t q_stride, const void *scales, dbs_dtype scale_dtype, int64_t scale_stride,
                                    const uint8_t *zeros, int64_t zero_stride, int64_t m, int64_t n, int32_t group,
                                    void *y, int64_t y_stride, void *stream)
{
    if (!dtype_ok(dtype) || !dtype_ok(scale_dtype) || tokens < 0 || m < 0 || n < 0 || m >= (int64_t(1) << 31) ||
        n >= (int64_t(1) << 31) || (group != 32 && group != 64 && group != 128 && group != 256))
        return DBS_ERR_INVALID_ARG;
    if (tokens == 0 || m == 0) return DBS_OK;
    if (!y || (n > 0 && (!x || !q || !scales)) || x_stride < 0 || q_stride < 0 || scale_stride < 0 ||
        (zeros && zero_stride < 0) || (tokens > 1 && y_stride < m) || (n > 0 && x == y))
        return DBS_ERR_INVALID_ARG;
    const W4 A{x, q, scales, zeros, y, tokens, x_stride, q_stride, scale_stride, zero_stride, m, n, y_stride, group, waits()};
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == DBS_F32   ? launch_scales<float>(A, scale_dtype, s)
           : dtype == DBS_F16 ? launch_scales<__half>(A, scale_dtype, s)
                              : launch_scales<__nv_bfloat16>(A, scale_dtype, s);
}
