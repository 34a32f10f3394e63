// Rotary positions (dbs_rotary, dbs_rotary_table, sm_103a): every pair (a, b)
// of a head's first `dim` entries becomes (a cos - b sin, a sin + b cos).
#include <cmath>

#include "places.h"
#include "vec_dev.h"

using namespace dbs::ops;

namespace {

struct Rotary {
    dbs_rotary_heads part[3];
    int32_t nparts, head_dim, dim;
    int64_t tokens, total;           // tokens of a sequence, tokens of all
    const float *table;
    int64_t table_rows;
    const int32_t *positions, *slots;
    int64_t page_size, slots_end;
    float sign;                      // of the sine
};

constexpr int NT = 256;

// A unit of a head is what one thread turns at once: vectors i and i + dim/2 of
// the half layout, or one vector of pairs of the interleaved one.  A thread
// keeps its token's cosines and sines for up to `span` heads of one group
// (blockIdx.y), four of whose loads are issued together.  The copied rest of the
// heads (and all of a group that is not turned) has blocks of its own, COPY, so
// that no warp does both.  Bound by HBM: every entry is read and written once (16,382
// tokens of 40 heads of 128, half of each turned, bf16: 54.9 us, 91% of a copy's rate;
// 8192 tokens of 32 heads of 96, interleaved, fp32: 34.8 us, 86%).
template <class T, bool INTERLEAVED, bool WIDE, bool COPY>
__device__ __forceinline__ void turn_heads(const Rotary &A, const dbs_rotary_heads &P, int h0, int heads, uint32_t units, uint32_t threads,
                                           int from)
{
    using V = Vec<T, WIDE>;
    using VT = typename V::type;
    constexpr int N = V::n;
    // interleaved pairs of single values: two entries a unit
    constexpr int PAIRS = INTERLEAVED ? (WIDE ? N / 2 : 1) : N;
    constexpr int F = !WIDE ? 1 : PAIRS < 4 ? PAIRS : 4;      // entries of the table in one load
    constexpr bool TWO = !COPY && (!INTERLEAVED || !WIDE);    // a second vector
    const uint32_t i = blockIdx.x * NT + threadIdx.x;
    if (i >= threads) return;
    const uint32_t tok = i / units, c = i - tok * units;
    const uint32_t b = tok / (uint32_t)A.tokens, t = tok - b * (uint32_t)A.tokens;
    const int half = A.dim / 2, pair = (int)c * PAIRS;        // the unit's first pair
    const int lo = COPY ? from + (int)c * N : INTERLEAVED ? 2 * pair : pair;
    const int apart = INTERLEAVED ? 1 : half;
    const T *in = (const T *)P.in + b * P.in_batch + t * P.in_token + h0 * P.in_head + lo;
    T *out = (T *)P.out + h0 * P.out_head + lo;
    if (P.to_slots) {
        const int64_t slot = A.slots[tok];
        if (slot < 0 || slot >= A.slots_end) return;
        const uint32_t size = (uint32_t)A.page_size, page = (uint32_t)slot / size;
        out += page * P.out_batch + ((uint32_t)slot - page * size) * P.out_token;
    } else {
        out += b * P.out_batch + t * P.out_token;
    }
    float cs[PAIRS], sn[PAIRS];
    if (!COPY) {
        const int64_t pos = A.positions[tok];
        const bool ok = pos >= 0 && pos < A.table_rows;
#pragma unroll
        for (int q = 0; q < PAIRS; q += F) {
            struct alignas(4 * F) Floats {
                float v[F];
            };
            Floats c4, s4;
            const float *row = A.table + pos * A.dim + pair + q;
            if (ok) {
                c4 = *(const Floats *)row;
                s4 = *(const Floats *)(row + half);
            }
#pragma unroll
            for (int e = 0; e < F; ++e) {
                cs[q + e] = ok ? c4.v[e] : nanf("");
                sn[q + e] = ok ? A.sign * s4.v[e] : nanf("");
            }
        }
    }
    for (int h = 0; h < heads; h += 4) {
        VT x[4], z[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (h + k < heads) {
                x[k] = *(const VT *)(in + k * P.in_head);
                if (TWO) z[k] = *(const VT *)(in + k * P.in_head + apart);
            }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (h + k < heads) {
                if (!COPY) {
                    float u[N], v[N];
                    open<T>(x[k], u);
                    if (TWO) open<T>(z[k], v);
#pragma unroll
                    for (int q = 0; q < PAIRS; ++q) {
                        float &a = u[TWO ? q : 2 * q], &d = TWO ? v[q] : u[TWO ? 0 : 2 * q + 1];
                        const float a0 = a, d0 = d;
                        a = a0 * cs[q] - d0 * sn[q];
                        d = a0 * sn[q] + d0 * cs[q];
                    }
                    shut<T>(u, x[k]);
                    if (TWO) shut<T>(v, z[k]);
                }
                *(VT *)(out + k * P.out_head) = x[k];
                if (TWO) *(VT *)(out + k * P.out_head + apart) = z[k];
            }
        in += 4 * P.in_head;
        out += 4 * P.out_head;
    }
}

// blockIdx.y: the chunks of `span` heads of every turned group, then those of
// every copied part.
template <class T, bool INTERLEAVED, bool WIDE>
__global__ void __launch_bounds__(NT) k_rotary(Rotary A, uint32_t turning, int span)
{
    constexpr int N = Vec<T, WIDE>::n;
    int y = blockIdx.y;
    for (int copy = 0; copy < 2; ++copy)
        for (int p = 0; p < A.nparts; ++p) {
            const dbs_rotary_heads &P = A.part[p];
            const int from = P.rotate ? A.dim : 0;
            if (copy ? from == A.head_dim : !P.rotate || turning == 0) continue;
            const int chunks = (P.heads + span - 1) / span;
            if (y >= chunks) {
                y -= chunks;
                continue;
            }
            const int h0 = y * span, heads = P.heads - h0 < span ? P.heads - h0 : span;
            if (!copy) {
                turn_heads<T, INTERLEAVED, WIDE, false>(A, P, h0, heads, turning, (uint32_t)A.total * turning, 0);
            } else {
                const uint32_t units = (uint32_t)(A.head_dim - from) / N;
                turn_heads<T, INTERLEAVED, WIDE, true>(A, P, h0, heads, units, (uint32_t)A.total * units, from);
            }
            return;
        }
}

template <class T, bool INTERLEAVED, bool WIDE>
dbs_status launch_units(const Rotary &A, cudaStream_t s)
{
    constexpr int N = Vec<T, WIDE>::n, E = INTERLEAVED ? (WIDE ? N : 2) : 2 * N;
    const int turning = A.dim / E;
    // Heads of a thread: eight, so that a token's angles are read once for all of
    // them, and fewer while that leaves some of the GPU's threads (2048 a
    // multiprocessor) idle.
    const int64_t room = (int64_t)multiprocessors() * 2048;
    if (room == 0) return DBS_ERR_CUDA;
    int64_t most = 0;
    int span = 8, chunks = 0;
    for (;; span /= 2) {
        int64_t threads = 0;
        chunks = 0;
        for (int copy = 0; copy < 2; ++copy)
            for (int p = 0; p < A.nparts; ++p) {
                const int from = A.part[p].rotate ? A.dim : 0;
                if (copy ? from == A.head_dim : !A.part[p].rotate || turning == 0) continue;
                const int64_t units = copy ? (A.head_dim - from) / N : turning;
                const int n = (A.part[p].heads + span - 1) / span;
                chunks += n;
                threads += A.total * units * n;
                most = most > A.total * units ? most : A.total * units;
            }
        if (span == 1 || threads >= room || 2 * chunks > 65535) break;      // (the grid's limit in y)
    }
    k_rotary<T, INTERLEAVED, WIDE><<<dim3((unsigned)((most + NT - 1) / NT), (unsigned)chunks), NT, 0, s>>>(A, (uint32_t)turning, span);
    return launched();
}

template <class T>
dbs_status launch(const Rotary &A, bool interleaved, cudaStream_t s)
{
    // 16-byte accesses: all heads on such boundaries, and whole vectors in each part of a head
    constexpr int N = 16 / (int)sizeof(T);
    bool wide = A.dim % (interleaved ? N : 2 * N) == 0 && A.head_dim % N == 0 && aligned16(A.table);
    for (int p = 0; p < A.nparts; ++p) {
        const dbs_rotary_heads &P = A.part[p];
        wide = wide && aligned16(P.in) && aligned16(P.out) &&
               ((P.in_batch | P.in_token | P.in_head | P.out_batch | P.out_token | P.out_head) & (N - 1)) == 0;
    }
    if (interleaved) return wide ? launch_units<T, true, true>(A, s) : launch_units<T, true, false>(A, s);
    return wide ? launch_units<T, false, true>(A, s) : launch_units<T, false, false>(A, s);
}

struct Freqs {
    double f[256];
};

__global__ void __launch_bounds__(NT) k_rotary_table(Freqs F, int half, int64_t rows, double factor, float *table)
{
    const int64_t all = rows * half;
    for (int64_t u = (int64_t)blockIdx.x * NT + threadIdx.x; u < all; u += (int64_t)gridDim.x * NT) {
        const int64_t p = u / half;
        const int i = (int)(u % half);
        double s, c;
        sincos((double)p * F.f[i], &s, &c);
        table[p * 2 * half + i] = (float)(c * factor);
        table[p * 2 * half + half + i] = (float)(s * factor);
    }
}

}  // namespace

extern "C" {

dbs_status dbs_rotary_table(int64_t positions, int32_t dim, double base, dbs_rotary_scaling scaling, double factor,
                            double trained, double beta_fast, double beta_slow, float *table, void *stream)
{
    if (positions < 0 || positions >= (int64_t(1) << 31) || dim < 2 || dim > 512 || (dim & 1) || !(base > 1) ||
        !std::isfinite(base) || scaling < DBS_ROTARY_PLAIN || scaling > DBS_ROTARY_YARN || (positions > 0 && !table))
        return DBS_ERR_INVALID_ARG;
    if (scaling != DBS_ROTARY_PLAIN && (!(factor >= 1) || !std::isfinite(factor))) return DBS_ERR_INVALID_ARG;
    if (scaling == DBS_ROTARY_NTK && dim < 4) return DBS_ERR_INVALID_ARG;   // the exponent dim / (dim - 2)
    if (scaling == DBS_ROTARY_YARN && (!(trained > 0) || !(beta_slow > 0) || !(beta_fast > beta_slow) ||
                                       !std::isfinite(trained) || !std::isfinite(beta_fast)))
        return DBS_ERR_INVALID_ARG;
    if (positions == 0) return DBS_OK;
    const int half = dim / 2;
    Freqs F{};
    double amplitude = 1;
    if (scaling == DBS_ROTARY_NTK) base *= std::pow(factor, (double)dim / (dim - 2));
    for (int i = 0; i < half; ++i) F.f[i] = std::pow(base, -2.0 * i / dim) / (scaling == DBS_ROTARY_LINEAR ? factor : 1);
    if (scaling == DBS_ROTARY_YARN) {
        // pair index at which a pair turns beta times within the trained positions; the ends of the
        // ramp, rounded outwards, are kept within 0 and dim - 1 as in the published method, not within
        // the pairs there are: where the slowest pair still turns more than beta_slow times, the ramp
        // ends behind it
        const double pi = 3.14159265358979323846;
        auto at = [&](double beta) { return dim * std::log(trained / (beta * 2 * pi)) / (2 * std::log(base)); };
        const double lo = std::fmax(0, std::floor(at(beta_fast)));
        double hi = std::fmin(dim - 1, std::ceil(at(beta_slow)));
        if (hi <= lo) hi = lo + 0.001;
        for (int i = 0; i < half; ++i) {
            const double r = std::fmin(1, std::fmax(0, (i - lo) / (hi - lo)));   // 0: kept, 1: divided
            F.f[i] *= (1 - r) + r / factor;
        }
        amplitude = 0.1 * std::log(factor) + 1;
    }
    const int64_t blocks = (positions * half + NT - 1) / NT;
    k_rotary_table<<<(unsigned)(blocks < 65536 ? blocks : 65536), NT, 0, (cudaStream_t)stream>>>(F, half, positions,
                                                                                                 amplitude, table);
    return launched();
}

dbs_status dbs_rotary(const dbs_rotary_heads *parts, int32_t nparts, dbs_dtype dtype, int64_t batch, int64_t tokens,
                      int32_t head_dim, int32_t dim, const float *table, int64_t table_rows, const int32_t *positions,
                      const int32_t *slots, int64_t pages, int64_t page_size, int32_t interleaved, int32_t transposed,
                      void *stream)
{
    if (!parts || nparts < 1 || nparts > 3 || !dtype_ok(dtype) || batch < 0 || tokens < 0 || head_dim < 1 ||
        head_dim > 1024 || dim < 0 || dim > head_dim || (dim & 1) || table_rows < 0)
        return DBS_ERR_INVALID_ARG;
    Rotary A{};
    Places writes[3], reads[3];
    int64_t heads = 0;
    const bool work = batch > 0 && tokens > 0;
    if (work && (batch > (int64_t(1) << 31) || tokens > (int64_t(1) << 31) || batch * tokens >= (int64_t(1) << 31)))
        return DBS_ERR_INVALID_ARG;
    for (int p = 0; p < nparts; ++p) {
        const dbs_rotary_heads &P = parts[p];
        if (P.heads < 0 || P.heads > 16384) return DBS_ERR_INVALID_ARG;
        if (P.heads == 0) continue;
        if (work && (!P.in || (P.rotate && dim > 0 && (!table || !positions)) ||
                     (P.to_slots && (!slots || pages < 0 || page_size < 1 || pages > (int64_t(1) << 31) / page_size))))
            return DBS_ERR_INVALID_ARG;
        if (work && P.to_slots && pages == 0) continue;                        // no slot is inside: nothing is written
        if (work && !P.out) return DBS_ERR_INVALID_ARG;
        // heads of the output that share memory
        const int64_t n_batch = P.to_slots ? pages : batch, n_token = P.to_slots ? page_size : tokens;
        const Places out(P.out, dtype == DBS_F32 ? 4 : 2, head_dim, {{n_batch, P.out_batch}, {n_token, P.out_token}, {P.heads, P.out_head}});
        if (work && (P.in_head < 0 || P.in_token < 0 || P.in_batch < 0 || !out.own || (P.to_slots && P.in == P.out))) return DBS_ERR_INVALID_ARG;
        // (of a cache only the slots are written, which the host does not know)
        if (work && !P.to_slots) writes[A.nparts] = out;
        if (work) reads[A.nparts] = {P.in, dtype == DBS_F32 ? 4 : 2, head_dim, {{batch, P.in_batch}, {tokens, P.in_token}, {P.heads, P.in_head}}};
        A.part[A.nparts++] = P;
        heads += P.heads;
    }
    if (!work || heads == 0) return DBS_OK;
    if (clash(writes, A.nparts, reads, A.nparts, true)) return DBS_ERR_INVALID_ARG;
    if (batch * tokens * head_dim >= (int64_t(1) << 32) - NT) return DBS_ERR_INVALID_ARG;
    A.head_dim = head_dim;
    A.dim = dim;
    A.tokens = tokens;
    A.total = batch * tokens;
    A.table = table;
    A.table_rows = table_rows;
    A.positions = positions;
    A.slots = slots;
    A.page_size = page_size;
    A.slots_end = slots ? pages * page_size : 0;
    A.sign = transposed ? -1.f : 1.f;
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == DBS_F32   ? launch<float>(A, interleaved != 0, s)
           : dtype == DBS_F16 ? launch<__half>(A, interleaved != 0, s)
                              : launch<__nv_bfloat16>(A, interleaved != 0, s);
}

}  // extern "C"
