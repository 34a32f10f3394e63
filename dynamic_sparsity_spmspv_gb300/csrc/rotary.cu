// Rotary positions (dbs_rotary, dbs_rotary_table, sm_103a): every pair (a, b)
// of a head's first `dim` entries becomes (a cos - b sin, a sin + b cos).
#include <cmath>

#include "ops_dev.h"

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

// One thread per pair (or copied entry) of one head of one token.
template <class T, bool INTERLEAVED>
__global__ void __launch_bounds__(NT) k_rotary(Rotary A, int heads)
{
    const int half = A.dim / 2, units = half + (A.head_dim - A.dim);
    const int64_t all = A.total * heads * units;
    for (int64_t u = (int64_t)blockIdx.x * NT + threadIdx.x; u < all; u += (int64_t)gridDim.x * NT) {
        const int c = (int)(u % units);
        const int64_t th = u / units, tok = th / heads;
        int h = (int)(th % heads), p = 0;
        while (h >= A.part[p].heads) h -= A.part[p++].heads;
        const dbs_rotary_heads &P = A.part[p];
        const int64_t b = tok / A.tokens, t = tok % A.tokens;
        const T *in = (const T *)P.in + b * P.in_batch + t * P.in_token + h * P.in_head;
        T *out = (T *)P.out + h * P.out_head;
        if (P.to_slots) {
            const int64_t s = A.slots[tok];
            if (s < 0 || s >= A.slots_end) continue;
            out += s / A.page_size * P.out_batch + s % A.page_size * P.out_token;
        } else {
            out += b * P.out_batch + t * P.out_token;
        }
        if (c >= half) {
            out[A.dim + c - half] = in[A.dim + c - half];
            continue;
        }
        const int i = INTERLEAVED ? 2 * c : c, j = INTERLEAVED ? 2 * c + 1 : c + half;
        if (!P.rotate) {
            const T a = in[i], b2 = in[j];
            out[i] = a;
            out[j] = b2;
            continue;
        }
        const int64_t pos = A.positions[tok];
        const bool ok = pos >= 0 && pos < A.table_rows;
        const float cs = ok ? A.table[pos * A.dim + c] : nanf("");
        const float sn = ok ? A.sign * A.table[pos * A.dim + half + c] : nanf("");
        const float x = to_f32(in[i]), y = to_f32(in[j]);
        out[i] = from_f32<T>(x * cs - y * sn);
        out[j] = from_f32<T>(x * sn + y * cs);
    }
}

template <class T>
void launch(const Rotary &A, int heads, bool interleaved, cudaStream_t s)
{
    const int64_t all = A.total * heads * (A.head_dim - A.dim / 2);
    const int64_t blocks = (all + NT - 1) / NT;
    const unsigned grid = (unsigned)(blocks < (int64_t(1) << 30) ? blocks : (int64_t(1) << 30));
    if (interleaved) k_rotary<T, true><<<grid, NT, 0, s>>>(A, heads);
    else k_rotary<T, false><<<grid, NT, 0, s>>>(A, heads);
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
        // pair index at which a pair turns beta times within the trained positions
        const double pi = 3.14159265358979323846;
        auto at = [&](double beta) { return dim * std::log(trained / (beta * 2 * pi)) / (2 * std::log(base)); };
        const double lo = std::fmax(0, std::floor(at(beta_fast)));
        double hi = std::fmin(half - 1, std::ceil(at(beta_slow)));
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
    int heads = 0;
    const bool work = batch > 0 && tokens > 0;
    if (work && (batch > (int64_t(1) << 31) || tokens > (int64_t(1) << 31) || batch * tokens >= (int64_t(1) << 31)))
        return DBS_ERR_INVALID_ARG;
    for (int p = 0; p < nparts; ++p) {
        const dbs_rotary_heads &P = parts[p];
        if (P.heads < 0 || P.heads > 65536) return DBS_ERR_INVALID_ARG;
        if (P.heads == 0) continue;
        if (work && (!P.in || !P.out || (P.rotate && dim > 0 && (!table || !positions)) ||
                     (P.to_slots && (!slots || pages < 0 || page_size < 1 || pages > (int64_t(1) << 31) / page_size))))
            return DBS_ERR_INVALID_ARG;
        A.part[A.nparts++] = P;
        heads += P.heads;
    }
    if (!work || heads == 0) return DBS_OK;
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
    if (dtype == DBS_F32) launch<float>(A, heads, interleaved != 0, s);
    else if (dtype == DBS_F16) launch<__half>(A, heads, interleaved != 0, s);
    else launch<__nv_bfloat16>(A, heads, interleaved != 0, s);
    return launched();
}

}  // extern "C"
