// Linear layer with 4-bit weights and group scales for one or a few tokens
// (dbs_w4_linear, sm_103a):
//     y[t, i] = sum_g s[i, g] * sum_{j in g} x[t, j] (q[i, j] - z[i, g]).
#include "ops_dev.h"

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
};

constexpr int ROWS_NT = 128;     // four warps, one row each
constexpr int ROWS_TOK = 4;      // tokens a warp carries at a time

// Any alignment: one warp per row and ROWS_TOK tokens, two columns per byte.
template <class T, class S>
__global__ void __launch_bounds__(ROWS_NT) k_w4_rows(W4 A)
{
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * (ROWS_NT / 32) + (threadIdx.x >> 5);
    if (i >= A.m) return;
    const uint8_t *q = A.q + i * A.q_stride;
    const S *s = (const S *)A.scales + i * A.scale_stride;
    const uint8_t *z = A.zeros ? A.zeros + i * A.zero_stride : nullptr;
    const int64_t bytes = (A.n + 1) >> 1;
    for (int64_t t0 = (int64_t)blockIdx.y * ROWS_TOK; t0 < A.tokens; t0 += (int64_t)gridDim.y * ROWS_TOK) {
        float acc[ROWS_TOK] = {};
        for (int64_t c = lane; c < bytes; c += 32) {
            const int64_t j = 2 * c, g = j / A.group;
            const float sc = to_f32(s[g]), zp = z ? (float)z[g] : 8.f;
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

template <class T, class S>
void launch(const W4 &A, cudaStream_t s)
{
    const int64_t chunks = (A.tokens + ROWS_TOK - 1) / ROWS_TOK;
    const dim3 grid((unsigned)((A.m + ROWS_NT / 32 - 1) / (ROWS_NT / 32)), (unsigned)(chunks < 65535 ? chunks : 65535));
    k_w4_rows<T, S><<<grid, ROWS_NT, 0, s>>>(A);
}

template <class T>
void launch_scales(const W4 &A, dbs_dtype sd, cudaStream_t s)
{
    if (sd == DBS_F32) launch<T, float>(A, s);
    else if (sd == DBS_F16) launch<T, __half>(A, s);
    else launch<T, __nv_bfloat16>(A, s);
}

}  // namespace

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
        (zeros && zero_stride < 0) || (tokens > 1 && y_stride < m))
        return DBS_ERR_INVALID_ARG;
    const W4 A{x, q, scales, zeros, y, tokens, x_stride, q_stride, scale_stride, zero_stride, m, n, y_stride, group};
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == DBS_F32) launch_scales<float>(A, scale_dtype, s);
    else if (dtype == DBS_F16) launch_scales<__half>(A, scale_dtype, s);
    else launch_scales<__nv_bfloat16>(A, scale_dtype, s);
    return launched();
}
