// Penalties for repeated tokens, biases and a grammar's mask on logits
// (dbs_penalize_logits, sm_103a), one pass over the logits.
#include "ops_dev.h"

using namespace dbs::ops;

namespace {

constexpr int NT = 256, BATCH = 8;       // BATCH loads of a thread in flight
constexpr unsigned SEEN = 0x80000000u;   // in the history; the other bits count the output part
constexpr unsigned NONE = 0xffffffffu;

// One block per (row, slice of the vocabulary).  The block reads the row's
// whole history and keeps what falls into its slice in shared memory, so no
// [batch, vocab] counts ever exist in global memory.  Bound by the latency of
// its few dependent steps for one row, by HBM for many; loads are issued
// BATCH at a time, since shared-memory atomics between them keep the compiler
// from doing so.
template <class T, class O>
__global__ void __launch_bounds__(NT) k_logits(dbs_logits_args A, int width)
{
    extern __shared__ unsigned smem[];
    __shared__ int listed_again;
    unsigned *count = smem, *first = smem + width;   // first: only with biases
    const int64_t b = blockIdx.y;
    const int v0 = blockIdx.x * width;
    const int w = (int)(A.vocab - v0 < width ? A.vocab - v0 : width);
    const bool bias = A.biases > 0;
    for (int i = threadIdx.x; i < w; i += NT) {
        count[i] = 0;
        if (bias) first[i] = NONE;
    }
    if (threadIdx.x == 0) listed_again = 0;
    __syncthreads();
    if (A.history) {
        int len = A.history_lens ? A.history_lens[b] : (int)A.history_max;
        len = len < 0 ? 0 : len > A.history_max ? (int)A.history_max : len;
        const int prompt = A.prompt_lens ? A.prompt_lens[b] : 0;
        const int32_t *h = A.history + b * A.history_stride;
        for (int64_t j0 = threadIdx.x; j0 < len; j0 += NT * BATCH) {
            int32_t id[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) id[k] = j0 + k * NT < len ? h[j0 + k * NT] : -1;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                // negative ids are below every slice, ids past the vocabulary beyond the last
                if (id[k] < v0 || id[k] - v0 >= w) continue;
                if (j0 + k * NT >= prompt) atomicAdd(&count[id[k] - v0], 1u);
                else atomicOr(&count[id[k] - v0], SEEN);
            }
        }
    }
    const int32_t *ids = A.bias_ids + b * A.bias_stride;
    const float *vals = A.bias_vals + b * A.bias_stride;
    if (bias) {
        for (int64_t i = threadIdx.x; i < A.biases; i += NT) {
            const int32_t id = ids[i];
            if (id >= v0 && id - v0 < w) {
                if (atomicMin(&first[id - v0], (unsigned)i) != NONE) listed_again = 1;
            }
        }
    }
    __syncthreads();
    const float rep = A.repetition ? A.repetition[b] : 1.f, pres = A.presence ? A.presence[b] : 0.f;
    const float freq = A.frequency ? A.frequency[b] : 0.f;
    const T *x = (const T *)A.logits + b * A.logits_stride + v0;
    O *y = (O *)A.out + b * A.out_stride + v0;
    const int32_t *allowed = A.allowed ? A.allowed + b * A.allowed_stride : nullptr;
    for (int i0 = threadIdx.x; i0 < w; i0 += NT * BATCH) {
        T in[BATCH];
        unsigned bits[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = i0 + k * NT;
            if (i < w) {
                in[k] = x[i];
                bits[k] = allowed ? (unsigned)allowed[(v0 + i) >> 5] : ~0u;
            }
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = i0 + k * NT;
            if (i >= w) break;
            float l = to_f32(in[k]);
            const unsigned c = count[i], n = c & ~SEEN;
            if (c && A.repetition) l = l > 0.f ? l / rep : l * rep;
            if (n) l -= freq * (float)n + pres;
            if (bias && first[i] != NONE) {
                l += vals[first[i]];
                if (listed_again)
                    for (int64_t m = (int64_t)first[i] + 1; m < A.biases; ++m)
                        if (ids[m] == v0 + i) l += vals[m];
            }
            if (!(bits[k] >> ((v0 + i) & 31) & 1u)) l = -__int_as_float(0x7f800000);
            y[i] = from_f32<O>(l);
        }
    }
}

// Slices of 512 to 4096 entries: small ones while the grid is small, so that a
// single row spreads over the GPU (each block reads the history again, from L2).
template <class T, class O>
void launch(const dbs_logits_args &A, cudaStream_t s)
{
    int width = 4096;
    while (width > 512 && (A.vocab + width - 1) / width * A.batch < 608) width /= 2;
    const dim3 grid((unsigned)((A.vocab + width - 1) / width), (unsigned)A.batch);
    k_logits<T, O><<<grid, NT, (A.biases > 0 ? 2 : 1) * width * sizeof(unsigned), s>>>(A, width);
}

template <class T>
void launch_out(const dbs_logits_args &A, cudaStream_t s)
{
    if (A.out_dtype == DBS_F32) launch<T, float>(A, s);
    else if (A.out_dtype == DBS_F16) launch<T, __half>(A, s);
    else launch<T, __nv_bfloat16>(A, s);
}

}  // namespace

extern "C" dbs_status dbs_penalize_logits(const dbs_logits_args *a, void *stream)
{
    if (!a || !dtype_ok(a->dtype) || !dtype_ok(a->out_dtype) || a->batch < 0 || a->vocab < 0 ||
        a->vocab >= (int64_t(1) << 31) || a->batch > 65535 || a->history_max < 0 || a->history_max >= (int64_t(1) << 31) ||
        a->biases < 0 || a->biases >= (int64_t(1) << 31))
        return DBS_ERR_INVALID_ARG;
    if (a->batch == 0 || a->vocab == 0) return DBS_OK;
    const bool rows = a->batch > 1;
    if (!a->logits || !a->out || a->logits_stride < 0 || (rows && a->out_stride < a->vocab) ||
        (a->history && a->history_stride < 0) ||
        (a->biases > 0 && (!a->bias_ids || !a->bias_vals || a->bias_stride < 0)) || (a->allowed && a->allowed_stride < 0))
        return DBS_ERR_INVALID_ARG;
    if (a->out == a->logits && (a->dtype != a->out_dtype || (rows && a->logits_stride != a->out_stride)))
        return DBS_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (a->dtype == DBS_F32) launch_out<float>(*a, s);
    else if (a->dtype == DBS_F16) launch_out<__half>(*a, s);
    else launch_out<__nv_bfloat16>(*a, s);
    return launched();
}
