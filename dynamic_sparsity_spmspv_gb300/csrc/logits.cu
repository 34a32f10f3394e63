// Penalties for repeated tokens, biases and a grammar's mask on logits
// (dbs_penalize_logits, sm_103a), one pass over the logits.
#include "ops_dev.h"

using namespace dbs::ops;

namespace {

constexpr int NT = 256;
constexpr unsigned SEEN = 0x80000000u;   // in the history; the other bits count the output part
constexpr unsigned NONE = 0xffffffffu;

// One block per (row, slice of the vocabulary).  The block reads the row's
// whole history and keeps what falls into its slice in shared memory, so no
// [batch, vocab] counts ever exist in global memory.
template <class T, class O>
__global__ void __launch_bounds__(NT) k_logits(dbs_logits_args A, int width)
{
    extern __shared__ unsigned smem[];
    __shared__ int listed_again;
    unsigned *count = smem, *first = smem + width;   // first: only with biases
    const int64_t b = blockIdx.y, v0 = (int64_t)blockIdx.x * width;
    const int w = (int)(A.vocab - v0 < width ? A.vocab - v0 : width);
    const bool bias = A.biases > 0;
    for (int i = threadIdx.x; i < w; i += NT) {
        count[i] = 0;
        if (bias) first[i] = NONE;
    }
    if (threadIdx.x == 0) listed_again = 0;
    __syncthreads();
    if (A.history) {
        int64_t len = A.history_lens ? A.history_lens[b] : A.history_max;
        len = len < 0 ? 0 : len > A.history_max ? A.history_max : len;
        const int64_t prompt = A.prompt_lens ? A.prompt_lens[b] : 0;
        const int32_t *h = A.history + b * A.history_stride;
        for (int64_t j = threadIdx.x; j < len; j += NT) {
            const int64_t d = h[j] - v0;
            if (d < 0 || d >= w) continue;
            if (j >= prompt) atomicAdd(&count[d], 1u);
            else atomicOr(&count[d], SEEN);
        }
    }
    const int32_t *ids = A.bias_ids + b * A.bias_stride;
    const float *vals = A.bias_vals + b * A.bias_stride;
    if (bias) {
        for (int64_t i = threadIdx.x; i < A.biases; i += NT) {
            const int64_t d = ids[i] - v0;
            if (d >= 0 && d < w) {
                if (atomicMin(&first[d], (unsigned)i) != NONE) listed_again = 1;
            }
        }
    }
    __syncthreads();
    const float rep = A.repetition ? A.repetition[b] : 1.f, pres = A.presence ? A.presence[b] : 0.f;
    const float freq = A.frequency ? A.frequency[b] : 0.f;
    const T *x = (const T *)A.logits + b * A.logits_stride + v0;
    O *y = (O *)A.out + b * A.out_stride + v0;
    const int32_t *allowed = A.allowed ? A.allowed + b * A.allowed_stride : nullptr;
    for (int i = threadIdx.x; i < w; i += NT) {
        float l = to_f32(x[i]);
        const unsigned c = count[i], n = c & ~SEEN;
        if (c && A.repetition) l = l > 0.f ? l / rep : l * rep;
        if (n) l -= freq * (float)n + pres;
        if (bias && first[i] != NONE) {
            l += vals[first[i]];
            if (listed_again)
                for (int64_t k = (int64_t)first[i] + 1; k < A.biases; ++k)
                    if (ids[k] == v0 + i) l += vals[k];
        }
        const int64_t v = v0 + i;
        if (allowed && !((unsigned)allowed[v >> 5] >> (v & 31) & 1u)) l = -__int_as_float(0x7f800000);
        y[i] = from_f32<O>(l);
    }
}

template <class T, class O>
void launch(const dbs_logits_args &A, cudaStream_t s)
{
    const int width = 4096;
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
