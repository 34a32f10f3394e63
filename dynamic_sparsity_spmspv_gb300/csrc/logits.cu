// Penalties for repeated tokens, biases and a grammar's mask on logits
// (dbs_penalize_logits, sm_103a), one pass over the logits.
#include "ops_dev.h"

using namespace dbs::ops;

namespace {

constexpr int NT = 512;
constexpr int RUN = 8;                   // neighbouring entries of a thread: 16 bytes of 16-bit logits
constexpr int BATCH = 8;                 // history entries of a thread in flight
constexpr unsigned SEEN = 0x80000000u;   // in the history; the low bits count the output part
constexpr unsigned BIAS = 0x40000000u;   // in the bias list
constexpr unsigned NONE = 0xffffffffu;

template <class T, int N> struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Run {
    T v[N];
};

// One block per (row, slice of the vocabulary).  The block reads the row's
// whole history and keeps what falls into its slice in shared memory, so no
// [batch, vocab] counts ever exist in global memory.  A slice's first logits
// and history entries are under way before the first wait.  Slices are cut at
// `lead` entries before the row, the distance to the 16-byte boundary below it,
// so that runs of eight are aligned whatever the vocabulary's size.
template <class T, class O>
__global__ void __launch_bounds__(NT, 2) k_logits(dbs_logits_args A, int width)
{
    extern __shared__ __align__(16) unsigned smem[];
    __shared__ int listed_again;
    unsigned *count = smem, *first = smem + width;   // first: only with biases, and of flagged entries
    const int64_t b = blockIdx.y;
    const T *x = (const T *)A.logits + b * A.logits_stride;
    O *y = (O *)A.out + b * A.out_stride;
    const int lead = (int)((reinterpret_cast<uintptr_t>(x) / sizeof(T)) % RUN);
    const bool whole_runs = (reinterpret_cast<uintptr_t>(y) / sizeof(O)) % RUN == lead;
    const int v0 = (int)blockIdx.x * width - lead;   // the slice's first entry, below 0 in the first slice
    if (v0 >= A.vocab) return;
    const int v1 = A.vocab - v0 < width ? (int)A.vocab : v0 + width;
    const int32_t *h = A.history + b * A.history_stride;
    int len = 0, prompt = 0;
    if (A.history) {
        len = A.history_lens ? A.history_lens[b] : (int)A.history_max;
        prompt = A.prompt_lens ? A.prompt_lens[b] : 0;
    }
    int32_t id[BATCH];
    auto ahead = [&](int j0) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k) id[k] = j0 + k * NT < (int)A.history_max ? h[j0 + k * NT] : -1;
    };
    Run<T, RUN> in;
    auto fetch = [&](int v) {
        if (v >= 0 && v + RUN <= v1) {
            in = *(const Run<T, RUN> *)(x + v);
        } else {
#pragma unroll
            for (int e = 0; e < RUN; ++e)
                if (v + e >= 0 && v + e < v1) in.v[e] = x[v + e];
        }
    };
    if (A.history) ahead(threadIdx.x);
    fetch(v0 + (int)threadIdx.x * RUN);
    for (int i = threadIdx.x; i < width / 4; i += NT) ((uint4 *)count)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) listed_again = 0;
    __syncthreads();
    len = len < 0 ? 0 : len > A.history_max ? (int)A.history_max : len;
    for (int j0 = threadIdx.x; j0 < len; j0 += NT * BATCH) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int j = j0 + k * NT;
            if (j >= len || id[k] < 0 || id[k] < v0 || id[k] >= v1) continue;
            if (j >= prompt) atomicAdd(&count[id[k] - v0], 1u);
            else atomicOr(&count[id[k] - v0], SEEN);
        }
        if (j0 + NT * BATCH < len) ahead(j0 + NT * BATCH);
    }
    const int nb = (int)A.biases;
    const int32_t *ids = A.bias_ids + b * A.bias_stride;
    const float *vals = A.bias_vals + b * A.bias_stride;
    if (nb) {
        // flag the listed entries, then find the first place of each in the list
        for (int i = threadIdx.x; i < nb; i += NT)
            if (ids[i] >= 0 && ids[i] >= v0 && ids[i] < v1) {
                atomicOr(&count[ids[i] - v0], BIAS);
                first[ids[i] - v0] = NONE;
            }
        __syncthreads();
        for (int i = threadIdx.x; i < nb; i += NT)
            if (ids[i] >= 0 && ids[i] >= v0 && ids[i] < v1)
                if (atomicMin(&first[ids[i] - v0], (unsigned)i) != NONE) listed_again = 1;
    }
    const float rep = A.repetition ? A.repetition[b] : 1.f, pres = A.presence ? A.presence[b] : 0.f;
    // (a row's reciprocal once, instead of a division for each repeated token: 2 roundings for 1)
    const float down = 1.f / rep;
    const float freq = A.frequency ? A.frequency[b] : 0.f;
    const unsigned *allowed = A.allowed ? (const unsigned *)A.allowed + b * A.allowed_stride : nullptr;
    const int last_word = (int)((A.vocab - 1) >> 5);
    __syncthreads();
    for (int i = threadIdx.x * RUN; i < v1 - v0; i += NT * RUN) {
        const int v = v0 + i;
        if (i >= NT * RUN) fetch(v);
        unsigned bits = ~0u;                         // of entries v .. v + 7
        if (allowed) {
            const int at = v < 0 ? 0 : v;
            const unsigned a0 = allowed[at >> 5], a1 = (at >> 5) < last_word ? allowed[(at >> 5) + 1] : 0u;
            bits = __funnelshift_r(a0, a1, at & 31) << (at - v);
        }
        float l[RUN];
        unsigned c[RUN];
        *(uint4 *)c = *(const uint4 *)(count + i);
        *(uint4 *)(c + 4) = *(const uint4 *)(count + i + 4);
#pragma unroll
        for (int e = 0; e < RUN; ++e) l[e] = to_f32(in.v[e]);
        const unsigned any = c[0] | c[1] | c[2] | c[3] | c[4] | c[5] | c[6] | c[7];
        if (any) {
#pragma unroll
            for (int e = 0; e < RUN; ++e) {
                const unsigned n = c[e] & ~(SEEN | BIAS);
                if (c[e] & ~BIAS) l[e] *= l[e] > 0.f ? down : rep;
                if (n) l[e] -= fmaf(freq, (float)n, pres);
            }
            if (any & BIAS) {
                for (int e = 0; e < RUN; ++e)
                    if (count[i + e] & BIAS) {
                        const unsigned k = first[i + e];
                        float add = l[0];
#pragma unroll
                        for (int m = 1; m < RUN; ++m) add = e == m ? l[m] : add;
                        add += vals[k];
                        if (listed_again)
                            for (int m = (int)k + 1; m < nb; ++m)
                                if (ids[m] == v + e) add += vals[m];
#pragma unroll
                        for (int m = 0; m < RUN; ++m) l[m] = e == m ? add : l[m];
                    }
            }
        }
#pragma unroll
        for (int e = 0; e < RUN; ++e) l[e] = bits >> e & 1u ? l[e] : -__int_as_float(0x7f800000);
        if (whole_runs && v >= 0 && v + RUN <= v1) {
            constexpr int N = 16 / sizeof(O) < RUN ? 16 / sizeof(O) : RUN;
#pragma unroll
            for (int e = 0; e < RUN; e += N) {
                Run<O, N> r;
#pragma unroll
                for (int k = 0; k < N; ++k) r.v[k] = from_f32<O>(l[e + k]);
                *(Run<O, N> *)(y + v + e) = r;
            }
        } else {
#pragma unroll
            for (int e = 0; e < RUN; ++e)
                if (v + e >= 0 && v + e < v1) y[v + e] = from_f32<O>(l[e]);
        }
    }
}

// Slices of 1024 to 8192 entries: small ones while the grid is small, so that a
// single row spreads over the GPU; large ones otherwise, since each block reads
// the history again (from L2) and meets the memory's latency once.
template <class T, class O>
void launch(const dbs_logits_args &A, cudaStream_t s)
{
    int width = 8192;
    while (width > 1024 && (A.vocab + RUN - 2 + width) / width * A.batch < 2 * 152) width /= 2;
    const dim3 grid((unsigned)((A.vocab + RUN - 2 + width) / width), (unsigned)A.batch);
    const int smem = (A.biases > 0 ? 2 : 1) * width * (int)sizeof(unsigned);
    cudaFuncSetAttribute(k_logits<T, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * 8192 * (int)sizeof(unsigned));
    k_logits<T, O><<<grid, NT, smem, s>>>(A, width);
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
        a->vocab >= (int64_t(1) << 31) - 8192 || a->batch > 65535 || a->history_max < 0 || a->history_max >= (int64_t(1) << 30) ||
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
