// Penalties for repeated tokens, biases and a grammar's mask on logits
// (dbs_penalize_logits, sm_103a), one pass over the logits.
#include "ops_dev.h"

using namespace dbs::ops;

namespace {

constexpr int NT = 512;
constexpr int RUN = 8;                   // neighbouring entries of a thread: 16 bytes of 16-bit logits
constexpr int NEAR = 8;                  // history entries of a thread in flight, narrow slices
constexpr int AHEAD = 4;                 // loads of four history entries of a thread in flight, wide slices
constexpr unsigned SEEN = 0x80000000u;   // in the history; the low bits count the output part
constexpr unsigned BIAS = 0x40000000u;   // in the bias list
constexpr unsigned NONE = 0xffffffffu;

template <class T, int N> struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Run {
    T v[N];
};

// How a call is cut up.
struct Cut {
    int width;                 // entries of a slice, a multiple of 128, 65536 at most
    int counts;                // different tokens of a row that a slice can hold, at most
    int counters;              // warps that count
};
constexpr int WIDTH_MAX = 65536, COUNTS_MAX = 16384;

// One block per (row, slice of the vocabulary).  The block reads the row's
// whole history and counts what falls into its slice in shared memory, so no
// [batch, vocab] counts ever exist in global memory.  Slices are cut at `lead`
// entries before the row, the distance to the 16-byte boundary below it, so that
// runs of eight are aligned whatever the vocabulary's size.
//
// Narrow slices, for calls whose blocks all run at once: a word of shared memory
// for each entry.  A slice's first logits and history entries are under way before
// the first wait; what is left is a chain of a few waits (one row of 32,000 with 700
// tokens: 6.1 us back to back), or, where the history is long, its atomics (12 rows of
// 100,003 with 20,000 tokens: 10.2 us; k_logits_wide takes 19.4).
template <class T, class O>
__global__ void __launch_bounds__(NT, 2) k_logits_narrow(dbs_logits_args A, int width)
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
    int32_t id[NEAR];
    auto ahead = [&](int j0) {
#pragma unroll
        for (int k = 0; k < NEAR; ++k) id[k] = j0 + k * NT < (int)A.history_max ? h[j0 + k * NT] : -1;
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
    for (int j0 = threadIdx.x; j0 < len; j0 += NT * NEAR) {
#pragma unroll
        for (int k = 0; k < NEAR; ++k) {
            const int j = j0 + k * NT;
            if (j >= len || id[k] < 0 || id[k] < v0 || id[k] >= v1) continue;
            if (j >= prompt) atomicAdd(&count[id[k] - v0], 1u);
            else atomicOr(&count[id[k] - v0], SEEN);
        }
        if (j0 + NT * NEAR < len) ahead(j0 + NT * NEAR);
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
                // (a division, not a product with the row's reciprocal: that is rounded twice, and infinite for
                // penalties below 2^-128; it took 5.9 us for one row of 32,000, this takes 6.1)
                const unsigned n = c[e] & ~(SEEN | BIAS);
                if (c[e] & ~BIAS) l[e] = l[e] > 0.f ? l[e] / rep : l[e] * rep;
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

// Wide slices, for calls with more blocks than run at once: each block reads the
// history and meets the memory's latency several times, so there are few of them.
// Some of a block's warps count what falls into its slice: they mark each token in a bitmap, sum up the
// bitmap's words, so that a marked token's rank among the marked ones is at hand,
// and then add the tokens up by rank.  No atomic's answer is waited for (a hashed
// table, whose words are claimed by compare and swap, took 15 us for 4096 tokens
// of four warps), and there is room for a slice of 65536 entries.  The others read, mask and write every
// entry as it is, in runs of eight, and the first ones help them then: bound by
// HBM (96 rows of 128,000 with 4096 tokens: 27 us; k_logits_narrow takes 38.1, in
// six waves of blocks).  Last the marked entries, few against the slice, are computed again with
// penalties and biases and written over.  Their logits are read a second time:
// where out is the logits themselves, an entry that the first part changed is a
// masked one, and those stay as they are.
template <class T, class O>
__global__ void __launch_bounds__(NT, 2) k_logits_wide(dbs_logits_args A, Cut C)
{
    extern __shared__ __align__(16) unsigned smem[];
    __shared__ int listed_again, next, listed, sums[NT / 32];
    const int words = C.width / 32;
    unsigned *marks = smem, *below = marks + words;                        // bitmap; marked tokens before each of its words
    unsigned *count = below + words, *first = count + C.counts;            // by rank: counts; places in the bias list, if there is one
    uint16_t *list = (uint16_t *)(first + (A.biases > 0 ? C.counts : 0));  // by rank: the entry
    const int64_t b = blockIdx.y;
    const T *x = (const T *)A.logits + b * A.logits_stride;
    O *y = (O *)A.out + b * A.out_stride;
    const int lead = (int)((reinterpret_cast<uintptr_t>(x) / sizeof(T)) % RUN);
    const bool whole_runs = (reinterpret_cast<uintptr_t>(y) / sizeof(O)) % RUN == lead;
    const int vocab = (int)A.vocab;
    const int v0 = (int)blockIdx.x * C.width - lead;   // the slice's first entry, below 0 in the first slice
    const int v1 = vocab - v0 < C.width ? vocab : v0 + C.width;
    if (v0 >= vocab) return;

    const int32_t *h = A.history + b * A.history_stride;
    const bool wide = (reinterpret_cast<uintptr_t>(h) & 15u) == 0;
    const int most = A.history ? (int)A.history_max : 0;
    const int lane = threadIdx.x & 31, counting = 32 * C.counters;
    // Entries j .. j + 3 of the history; AHEAD such loads of a thread are under way.
    int4 id[AHEAD];
    auto entries = [&](int64_t j) {
        int4 v = make_int4(-1, -1, -1, -1);
        if (wide && j + 4 <= most) {
            v = *(const int4 *)(h + j);
        } else if (j < most) {
            v.x = h[j];
            if (j + 1 < most) v.y = h[j + 1];
            if (j + 2 < most) v.z = h[j + 2];
            if (j + 3 < most) v.w = h[j + 3];
        }
        return v;
    };
    // all that the row needs, before the first wait
    const float rep = A.repetition ? A.repetition[b] : 1.f, pres = A.presence ? A.presence[b] : 0.f;
    const float freq = A.frequency ? A.frequency[b] : 0.f;
    const int nb = (int)A.biases;
    const int32_t *ids = A.bias_ids + b * A.bias_stride;
    const float *vals = A.bias_vals + b * A.bias_stride;
    int len = 0, prompt = 0;
    if (most > 0) {
        if ((int)threadIdx.x < counting)
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) id[k] = entries(4 * threadIdx.x + (int64_t)4 * counting * k);
        len = A.history_lens ? A.history_lens[b] : most;
        prompt = A.prompt_lens ? A.prompt_lens[b] : 0;
        len = len < 0 ? 0 : len > most ? most : len;
    }
    for (int i = threadIdx.x; i < words / 4; i += NT) ((uint4 *)marks)[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < C.counts / 4; i += NT) {
        ((uint4 *)count)[i] = make_uint4(0, 0, 0, 0);
        if (nb) ((uint4 *)first)[i] = make_uint4(NONE, NONE, NONE, NONE);
    }
    if (threadIdx.x == 0) listed_again = next = 0;
    __syncthreads();

    const int low = v0 < 0 ? 0 : v0;
    const unsigned span = (unsigned)(v1 - low);
    // (what lies below the slice is far above it as an unsigned distance)
    auto here = [&](int v) { return (unsigned)v - (unsigned)low < span; };
    auto rank_of = [&](unsigned d) { return below[d >> 5] + __popc(marks[d >> 5] & ((1u << (d & 31)) - 1u)); };

    // ---- counts ----
    if ((int)threadIdx.x < counting) {
        const int warp = threadIdx.x >> 5;
        // both passes over the history and the biases
        auto each = [&](auto token, auto bias) {
            const bool long_one = len > 4 * counting * AHEAD;              // else the registers hold all of it
            for (int64_t j0 = 0; j0 < len; j0 += 4 * counting * AHEAD) {
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const int64_t jk = j0 + 4 * counting * k;
                    const int v[4] = {id[k].x, id[k].y, id[k].z, id[k].w};
                    if (long_one) {
                        // the next round's, or, at the end, the first again
                        const int64_t to = jk + 4 * counting * AHEAD;
                        id[k] = entries((j0 + 4 * counting * AHEAD < len ? to : (int64_t)4 * counting * k) + 4 * threadIdx.x);
                    }
                    if (jk >= len) continue;
                    const int j = (int)jk + 4 * (int)threadIdx.x;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (here(v[e]) && j + e < len) token((unsigned)(v[e] - low), j + e >= prompt);
                }
            }
            for (int i = threadIdx.x; i < nb; i += counting) {
                const int v = ids[i];
                if (here(v)) bias((unsigned)(v - low), i);
            }
        };
        auto meet = [&] { asm volatile("bar.sync 1, %0;" ::"r"(counting) : "memory"); };
        auto mark = [&](unsigned d) { atomicOr(&marks[d >> 5], 1u << (d & 31)); };
        each([&](unsigned d, bool) { mark(d); }, [&](unsigned d, int) { mark(d); });
        meet();
        // ranks: each thread has neighbouring words
        const int per = (words + counting - 1) / counting, w0 = threadIdx.x * per, w1 = w0 + per < words ? w0 + per : words;
        int mine = 0;
        for (int i = w0; i < w1; ++i) mine += __popc(marks[i]);
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(~0u, upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 31) sums[warp] = upto;
        meet();
        int at = upto - mine;
        for (int i = 0; i < warp; ++i) at += sums[i];
        if ((int)threadIdx.x == counting - 1) listed = at + mine;
        for (int i = w0; i < w1; ++i) {
            below[i] = at;
            for (unsigned m = marks[i]; m; m &= m - 1) list[at++] = (uint16_t)(32 * i + __ffs(m) - 1);
        }
        meet();
        each([&](unsigned d, bool output) {
                const unsigned r = rank_of(d);
                if (output) atomicAdd(&count[r], 1u);
                else atomicOr(&count[r], SEEN);
            },
            [&](unsigned d, int i) {
                const unsigned r = rank_of(d);
                atomicOr(&count[r], BIAS);
                if (atomicMin(&first[r], (unsigned)i) != NONE) listed_again = 1;
            });
    }

    // ---- every entry ----
    const unsigned *allowed = A.allowed ? (const unsigned *)A.allowed + b * A.allowed_stride : nullptr;
    const int last_word = (vocab - 1) >> 5;
    for (;;) {
        int part = 0;
        if (lane == 0) part = atomicAdd(&next, 1);
        const int64_t at = v0 + (int64_t)__shfl_sync(~0u, part, 0) * (2 * 32 * RUN) + lane * RUN;
        if (at - lane * RUN >= v1) break;
        Run<T, RUN> in[2];
        unsigned bits[2] = {~0u, ~0u};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t v = at + k * 32 * RUN;
            if (v >= v1) continue;
            if (v >= 0 && v + RUN <= v1) {
                in[k] = *(const Run<T, RUN> *)(x + v);
            } else {
#pragma unroll
                for (int e = 0; e < RUN; ++e)
                    if (v + e >= 0 && v + e < v1) in[k].v[e] = x[v + e];
            }
            if (allowed) {
                const int from = v < 0 ? 0 : (int)v;
                const unsigned a0 = allowed[from >> 5], a1 = (from >> 5) < last_word ? allowed[(from >> 5) + 1] : 0u;
                bits[k] = __funnelshift_r(a0, a1, from & 31) << (from - (int)v);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t v = at + k * 32 * RUN;
            if (v >= v1) continue;
            float l[RUN];
#pragma unroll
            for (int e = 0; e < RUN; ++e) l[e] = (int)(bits[k] << (31 - e)) < 0 ? to_f32(in[k].v[e]) : -__int_as_float(0x7f800000);
            if (whole_runs && v >= 0 && v + RUN <= v1) {
                constexpr int N = 16 / sizeof(O) < RUN ? 16 / sizeof(O) : RUN;
#pragma unroll
                for (int e = 0; e < RUN; e += N) {
                    Run<O, N> r;
#pragma unroll
                    for (int m = 0; m < N; ++m) r.v[m] = from_f32<O>(l[e + m]);
                    *(Run<O, N> *)(y + v + e) = r;
                }
            } else {
#pragma unroll
                for (int e = 0; e < RUN; ++e)
                    if (v + e >= 0 && v + e < v1) y[v + e] = from_f32<O>(l[e]);
            }
        }
    }
    __syncthreads();

    // ---- the marked entries ----
    for (int i = threadIdx.x; i < listed; i += NT) {
        const int v = low + (int)list[i];
        const unsigned c = count[i], n = c & ~(SEEN | BIAS), k = c & BIAS ? first[i] : 0u;
        const unsigned mask = allowed ? allowed[v >> 5] : ~0u;             // (three loads at once)
        const float add = c & BIAS ? vals[k] : 0.f;
        float l = to_f32(x[v]);
        if (!(mask >> (v & 31) & 1u)) continue;
        if (c & ~BIAS) l = l > 0.f ? l / rep : l * rep;
        if (n) l -= fmaf(freq, (float)n, pres);
        if (c & BIAS) {
            l += add;
            if (listed_again)
                for (int m = (int)k + 1; m < nb; ++m)
                    if (ids[m] == v) l += vals[m];
        }
        y[v] = from_f32<O>(l);
    }
}

// Narrow slices where all of them run at once, two blocks an SM; a single row
// spreads over the GPU.
template <class T, class O>
dbs_status launch(const dbs_logits_args &A, cudaStream_t s)
{
    const int64_t places = 2 * multiprocessors(), all = A.vocab + RUN - 1, tokens = (A.history ? A.history_max : 0) + A.biases;
    if (places == 0) return DBS_ERR_CUDA;
    constexpr int NARROW = 8192;
    auto slices_of = [&](int64_t width) { return (all + width - 1) / width; };
    if (slices_of(NARROW) * A.batch <= places) {
        int width = NARROW;
        while (width > 1024 && slices_of(width / 2) * A.batch <= places) width /= 2;
        static Once once;
        if (!room_for(once, k_logits_narrow<T, O>, 2 * NARROW * (int)sizeof(unsigned))) return DBS_ERR_CUDA;
        const int bytes = (A.biases > 0 ? 2 : 1) * width * (int)sizeof(unsigned);
        k_logits_narrow<T, O><<<dim3((unsigned)slices_of(width), (unsigned)A.batch), NT, bytes, s>>>(A, width);
        return launched();
    }
    // Wide ones: the time of a block in ns is 1200 for two runs of each thread, 1000
    // for a round of history and 4000 for the rest.
    const int64_t room = A.biases > 0 ? COUNTS_MAX / 2 : COUNTS_MAX;         // (10 or 6 bytes a count)
    const int64_t most = tokens > room ? room : WIDTH_MAX, least = slices_of(most);
    Cut C{};
    double best = 0;
    for (int64_t n = least; n < least + 128 && (n == least || (n - 1) * 1024 < all); ++n) {
        const int64_t width = ((all + n - 1) / n + 127) / 128 * 128;
        const double waves = (double)((A.batch * n + places - 1) / places);
        const double cost = waves * ((double)((width + 2 * NT * RUN - 1) / (2 * NT * RUN)) * 1200 + (double)(1 + tokens / (4 * NT * AHEAD)) * 1000 + 4000);
        if (C.width == 0 || cost <= best) {
            best = cost;
            C.width = (int)width;
        }
    }
    C.counts = (int)(tokens < C.width ? (tokens + 3) / 4 * 4 : C.width);
    // as many warps count as are done with it while the others go over the entries
    C.counters = 8;
    while (C.counters < NT / 32 && tokens / (C.counters * 32 * 4 * AHEAD) * 1500 > (double)C.width / (2 * NT * RUN) * 1200) C.counters *= 2;
    static Once once;
    if (!room_for(once, k_logits_wide<T, O>, 113 * 1024)) return DBS_ERR_CUDA;
    const int bytes = C.width / 32 * 8 + C.counts * (A.biases > 0 ? 10 : 6);
    k_logits_wide<T, O><<<dim3((unsigned)slices_of(C.width), (unsigned)A.batch), NT, bytes, s>>>(A, C);
    return launched();
}

template <class T>
dbs_status launch_out(const dbs_logits_args &A, cudaStream_t s)
{
    return A.out_dtype == DBS_F32 ? launch<T, float>(A, s) : A.out_dtype == DBS_F16 ? launch<T, __half>(A, s) : launch<T, __nv_bfloat16>(A, s);
}

}  // namespace

extern "C" dbs_status dbs_penalize_logits(const dbs_logits_args *a, void *stream)
{
    if (!a || !dtype_ok(a->dtype) || !dtype_ok(a->out_dtype) || a->batch < 0 || a->vocab < 0 ||
        a->vocab >= (int64_t(1) << 31) - 8192 || a->batch > 65535 || a->history_max < 0 || a->history_max >= (int64_t(1) << 29) ||
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
    return a->dtype == DBS_F32 ? launch_out<float>(*a, s) : a->dtype == DBS_F16 ? launch_out<__half>(*a, s) : launch_out<__nv_bfloat16>(*a, s);
}
