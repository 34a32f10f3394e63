// Pages of a cache (dbs_cache_resize, dbs_cache_fork, dbs_cache_compact, sm_103a).
#include "ops_dev.h"
#include "places.h"

using namespace dbs::ops;

namespace {

constexpr int PLAN_NT = 1024, PLAN_W = PLAN_NT / 32;
static_assert(PLAN_W == 32, "a lane for each warp's sum");

struct Sums {
    int64_t warp[PLAN_W], total;
};

// Sum of the values of the threads before this one, and of all in S.total; by the whole block.
__device__ __forceinline__ int64_t before(int64_t v, Sums &S)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t in = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(~0u, in, d);
        if (lane >= d) in += o;
    }
    __syncthreads();                               // (the sums of the turn before have been read)
    if (lane == 31) S.warp[w] = in;
    __syncthreads();
    if (w == 0) {
        const int64_t mine = S.warp[lane];
        int64_t all = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(~0u, all, d);
            if (lane >= d) all += o;
        }
        S.warp[lane] = all - mine;
        if (lane == 31) S.total = all;
    }
    __syncthreads();
    return S.warp[w] + in - v;
}

__device__ __forceinline__ int pages_of(int entries, int page) { return (int)(((int64_t)entries + page - 1) / page); }
__device__ __forceinline__ int length(const dbs_page_state &s, int64_t b)
{
    const int n = __ldcg(s.kv_lens + b);
    const int64_t room = s.max_pages * s.page_size;
    return n < 0 ? 0 : n > room ? (int)room : n;
}
__device__ __forceinline__ bool is_page(const dbs_page_state &s, int p) { return p >= 0 && p < s.pages; }
// (what other threads of the block changed is read behind the first-level cache)
__device__ __forceinline__ int refs_of(const dbs_page_state &s, int p) { return __ldcg(s.refs + p); }

// The numbers of the first `want` free pages, ascending, into `list`; returns how many there
// are (at most `want`, or a turn's more).  By the whole block.
constexpr int RUN = 16;                            // pages of a thread in a turn
__device__ __forceinline__ int find_free(const dbs_page_state &s, int64_t want, int *list, Sums &S)
{
    int found = 0;
    for (int64_t p0 = 0; p0 < s.pages && found < want; p0 += PLAN_NT * RUN) {
        const int64_t mine = p0 + (int64_t)threadIdx.x * RUN;
        unsigned free = 0;
#pragma unroll
        for (int i = 0; i < RUN; ++i)
            if (mine + i < s.pages && refs_of(s, (int)(mine + i)) == 0) free |= 1u << i;
        int at = found + (int)before(__popc(free), S);
        for (; free && at < want; free &= free - 1) list[at++] = (int)mine + __ffs(free) - 1;
        found += (int)S.total;
    }
    __syncthreads();
    return found;
}

// ---- lengths ----

struct Resize {
    dbs_page_state s;
    const int32_t *lens;
    int32_t *status, *slots;
    int64_t columns;
    // of every sequence: its length before; the pages that it asks for, and those that it and all before it ask for
    int32_t *old, *need, *end;
    int32_t *list;
};

// Slots of the new entries u, u + step, ... of all sequences.
__device__ __forceinline__ void write_slots(const Resize &A, int64_t u, int64_t step)
{
    const dbs_page_state &s = A.s;
    const int64_t all = s.batch * A.columns;
    const int page = (int)s.page_size;
    for (; u < all; u += step) {
        const int64_t b = u / A.columns;
        const int i = (int)(u - b * A.columns), old = __ldcg(A.old + b), n = length(s, b);
        int slot = -1;
        if (i < n - old) {
            const int j = old + i, p = __ldcg(s.page_table + b * s.page_row + j / page);
            if (is_page(s, p)) slot = p * page + j % page;
        }
        A.slots[u] = slot;
    }
}

__global__ void __launch_bounds__(256) k_slots(Resize A) { write_slots(A, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256); }

// One block does all: cuts, a sum over what the sequences ask for, a walk over refs
// that ends when enough pages are found, growth.  Bound by the latency of those steps.
__global__ void __launch_bounds__(PLAN_NT) k_resize(Resize A, int slots_here)
{
    __shared__ Sums S;
    const dbs_page_state &s = A.s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, page = (int)s.page_size;
    const int64_t room = s.max_pages * s.page_size;
    // a warp a sequence: what is cut off
    for (int64_t b = warp; b < s.batch; b += PLAN_W) {
        const int old = length(s, b), n = A.lens[b];
        if (n >= 0 && n < old)
            for (int c = pages_of(n, page) + lane; c < pages_of(old, page); c += 32) {
                const int p = s.page_table[b * s.page_row + c];
                if (is_page(s, p)) atomicSub(s.refs + p, 1);
            }
        __syncwarp();                              // (every lane has read the length)
        if (lane == 0) {
            A.old[b] = old;
            if (n >= 0 && n <= old) s.kv_lens[b] = n;
        }
    }
    __syncthreads();
    int64_t asked = 0;
    for (int64_t b0 = 0; b0 < s.batch; b0 += PLAN_NT) {
        const int64_t b = b0 + threadIdx.x;
        int need = 0;
        if (b < s.batch) {
            const int old = __ldcg(A.old + b), n = A.lens[b];
            int status = 0;
            if (n > room) {
                status = 3;
            } else if (n > old) {
                need = pages_of(n, page) - pages_of(old, page);
                if (old % page) {
                    const int p = s.page_table[b * s.page_row + old / page];
                    if (is_page(s, p) && refs_of(s, p) > 1) {
                        status = 2;
                        need = 0;
                    }
                }
            }
            A.need[b] = need;
            A.status[b] = status;
        }
        // (what is above 2^31 - 1 is above the number of pages too)
        const int64_t end = asked + before(need, S) + need;
        if (b < s.batch) A.end[b] = end > 0x7fffffff ? 0x7fffffff : (int)end;
        asked += S.total;
    }
    __syncthreads();
    const int found = asked > 0 ? find_free(s, asked < s.pages ? asked : s.pages, A.list, S) : 0;
    for (int64_t b = warp; b < s.batch; b += PLAN_W) {
        const int old = __ldcg(A.old + b), n = A.lens[b], need = __ldcg(A.need + b), end = __ldcg(A.end + b);
        if (n <= old || __ldcg(A.status + b) != 0) continue;
        if (need > 0 && end > found) {
            if (lane == 0) A.status[b] = 1;
            continue;
        }
        for (int i = lane; i < need; i += 32) {
            const int p = __ldcg(A.list + end - need + i);
            s.page_table[b * s.page_row + pages_of(old, page) + i] = p;
            s.refs[p] = 1;
        }
        if (lane == 0) s.kv_lens[b] = n;
    }
    if (!slots_here) return;
    __syncthreads();
    write_slots(A, threadIdx.x, PLAN_NT);
}

// ---- the same for few sequences: a thread has one, and everything stays in shared memory ----

constexpr int WORDS = PLAN_NT * RUN / 32;          // of a turn of pages, a bit each

// Of the pages p0 .. p0 + 32 WORDS - 1: which are free, and how many before each word.
struct Turn {
    uint32_t free[WORDS];
    int before[WORDS + 1];
};
// This thread's RUN pages of a turn; the bits of those that are free, and of those with two owners or more.
struct Run {
    uint32_t free, many;
};
__device__ __forceinline__ Run run_of(const dbs_page_state &s, int64_t p0)
{
    const int64_t mine = p0 + (int64_t)threadIdx.x * RUN;
    Run r{0, 0};
    int n[RUN];
    if (mine + RUN <= s.pages && (reinterpret_cast<uintptr_t>(s.refs) & 15u) == 0) {
#pragma unroll
        for (int i = 0; i < RUN / 4; ++i) {
            const int4 v = __ldcg((const int4 *)(s.refs + mine) + i);
            n[4 * i] = v.x;
            n[4 * i + 1] = v.y;
            n[4 * i + 2] = v.z;
            n[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < RUN; ++i) n[i] = mine + i < s.pages ? refs_of(s, (int)(mine + i)) : 1;
    }
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
        r.free |= (uint32_t)(n[i] == 0) << i;
        r.many |= (uint32_t)(n[i] > 1) << i;
    }
    return r;
}
// Two threads have a word.
__device__ __forceinline__ uint32_t word_of(uint32_t half)
{
    return half | __shfl_down_sync(~0u, half, 1) << 16;
}
// Counts the free pages of a turn whose words are there; by the whole block.
__device__ __forceinline__ int count_free(Turn &T, Sums &S)
{
    const int n = threadIdx.x < WORDS ? __popc(T.free[threadIdx.x]) : 0, at = (int)before(n, S);
    if (threadIdx.x < WORDS) T.before[threadIdx.x] = at;
    if (threadIdx.x == 0) T.before[WORDS] = (int)S.total;
    __syncthreads();
    return (int)S.total;
}
// The k-th free page of a turn (k below their number).
__device__ __forceinline__ int nth_free(const Turn &T, int k)
{
    int lo = 0;
#pragma unroll
    for (int d = WORDS / 2; d; d >>= 1)
        if (T.before[lo + d] <= k) lo += d;
    uint32_t w = T.free[lo];
    for (int i = k - T.before[lo]; i; --i) w &= w - 1;
    return 32 * lo + __ffs(w) - 1;
}
// The last of n ascending offsets that is at most k (the first is 0; equal ones: the last).
__device__ __forceinline__ int owner(const int *from, int n, int k)
{
    int lo = 0;
    for (int d = PLAN_NT / 2; d; d >>= 1)
        if (lo + d < n && from[lo + d] <= k) lo += d;
    return lo;
}

// Free pages in order, as many as are asked for: of one turn in its bits, of more in `list`.  Returns how
// many there are (all that exist, if they do not suffice); by the whole block, the first turn's bits being there.
__device__ __forceinline__ int find_few(const dbs_page_state &s, int64_t asked, Turn &T, int *list, Sums &S)
{
    __syncthreads();
    int found = asked > 0 ? count_free(T, S) : 0;
    if (s.pages <= 32 * WORDS || asked == 0) return found;
    const int total = (int)(asked < s.pages ? asked : s.pages);
    for (int k = threadIdx.x; k < found && k < total; k += PLAN_NT) list[k] = nth_free(T, k);
    for (int64_t p0 = 32 * WORDS; p0 < s.pages && found < total; p0 += 32 * WORDS) {
        const uint32_t f = word_of(run_of(s, p0).free);
        __syncthreads();                           // the bits of the turn before have been read
        if (!(threadIdx.x & 1)) T.free[threadIdx.x >> 1] = f;
        __syncthreads();
        const int here = count_free(T, S);
        for (int k = threadIdx.x; k < here && found + k < total; k += PLAN_NT) list[found + k] = (int)p0 + nth_free(T, k);
        found += here;
    }
    __syncthreads();
    return found;
}
__device__ __forceinline__ int found_page(const dbs_page_state &s, const Turn &T, const int *list, int k)
{
    return s.pages <= 32 * WORDS ? nth_free(T, k) : __ldcg(list + k);
}

// At most PLAN_NT sequences.  Cuts, new pages and slots are shared out among all threads one by one, so
// that long sequences take no longer than short ones; refs are read beside the lengths.  Bound by the latency of
// some twenty block-wide steps and three reads in a row (8, 256 and 1024 sequences, a slot each: 5.8, 6.5 and 7.1 us; by
// k_resize 5.9, 15.6 and 46).
__global__ void __launch_bounds__(PLAN_NT) k_resize_few(Resize A, int slots_here)
{
    __shared__ Sums S;
    __shared__ Turn T;
    __shared__ uint32_t many[WORDS];
    __shared__ int from[PLAN_NT], base[PLAN_NT], was[PLAN_NT], now[PLAN_NT];
    const dbs_page_state &s = A.s;
    const int t = threadIdx.x, n = (int)s.batch, page = (int)s.page_size;
    const int64_t room = s.max_pages * s.page_size;
    const bool mine = t < n;
    const int old = mine ? length(s, t) : 0, want = mine ? A.lens[t] : -1;
    const Run run = run_of(s, 0);
    const int had = pages_of(old, page), have = want < 0 || want > room ? had : pages_of(want, page);
    // the page that growth would go on in
    const int last = mine && want > old && want <= room && old % page ? __ldcg(s.page_table + (int64_t)t * s.page_row + old / page) : -1;
    const uint32_t free = word_of(run.free), shared = word_of(run.many);
    if (!(t & 1)) {
        T.free[t >> 1] = free;
        many[t >> 1] = shared;
    }
    const int cut = want >= 0 && want < old ? had - have : 0;
    const int64_t before_me = before(cut, S), cuts = S.total;
    if (cuts > 0) {
        // (owned pages are fewer than 2^31 in all, or the lengths are not a state: then the rest is passed over)
        const int most = (int)(cuts < 0x7fffffff ? cuts : 0x7fffffff);
        from[t] = before_me < most ? (int)before_me : most;
        base[t] = have;
        __syncthreads();
        for (int64_t k = t; k < most; k += PLAN_NT) {
            const int b = owner(from, n, (int)k), p = __ldcg(s.page_table + b * s.page_row + base[b] + ((int)k - from[b]));
            if (!is_page(s, p)) continue;
            const int left = atomicSub(s.refs + p, 1) - 1;
            if (p >= 32 * WORDS) continue;
            const uint32_t bit = 1u << (p & 31);
            if (left == 0) atomicOr(T.free + (p >> 5), bit);
            if (left == -1) atomicAnd(T.free + (p >> 5), ~bit);            // (a count that was wrong: not free)
            if (left == 1) atomicAnd(many + (p >> 5), ~bit);
        }
        __syncthreads();
    }
    int status = want > room ? 3 : 0, need = 0;
    if (status == 0 && want > old) {
        need = have - had;
        if (is_page(s, last) && (last < 32 * WORDS ? many[last >> 5] >> (last & 31) & 1u : refs_of(s, last) > 1)) {
            status = 2;
            need = 0;
        }
    }
    const int64_t start = before(need, S), asked = S.total;
    const int found = find_few(s, asked, T, A.list, S);
    if (need > 0 && start + need > found) {
        status = 1;
        need = 0;
    }
    // (those that get their pages come before all that do not)
    before(need, S);
    const int taken = (int)S.total;
    from[t] = start < taken ? (int)start : taken;
    base[t] = had;
    was[t] = old;
    now[t] = status == 0 && want >= 0 ? want : old;
    __syncthreads();
    for (int k = t; k < taken; k += PLAN_NT) {
        const int b = owner(from, n, k), p = found_page(s, T, A.list, k);
        s.page_table[b * s.page_row + base[b] + (k - from[b])] = p;
        s.refs[p] = 1;
    }
    if (mine) {
        A.status[t] = status;
        if (status == 0 && want >= 0) s.kv_lens[t] = want;
        if (A.old) A.old[t] = old;
    }
    if (!slots_here) return;
    __syncthreads();
    const uint32_t columns = (uint32_t)A.columns, all = (uint32_t)n * columns;
    for (uint32_t u = t; u < all; u += PLAN_NT) {
        const uint32_t b = u / columns;
        const int i = (int)(u - b * columns);
        int slot = -1;
        if (i < now[b] - was[b]) {
            const int j = was[b] + i, p = __ldcg(s.page_table + b * s.page_row + j / page);
            if (is_page(s, p)) slot = p * page + j % page;
        }
        A.slots[u] = slot;
    }
}

// ---- copies of entries ----

// Bytes of a row of one entry that lie together, and where rows lie.
struct Data {
    char *k, *v;
    int64_t heads, row;                // rows of an entry, and their units of V bytes
    int64_t k_layer, k_page, k_entry, k_head, v_layer, v_page, v_entry, v_head;   // in units
};

struct Fork {
    int from, to;                      // pages; to: -1 where there is nothing to copy
    int entries;                       // of that page
    int parent, child, full;           // sequences and full pages; child: -1 if it stayed empty
};

// One block: lengths before the call, the children that are taken, pages for those parents'
// entries that do not fill a page.  A child is claimed by the first that names it: the least of
// the marks i - n that the claimants leave in its length.
__global__ void __launch_bounds__(PLAN_NT) k_fork_plan(dbs_page_state s, const int32_t *parents, const int32_t *children, int n,
                                                       int32_t *status, Fork *forks, int32_t *list)
{
    __shared__ Sums S;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int page = (int)s.page_size;
    for (int i = threadIdx.x; i < n; i += PLAN_NT) {
        const int p = parents[i], c = children[i];
        Fork f{0, -1, 0, p, -1, 0};
        if (p >= 0 && p < s.batch && c >= 0 && c < s.batch) {
            const int len = length(s, p);
            f.full = len / page;
            f.entries = len % page;
            if (length(s, c) == 0) f.child = c;
        }
        forks[i] = f;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += PLAN_NT)
        if (forks[i].child >= 0) s.kv_lens[forks[i].child] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += PLAN_NT)
        if (forks[i].child >= 0) atomicMin(s.kv_lens + forks[i].child, i - n);
    __syncthreads();
    int asked = 0;
    for (int i0 = 0; i0 < n; i0 += PLAN_NT) {
        const int i = i0 + threadIdx.x;
        int need = 0;
        if (i < n) {
            Fork &f = forks[i];
            const bool won = f.child >= 0 && __ldcg(s.kv_lens + f.child) == i - n;
            status[i] = won ? 0 : 2;
            need = won && f.entries > 0;
            if (won && need) {
                f.from = s.page_table[f.parent * s.page_row + f.full];
                if (!is_page(s, f.from)) f.from = -1;
            }
        }
        const int at = asked + (int)before(need, S);
        if (need) forks[i].to = at;                // its place among the free pages
        asked += (int)S.total;
    }
    __syncthreads();
    const int found = asked > 0 ? find_free(s, asked, list, S) : 0;
    for (int i = threadIdx.x; i < n; i += PLAN_NT) {
        Fork &f = forks[i];
        if (status[i] != 0) {
            f.child = f.to = -1;
            continue;
        }
        if (f.to >= found) {
            status[i] = 1;
            s.kv_lens[f.child] = 0;
            f.child = f.to = -1;
            continue;
        }
        s.kv_lens[f.child] = f.full * page + f.entries;
        if (f.to >= 0) {
            f.to = __ldcg(list + f.to);
            s.page_table[f.child * s.page_row + f.full] = f.to;
            s.refs[f.to] = 1;
            if (f.from < 0) f.to = -1;             // (nothing to copy from)
        }
    }
}

// The same for at most PLAN_NT forks, in shared memory: the children are kept in a table twice as large as they
// are many, each with the first valid fork that names it.  (4, 256 and 1024 forks with the copies of two small
// states 7.2, 8.5 and 13.4 us; by the other kernel 9.3, 10.7 and 16.6; with a comparison of every two children 7, 15 and 41.)
__global__ void __launch_bounds__(PLAN_NT) k_fork_plan_few(dbs_page_state s, const int32_t *parents, const int32_t *children, int n,
                                                           int32_t *status, Fork *forks, int32_t *list)
{
    __shared__ Sums S;
    __shared__ Turn T;
    __shared__ int child[2 * PLAN_NT], by[2 * PLAN_NT];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = threadIdx.x, page = (int)s.page_size;
    const bool mine = t < n;
    const int p = mine ? parents[t] : -1, c = mine ? children[t] : -1;
    const Run run = run_of(s, 0);
    child[t] = child[t + PLAN_NT] = -1;
    by[t] = by[t + PLAN_NT] = PLAN_NT;
    bool good = p >= 0 && p < s.batch && c >= 0 && c < s.batch;
    const int len = good ? length(s, p) : 0, taken = good ? length(s, c) : 1;
    good = good && taken == 0;
    Fork f{-1, -1, len % page, p, c, len / page};
    if (good && f.entries) f.from = __ldcg(s.page_table + p * s.page_row + f.full);
    const uint32_t free = word_of(run.free);
    if (!(t & 1)) T.free[t >> 1] = free;
    __syncthreads();
    uint32_t at_child = (uint32_t)c * 2654435769u >> 21;           // (Fibonacci hashing: 2^32 over the golden ratio, 11 bits)
    static_assert(2 * PLAN_NT == 1 << 11, "11 bits");
    if (good) {
        for (;; at_child = (at_child + 1) % (2 * PLAN_NT)) {       // (ends: at least half of the places stay free)
            const int there = atomicCAS(child + at_child, -1, c);
            if (there == -1 || there == c) break;
        }
        atomicMin(by + at_child, t);
    }
    __syncthreads();
    good = good && by[at_child] == t;
    const int need = good && f.entries > 0, at = (int)before(need, S), asked = (int)S.total;
    const int found = find_few(s, asked, T, list, S);
    const bool fits = good && (!need || at < found);
    if (mine) {
        status[t] = fits ? 0 : good ? 1 : 2;
        if (fits) {
            s.kv_lens[c] = len;
            if (need) {
                f.to = found_page(s, T, list, at);
                s.page_table[c * s.page_row + f.full] = f.to;
                s.refs[f.to] = 1;
                if (!is_page(s, f.from)) f.to = -1;            // (nothing to copy from)
            }
        } else {
            f.child = -1;
        }
        forks[t] = f;
    }
}

// blockIdx.z: the fork; y: K and V of each layer, and before them the names of the
// shared pages; x: the page's entries, `across` threads (a power of two) to each, four entries a thread at once.
template <class V>
__global__ void __launch_bounds__(256) k_fork_copy(Data D, dbs_page_state s, const Fork *forks, int across)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Fork f = forks[blockIdx.z];
    if (f.child < 0) return;
    const int64_t u0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    if (blockIdx.y == 0) {
        for (int64_t c = u0; c < f.full; c += step) {
            const int p = s.page_table[f.parent * s.page_row + c];
            s.page_table[f.child * s.page_row + c] = p;
            if (is_page(s, p)) atomicAdd(s.refs + p, 1);
        }
        return;
    }
    if (f.to < 0) return;
    const int layer = (int)(blockIdx.y - 1) >> 1, is_v = (int)(blockIdx.y - 1) & 1;
    V *base = (V *)(is_v ? D.v : D.k) + layer * (is_v ? D.v_layer : D.k_layer);
    const int64_t by_page = is_v ? D.v_page : D.k_page, by_entry = is_v ? D.v_entry : D.k_entry, by_head = is_v ? D.v_head : D.k_head;
    const int down = 256 / across, e0 = (int)blockIdx.x * down + (int)threadIdx.x / across, turn = (int)gridDim.x * down;
    const uint32_t per = (uint32_t)(D.heads * D.row), row = (uint32_t)D.row;           // (below 2^31)
    V *const to = base + f.to * by_page;
    const V *const from = base + f.from * by_page;
    for (uint32_t u = threadIdx.x & (across - 1); u < per; u += across) {
        const uint32_t h = D.heads == 1 ? 0u : u / row;
        const int64_t at = h * by_head + (u - h * row);
        for (int64_t e = e0; e < f.entries; e += 4 * (int64_t)turn) {
            V x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (e + k * turn < f.entries) x[k] = from[(e + k * turn) * by_entry + at];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (e + k * turn < f.entries) to[(e + k * turn) * by_entry + at] = x[k];
        }
    }
}

// ---- accepted drafted tokens ----

struct Compact {
    Data d;
    dbs_page_state s;
    const int32_t *tree_lens, *accepted, *accepted_lens;
    int64_t max_accepted, stride;
    int32_t *new_lens;
};

constexpr int MOVE_NT = 256;               // threads of a block, at most: as many as an entry has units

// blockIdx.z: the sequence; y: K or V of a layer; x: units of an entry, one a thread.
// Bound by latency: lengths and lists, page table and entries are three reads in a row (16 layers, 32 sequences of up to
// 48 drafted tokens: 18 MB in 8.2 us).  Numbers ascend, so place i is behind no number that comes later: a thread may load any of its
// units before it stores those of earlier places, in the list's order.
template <class V>
__global__ void __launch_bounds__(MOVE_NT) k_compact(Compact A)
{
    const dbs_page_state &s = A.s;
    __shared__ int64_t from[MOVE_NT], to[MOVE_NT];         // units
    __shared__ int ends;
    const int64_t b = blockIdx.z;
    const int32_t *list = A.accepted + b * A.stride;
    const int NT = (int)blockDim.x;
    // (the list's first numbers are read beside the lengths)
    auto number = [&](int64_t i) { return i >= 0 && i < A.max_accepted ? list[i] : -1; };
    int a = number(threadIdx.x), prior = number((int64_t)threadIdx.x - 1);
    const int layer = (int)blockIdx.y >> 1, is_v = (int)blockIdx.y & 1;
    const Data &D = A.d;
    V *base = (V *)(is_v ? D.v : D.k) + layer * (is_v ? D.v_layer : D.k_layer);
    const int64_t by_page = is_v ? D.v_page : D.k_page, by_entry = is_v ? D.v_entry : D.k_entry, by_head = is_v ? D.v_head : D.k_head;
    const int kv = length(s, b);
    int tree = A.tree_lens[b];
    tree = tree < 0 ? 0 : tree > kv ? kv : tree;
    const int first = kv - tree;
    const int64_t given = A.accepted_lens ? A.accepted_lens[b] : A.max_accepted;
    const int n = (int)(given < 0 ? 0 : given > A.max_accepted ? A.max_accepted : given);
    const uint32_t u = blockIdx.x * NT + threadIdx.x, per = (uint32_t)(D.heads * D.row), row = (uint32_t)D.row;    // (below 2^31)
    const uint32_t h = D.heads == 1 ? 0u : u / row;
    const int64_t mine = h * by_head + (u - h * row);
    int kept = 0;
    // Where entry j lies; -1 if its page is none.
    auto place = [&](int j) -> int64_t {
        int64_t page = b;
        int in = j;
        if (s.page_table) {
            const int size = (int)s.page_size, p = s.page_table[b * s.page_row + j / size];
            if (!is_page(s, p)) return -1;
            page = p;
            in = j % size;
        }
        return page * by_page + in * by_entry;
    };
    for (int64_t i0 = 0; i0 < n; i0 += NT) {
        const int i = (int)i0 + (int)threadIdx.x, most = n - i0 < NT ? (int)(n - i0) : NT;
        if (i0) {
            a = number(i0 + threadIdx.x);
            prior = number(i0 + threadIdx.x - 1);
        }
        if (threadIdx.x == 0) ends = most;
        __syncthreads();
        if (i0 + threadIdx.x < n) {
            // (in a list that ascends up to here a is i at least; behind its end, where anything may stand,
            // the check keeps place i within the tree)
            if (a < i || a >= tree || a <= prior) {
                atomicMin(&ends, (int)threadIdx.x);
            } else {
                // (what comes from no page, or would go to none, stays where it is)
                const int64_t dst = place(first + i);
                from[threadIdx.x] = a == i || dst < 0 ? -1 : place(first + a);
                to[threadIdx.x] = dst;
            }
        }
        __syncthreads();
        const int m = ends;
        if (u < per)
            for (int k0 = 0; k0 < m; k0 += 8) {
                V x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k0 + k < m && from[k0 + k] >= 0) x[k] = base[from[k0 + k] + mine];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k0 + k < m && from[k0 + k] >= 0) base[to[k0 + k] + mine] = x[k];
            }
        kept += m;
        if (m < most) break;
        __syncthreads();                                   // the list has been read
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) A.new_lens[b] = first + kept;
}

// ---- host ----

bool state_ok(const dbs_page_state *s, bool table)
{
    return s && s->batch >= 0 && s->batch < (int64_t(1) << 24) && s->max_pages >= 0 && s->pages >= 0 && s->page_size >= 1 &&
           s->page_size < (int64_t(1) << 31) && s->pages < 0x7fffffff && s->max_pages < (int64_t(1) << 31) &&
           s->pages * s->page_size < (int64_t(1) << 31) && s->max_pages * s->page_size < (int64_t(1) << 31) &&
           (s->batch == 0 || (s->kv_lens && (!table || ((s->page_table || s->max_pages == 0) && (s->batch == 1 || s->page_row >= s->max_pages)))));
}

// Rows as long as they lie together, and the width of a unit: 16 bytes where everything is a
// multiple of that, else an element.
bool data_of(const dbs_cache_data &c, Data &D, int &unit)
{
    const int64_t e = c.element_bytes;
    int64_t k[4] = {c.k_layer, c.k_page, c.k_entry, c.k_head}, v[4] = {c.v_layer, c.v_page, c.v_entry, c.v_head};
    int64_t heads = c.heads, row = c.head_dim;
    if (heads == 1 || (k[3] == row && v[3] == row)) {
        row *= heads;
        heads = 1;
        k[3] = v[3] = 0;
    }
    bool wide = aligned16(c.k) && aligned16(c.v) && row * e % 16 == 0;
    for (int i = 0; i < 4; ++i) wide = wide && k[i] * e % 16 == 0 && v[i] * e % 16 == 0;
    unit = wide ? 16 : (int)e;
    const int64_t by = unit / e;
    D = {(char *)c.k, (char *)c.v, heads, row / by, k[0] / by, k[1] / by, k[2] / by, k[3] / by, v[0] / by, v[1] / by, v[2] / by, v[3] / by};
    return true;
}

// (`same`: K and V may be one tensor)
bool data_ok(const dbs_cache_data *c, const dbs_page_state *s, bool work, bool same)
{
    if (!c || c->layers < 0 || c->layers >= 32768 || c->heads < 0 || c->heads >= (int64_t(1) << 31) || c->head_dim < 0 ||
        c->head_dim >= (int64_t(1) << 31) || c->heads * c->head_dim >= (int64_t(1) << 31) ||
        (c->element_bytes != 1 && c->element_bytes != 2 && c->element_bytes != 4 && c->element_bytes != 8))
        return false;
    if (!work || c->layers == 0 || c->heads == 0 || c->head_dim == 0) return true;
    if (!c->k || !c->v) return false;
    for (int64_t by : {c->k_layer, c->k_page, c->k_entry, c->k_head, c->v_layer, c->v_page, c->v_entry, c->v_head})
        if (by < 0 || by >= int64_t(1) << 50) return false;
    const Places k(c->k, c->element_bytes, c->head_dim, {{c->layers, c->k_layer}, {s->pages, c->k_page}, {s->page_size, c->k_entry}, {c->heads, c->k_head}}),
        v(c->v, c->element_bytes, c->head_dim, {{c->layers, c->v_layer}, {s->pages, c->v_page}, {s->page_size, c->v_entry}, {c->heads, c->v_head}});
    return k.own && v.own && (!k.meets(v) || (same && k.same(v)));
}

// f(V) with V the unit's type.
template <class F> dbs_status by_unit(int unit, F f)
{
    return unit == 16 ? f(uint4{}) : unit == 8 ? f(uint64_t{}) : unit == 4 ? f(uint32_t{}) : unit == 2 ? f(uint16_t{}) : f(uint8_t{});
}

Places ints(const int32_t *p, int64_t n) { return p ? Places(p, 4, n, {}) : Places(); }
Places rows(const int32_t *p, int64_t n, int64_t columns, int64_t stride) { return p ? Places(p, 4, columns, {{n, stride}}) : Places(); }
Places table_of(const dbs_page_state &s) { return rows(s.page_table, s.batch, s.max_pages, s.page_row); }

constexpr int64_t up16(int64_t n) { return (n + 15) & ~int64_t(15); }

// Slots that the one block writes; of more a second launch is through earlier (64, 2048, 8192 and 32,768 slots: 5.8, 6.5, 9.6
// and 18.4 us in the one block, 6.9, 7.2, 8.5 and 9.7 with a second).
constexpr int64_t SLOTS_HERE = 4 * PLAN_NT;

// Scratch of a resize: of few sequences only what does not stay in shared memory.
int64_t scratch_of(const dbs_page_state &s, int64_t columns)
{
    if (s.batch > PLAN_NT) return up16(4 * (3 * s.batch + s.pages));
    return up16(4 * ((s.batch * columns > SLOTS_HERE ? s.batch : 0) + (s.pages > 32 * WORDS ? s.pages : 0)));
}

}  // namespace

extern "C" {

dbs_status dbs_cache_resize_scratch(const dbs_page_state *s, int64_t columns, int64_t *bytes)
{
    if (!bytes || !state_ok(s, false) || columns < 0 || columns >= (int64_t(1) << 31)) return DBS_ERR_INVALID_ARG;
    *bytes = scratch_of(*s, columns);
    return DBS_OK;
}

dbs_status dbs_cache_resize(const dbs_page_state *s, const int32_t *lens, int32_t *status, int32_t *slots, int64_t columns, void *scratch,
                            int64_t scratch_bytes, void *stream)
{
    if (!state_ok(s, true) || columns < 0 || columns >= (int64_t(1) << 31)) return DBS_ERR_INVALID_ARG;
    if (s->batch == 0) return DBS_OK;
    const int64_t need = scratch_of(*s, columns), all = slots ? s->batch * columns : 0;
    if (!lens || !status || (s->pages > 0 && !s->refs) || (need > 0 && (!scratch || !aligned16(scratch) || scratch_bytes < need)))
        return DBS_ERR_INVALID_ARG;
    const Places writes[5] = {ints(status, s->batch), ints(slots, all), ints(s->kv_lens, s->batch), ints(s->refs, s->pages), table_of(*s)}, want = ints(lens, s->batch);
    if (clash(writes, 5, &want, 1, false)) return DBS_ERR_INVALID_ARG;
    const bool here = all > 0 && all <= SLOTS_HERE;
    int32_t *at = (int32_t *)scratch;
    cudaStream_t st = (cudaStream_t)stream;
    Resize A{*s, lens, status, all ? slots : nullptr, columns, nullptr, nullptr, nullptr, at};
    if (s->batch <= PLAN_NT) {
        if (s->batch * columns > SLOTS_HERE) {
            A.old = at;
            A.list = at + s->batch;
        }
        k_resize_few<<<1, PLAN_NT, 0, st>>>(A, here);
    } else {
        A.old = at;
        A.need = at + s->batch;
        A.end = at + 2 * s->batch;
        A.list = at + 3 * s->batch;
        k_resize<<<1, PLAN_NT, 0, st>>>(A, here);
    }
    if (all > 0 && !here) {
        const int64_t blocks = (all + 255) / 256;
        k_slots<<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, st>>>(A);
    }
    return launched();
}

dbs_status dbs_cache_fork_scratch(const dbs_page_state *s, int64_t n, int64_t *bytes)
{
    if (!bytes || !state_ok(s, false) || n < 0 || n >= 65536) return DBS_ERR_INVALID_ARG;
    *bytes = up16(n * (int64_t)(sizeof(Fork) + 4));
    return DBS_OK;
}

dbs_status dbs_cache_fork(const dbs_cache_data *data, const dbs_page_state *s, const int32_t *parents, const int32_t *children, int64_t n,
                          int32_t *status, void *scratch, int64_t scratch_bytes, void *stream)
{
    if (!state_ok(s, true) || n < 0 || n >= 65536 || !data_ok(data, s, n > 0, true)) return DBS_ERR_INVALID_ARG;
    if (n == 0) return DBS_OK;
    int64_t need = 0;
    if (dbs_cache_fork_scratch(s, n, &need) != DBS_OK || !parents || !children || !status || (s->pages > 0 && !s->refs) || !scratch ||
        !aligned16(scratch) || scratch_bytes < need)
        return DBS_ERR_INVALID_ARG;
    const Places writes[4] = {ints(status, n), ints(s->kv_lens, s->batch), ints(s->refs, s->pages), table_of(*s)}, reads[2] = {ints(parents, n), ints(children, n)};
    if (clash(writes, 4, reads, 2, false)) return DBS_ERR_INVALID_ARG;
    Fork *forks = (Fork *)scratch;
    int32_t *list = (int32_t *)(forks + n);
    cudaStream_t st = (cudaStream_t)stream;
    if (n <= PLAN_NT) k_fork_plan_few<<<1, PLAN_NT, 0, st>>>(*s, parents, children, (int)n, status, forks, list);
    else k_fork_plan<<<1, PLAN_NT, 0, st>>>(*s, parents, children, (int)n, status, forks, list);
    dbs_status got = launched();
    if (got != DBS_OK || s->batch == 0) return got;
    Data D{};
    int unit = 16;
    const bool any = data->layers > 0 && data->heads > 0 && data->head_dim > 0;
    if (any) data_of(*data, D, unit);
    int across = 256;
    while (across > 1 && any && across / 2 >= D.heads * D.row) across /= 2;
    const int64_t each = 4 * (256 / across), blocks = (s->page_size + each - 1) / each;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(blocks < 256 ? blocks : 256), any ? (unsigned)(1 + 2 * data->layers) : 1u, (unsigned)n);
    c.blockDim = 256;
    c.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    return by_unit(unit, [&](auto v) {
        return cudaLaunchKernelEx(&c, k_fork_copy<decltype(v)>, D, *s, (const Fork *)forks, across) == cudaSuccess ? DBS_OK
                                                                                                                   : (cudaGetLastError(), DBS_ERR_CUDA);
    });
}

dbs_status dbs_cache_compact(const dbs_cache_data *data, const dbs_page_state *s, const int32_t *tree_lens, const int32_t *accepted,
                             int64_t max_accepted, int64_t accepted_stride, const int32_t *accepted_lens, int32_t *new_lens, void *stream)
{
    if (!state_ok(s, s && s->page_table) || s->batch >= 65536 || max_accepted < 0 || max_accepted >= (int64_t(1) << 31) ||
        !data_ok(data, s, s->batch > 0, false))
        return DBS_ERR_INVALID_ARG;
    if (s->batch == 0) return DBS_OK;
    if (!tree_lens || !new_lens || (max_accepted > 0 && (!accepted || accepted_stride < 0)) ||
        (!s->page_table && (s->max_pages > 1 || s->pages < s->batch)) || (s->max_pages > 0 && s->pages < 1))
        return DBS_ERR_INVALID_ARG;
    const Places writes = ints(new_lens, s->batch), reads[5] = {ints(s->kv_lens, s->batch), ints(tree_lens, s->batch), ints(accepted_lens, s->batch),
                                                                rows(accepted, s->batch, max_accepted, accepted_stride), table_of(*s)};
    if (clash(&writes, 1, reads, 5, false)) return DBS_ERR_INVALID_ARG;
    Compact A{{}, *s, tree_lens, accepted, accepted_lens, max_accepted, accepted_stride, new_lens};
    int unit = 16;
    const bool any = data->layers > 0 && data->heads > 0 && data->head_dim > 0;
    if (any) data_of(*data, A.d, unit);
    else A.d.row = 1;
    const int64_t per = any ? A.d.heads * A.d.row : 1;
    const int nt = per >= MOVE_NT ? MOVE_NT : (int)((per + 31) / 32 * 32);
    const dim3 grid((unsigned)((per + nt - 1) / nt), any ? (unsigned)(2 * data->layers) : 1u, (unsigned)s->batch);
    return by_unit(unit, [&](auto v) {
        k_compact<decltype(v)><<<grid, nt, 0, (cudaStream_t)stream>>>(A);
        return launched();
    });
}

}  // extern "C"
