// What tensors take of memory, for the checks of arguments (host).
#pragma once
#include <stdint.h>

#include <initializer_list>

namespace dbs::ops {

// A strided tensor: runs of contiguous elements, in each of up to four dimensions
// `count` of them, `step` bytes apart.  Dimensions of one run are left out, the others
// lie by ascending steps.  (In bytes; what no memory holds counts as MOST.)
struct Places {
    static constexpr int64_t MOST = int64_t(1) << 58;      // (sums of a few of it fit)
    struct Dim {
        int64_t count, stride;     // in elements, 0 or more
    };
    uintptr_t at;
    int64_t run, extent;           // bytes of a run, and from the first one's begin to the last one's end
    int64_t count[4], step[4];
    int n = 0;
    bool none = true;              // no run at all
    // Whether every run has a place of its own: each dimension steps over all that the finer ones
    // take.  (Dimensions permuted or cut out of a contiguous tensor do; strides whose runs lie
    // apart without that are not known as such.)
    bool own = true;

    Places() : at(0), run(0), extent(0) {}
    Places(const void *p, int64_t element, int64_t run_elements, std::initializer_list<Dim> dims)
        : at(reinterpret_cast<uintptr_t>(p)), run(product(element, run_elements)), extent(run), none(run_elements <= 0)
    {
        for (const Dim &d : dims) {
            none = none || d.count <= 0;
            if (d.count <= 1) continue;
            const int64_t s = product(element, d.stride);
            int i = n++;
            for (; i > 0 && step[i - 1] > s; --i) {
                step[i] = step[i - 1];
                count[i] = count[i - 1];
            }
            step[i] = s;
            count[i] = d.count;
        }
        for (int i = 0; i < n; ++i) {
            own = own && (none || step[i] >= extent);
            extent = capped(product(count[i] - 1, step[i]) + extent);
        }
    }
    bool dense() const
    {
        int64_t all = run;
        for (int i = 0; i < n; ++i) all = product(all, count[i]);
        return own && all == extent && extent < MOST;
    }
    bool same(const Places &o) const
    {
        bool is = at == o.at && run == o.run && n == o.n;
        for (int i = 0; is && i < n; ++i) is = count[i] == o.count[i] && step[i] == o.step[i];
        return is;
    }
    // Whether some byte is surely in both: both are without gaps and their spans meet, or two runs are
    // found that do (always, if there are any, where each larger step of the two goes over what the
    // smaller ones take: tensors of one layout cut out of one buffer; else among a thousand tries).
    bool meets(const Places &o) const
    {
        if (none || o.none) return false;
        const int64_t gap = (int64_t)(o.at - at);          // (addresses are below 2^62)
        if (gap >= extent || -gap >= o.extent) return false;
        if ((gap < run && -gap < o.run) || (dense() && o.dense())) return true;        // (the first runs meet)
        if (extent >= MOST || o.extent >= MOST) return false;
        // Run y of `o` begins gap + sum y step' - sum x step behind run x of this: from -o.run + 1 to run - 1
        // they meet.  By steps, with the differences of index that there are of each:
        int64_t by[8], lo[8], hi[8];
        int k = 0;
        for (int i = 0, j = 0; i < n || j < o.n;) {
            const int64_t s = j == o.n || (i < n && step[i] < o.step[j]) ? step[i] : o.step[j];
            by[k] = s;
            lo[k] = hi[k] = 0;
            for (; i < n && step[i] == s; ++i) lo[k] -= count[i] - 1;
            for (; j < o.n && o.step[j] == s; ++j) hi[k] += o.count[j] - 1;
            k += s > 0;
        }
        int tries = 1000;
        return found(gap, by, lo, hi, k, o.run, tries);
    }

private:
    static int64_t capped(int64_t v) { return v < MOST ? v : MOST; }
    static int64_t product(int64_t a, int64_t b)
    {
        int64_t v;
        return __builtin_mul_overflow(a, b, &v) ? MOST : capped(v);
    }
    bool found(int64_t gap, const int64_t *by, const int64_t *lo, const int64_t *hi, int k, int64_t other, int &tries) const
    {
        if (--tries < 0) return false;
        if (k == 0) return gap > -other && gap < run;
        // what is left of the gap has to be within reach of the smaller steps
        int64_t down = other, up = run;
        for (int i = 0; i < k - 1; ++i) {
            down += hi[i] * by[i];
            up -= lo[i] * by[i];
        }
        const int64_t s = by[k - 1];
        auto floor_of = [&](int64_t v) { return v >= 0 ? v / s : -((-v + s - 1) / s); };
        int64_t first = -floor_of(down + gap), last = floor_of(up - gap);
        if (first < lo[k - 1]) first = lo[k - 1];
        if (last > hi[k - 1]) last = hi[k - 1];
        for (int64_t x = first; x <= last && tries > 0; ++x)
            if (found(gap + x * s, by, lo, hi, k - 1, other, tries)) return true;
        return false;
    }
};

// Whether one of `writes` shares memory with another or with one of `reads`; in place: but the i-th
// output may be the very same as the i-th input (each place is read before it is written, by the same threads).
inline bool clash(const Places *writes, int n_writes, const Places *reads, int n_reads, bool in_place)
{
    for (int i = 0; i < n_writes; ++i) {
        for (int j = 0; j < i; ++j)
            if (writes[i].meets(writes[j])) return true;
        for (int j = 0; j < n_reads; ++j)
            if (writes[i].meets(reads[j]) && !(in_place && i == j && writes[i].same(reads[j]))) return true;
    }
    return false;
}

}  // namespace dbs::ops
