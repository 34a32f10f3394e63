// What tensors take of memory, for the checks of arguments (host).
#pragma once
#include <stdint.h>

#include <initializer_list>

namespace dbs::ops {

// A strided tensor: runs of contiguous elements, in each of up to four dimensions
// `count` of them, `step` bytes apart.  Dimensions of one run are left out, the others
// lie by ascending steps.  (Wide numbers: a product of any two sizes fits.)
struct Places {
    using Big = __int128;
    struct Dim {
        int64_t count, stride;     // in elements, 0 or more
    };
    uintptr_t at;
    Big run, count[4], step[4];
    int n = 0;
    bool none;                     // no run at all

    Places(const void *p, int64_t element, int64_t run_elements, std::initializer_list<Dim> dims)
        : at(reinterpret_cast<uintptr_t>(p)), run((Big)element * run_elements), none(run_elements <= 0)
    {
        for (const Dim &d : dims) {
            none = none || d.count <= 0;
            if (d.count <= 1) continue;
            const Big s = (Big)element * d.stride;
            int i = n++;
            for (; i > 0 && step[i - 1] > s; --i) {
                step[i] = step[i - 1];
                count[i] = count[i - 1];
            }
            step[i] = s;
            count[i] = d.count;
        }
    }
    // Whether every run has a place of its own: each dimension steps over all that the finer ones
    // take.  (Dimensions permuted or cut out of a contiguous tensor do; strides whose runs lie
    // apart without that are not known as such.)
    bool own() const
    {
        Big extent = run;
        for (int i = 0; !none && i < n; ++i) {
            if (step[i] < extent) return false;
            extent += (count[i] - 1) * step[i];
        }
        return true;
    }
};

}  // namespace dbs::ops
