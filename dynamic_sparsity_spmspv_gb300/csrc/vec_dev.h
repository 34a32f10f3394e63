// Vectors of a head's values (rotary.cu, norm.cu): what one thread moves at once.
#pragma once
#include "ops_dev.h"

namespace dbs::ops {

// What a thread moves of a head at once: 16 bytes, or one value where rows are
// not aligned for that.
template <class T, bool WIDE> struct Vec {
    static constexpr int n = WIDE ? 16 / (int)sizeof(T) : 1;
    using type = uint4;
};
template <> struct Vec<float, false> {
    static constexpr int n = 1;
    using type = uint32_t;
};
template <> struct Vec<__half, false> {
    static constexpr int n = 1;
    using type = uint16_t;
};
template <> struct Vec<__nv_bfloat16, false> {
    static constexpr int n = 1;
    using type = uint16_t;
};

// The values of a vector in fp32, and back with their one rounding.
template <class T> __device__ __forceinline__ void open(const uint4 &w, float (&v)[16 / sizeof(T)])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) open2<T>(u[i], v, i);
}
template <class T> __device__ __forceinline__ uint4 shut(const float (&v)[16 / sizeof(T)])
{
    return make_uint4(shut2<T>(v, 0), shut2<T>(v, 1), shut2<T>(v, 2), shut2<T>(v, 3));
}
template <class T> __device__ __forceinline__ void open(uint16_t w, float (&v)[1]) { v[0] = to_f32(*reinterpret_cast<const T *>(&w)); }
template <class T> __device__ __forceinline__ void open(uint32_t w, float (&v)[1]) { v[0] = __uint_as_float(w); }
template <class T> __device__ __forceinline__ void shut(const float (&v)[1], uint16_t &w)
{
    const T t = from_f32<T>(v[0]);
    w = *reinterpret_cast<const uint16_t *>(&t);
}
template <class T> __device__ __forceinline__ void shut(const float (&v)[1], uint32_t &w) { w = __float_as_uint(v[0]); }
template <class T, int N> __device__ __forceinline__ void shut(const float (&v)[N], uint4 &w) { w = shut<T>(v); }

}  // namespace dbs::ops
