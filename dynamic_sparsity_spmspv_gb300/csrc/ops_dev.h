// Device helpers shared by the decoding-step operators (w4.cu, rotary.cu,
// attention.cu, logits.cu).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/dbspmspv.h"

namespace dbs::ops {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// The one rounding of a result to its type.
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two 16-bit values of a word (or one fp32) to fp32, values 2i and 2i + 1 (or
// i) of an array, and back, rounded once.
template <class T, int N> __device__ __forceinline__ void open2(uint32_t w, float (&v)[N], int i)
{
    if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w);
    } else if constexpr (__is_same(T, __nv_bfloat16)) {
        v[2 * i] = __uint_as_float(w << 16);
        v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <class T> __device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (__is_same(T, __nv_bfloat16)) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
template <class T, int N> __device__ __forceinline__ uint32_t shut2(const float (&v)[N], int i)
{
    if constexpr (sizeof(T) == 4) return __float_as_uint(v[i]);
    else return pack2<T>(v[2 * i], v[2 * i + 1]);
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// ---- barriers in shared memory ----

// Waits on these barriers end: after `limit` they give up, and so does the block
// (cluster barriers and the allocation of tensor memory have no limit: they wait for
// blocks that end by themselves).  A test can make waits of one block, or of all,
// run out (dbs_debug_operator_waits): its copies are announced as `VAIN` bytes
// longer than they are.
struct Waits {
    uint32_t limit;            // ns
    int vain;                  // that block; -1: none; -2: all
};
constexpr uint32_t VAIN = 16;
inline std::atomic<uint32_t> wait_limit{2000000000};
inline std::atomic<int32_t> wait_vain{-1};
inline Waits waits() { return {wait_limit.load(std::memory_order_relaxed), wait_vain.load(std::memory_order_relaxed)}; }
__device__ __forceinline__ uint32_t vain_bytes(const Waits &w) { return w.vain == -2 || w.vain == (int)blockIdx.x ? VAIN : 0u; }

__device__ __forceinline__ void bar_init(uint32_t bar, int count) { asm volatile("mbarrier.init.shared.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory"); }
__device__ __forceinline__ void bar_arrive(uint32_t bar) { asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(bar) : "memory"); }
// Waits for the phase of that parity to end; false when the limit ran out, here or in another warp.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *stop, uint32_t limit)
{
    uint32_t began = 0;
    for (int i = 0;; ++i) {
        uint32_t done;
        asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
        if ((i & 31) != 31) continue;
        if (*stop) return false;
        uint32_t now;                                    // (the lower word: 4 s)
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
        now |= 1;
        if (began == 0) began = now;
        else if (now - began > limit) break;
    }
    *stop = 1;
    return false;
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// One lane of a warp, in a way that the compiler knows to be one.
__device__ __forceinline__ bool elected()
{
    uint32_t e;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(e));
    return e != 0;
}

// Tensor maps for tiled copies, made by the driver (whose entry point is looked
// up until it is found; no library is linked for it).
typedef CUresult (*encode_tiled_fn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                    const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                    CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline encode_tiled_fn encode_tiled()
{
    static std::atomic<encode_tiled_fn> found{nullptr};
    if (const encode_tiled_fn fn = found.load(std::memory_order_relaxed)) return fn;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    found.store((encode_tiled_fn)p, std::memory_order_relaxed);
    return (encode_tiled_fn)p;
}

inline bool dtype_ok(int32_t d) { return d == DBS_F32 || d == DBS_F16 || d == DBS_BF16; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Multiprocessors of the current device; 0 if there is none.
inline int multiprocessors()
{
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}
// Room for a kernel's dynamic shared memory, and leave for clusters of more than eight
// blocks, asked for once on a device (noted when it is there, so that another thread's
// launch never comes before it; a failure is not kept).  `registers`, if not 0: what the
// kernel's threads have to start with, as its warps share them out (a share above that
// would be waited for without end).
using Once = std::atomic<uint64_t>;
template <class K> inline bool room_for(Once &once, K kernel, int bytes, bool large_clusters = false, int registers = 0)
{
    int dev = 0;
    const bool known = cudaGetDevice(&dev) == cudaSuccess && dev < 64;
    const uint64_t bit = uint64_t(known) << (dev & 63);
    if (once.load(std::memory_order_acquire) & bit) return true;
    cudaFuncAttributes has{};
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
        (large_clusters && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) ||
        (registers && cudaFuncGetAttributes(&has, kernel) != cudaSuccess)) {
        cudaGetLastError();
        return false;
    }
    if (registers && has.numRegs != registers) return false;
    once.fetch_or(bit, std::memory_order_release);
    return true;
}

// Status of the launches since the last check.
inline dbs_status launched() { return cudaGetLastError() == cudaSuccess ? DBS_OK : DBS_ERR_CUDA; }

}  // namespace dbs::ops
