// Device helpers shared by the decoding-step operators (w4.cu, rotary.cu,
// attention.cu, logits.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

inline int dtype_size(int32_t d) { return d == DBS_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t d) { return d == DBS_F32 || d == DBS_F16 || d == DBS_BF16; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Status of the launches since the last check.
inline dbs_status launched() { return cudaGetLastError() == cudaSuccess ? DBS_OK : DBS_ERR_CUDA; }

}  // namespace dbs::ops
