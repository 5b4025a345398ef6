// Element types of the calls whose tensors are fp32, bf16 or fp16: loads to
// and stores from fp32, one element at a time or a 16-byte vector of eight.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// An element of an array whose type is known only at run time.
__device__ __forceinline__ float load_any(const void* p, int dtype, long long i) {
  if (dtype == MOE_DT_F32) return reinterpret_cast<const float*>(p)[i];
  if (dtype == MOE_DT_BF16) return to_f32(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(reinterpret_cast<const __half*>(p)[i]);
}

// SM count of the current device (asked for once per device).
inline int device_sms() {
  static int known[64];   // 0: not asked yet; threads that ask at once store the same value
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && (n = __atomic_load_n(&known[dev], __ATOMIC_RELAXED)) > 0) return n;
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (n < 1) n = 1;
  if (dev >= 0 && dev < 64) __atomic_store_n(&known[dev], n, __ATOMIC_RELAXED);
  return n;
}

// Raises a kernel's dynamic shared memory limit, once per device: `done` is the
// kernel's own array of flags.
template <typename K>
inline cudaError_t allow_smem(K kernel, size_t bytes, char (&done)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && __atomic_load_n(&done[dev], __ATOMIC_RELAXED)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) cudaGetLastError();   // reported here, not by the next launch's check
  if (e == cudaSuccess && dev >= 0 && dev < 64) __atomic_store_n(&done[dev], (char)1, __ATOMIC_RELAXED);
  return e;
}

inline bool known_dtype(int d) { return d == MOE_DT_F32 || d == MOE_DT_BF16 || d == MOE_DT_F16; }
inline size_t dtype_size(int d) { return d == MOE_DT_F32 ? 4 : 2; }

}  // namespace moe
