// Device helpers of the training-step operators: element formats, vector
// accesses at element alignment, and wave and block reductions.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace dion {

// Element types as stored.  Conversions from fp32 round to nearest even (the
// compiler's casts: one v_cvt instruction each on gfx950).
typedef __bf16 bf16_t;
typedef _Float16 fp16_t;

template <typename T> __device__ __forceinline__ float to_f(T v) { return (float)v; }
template <typename T> __device__ __forceinline__ T from_f(float v) { return (T)v; }

__device__ __forceinline__ float load_fmt(const void* p, int64_t i, int fmt) {
  if (fmt == 1) return ((const float*)p)[i];
  if (fmt == 0) return (float)((const bf16_t*)p)[i];
  return (float)((const fp16_t*)p)[i];
}
__device__ __forceinline__ void store_fmt(void* p, int64_t i, int fmt, float v) {
  if (fmt == 1) ((float*)p)[i] = v;
  else if (fmt == 0) ((bf16_t*)p)[i] = (bf16_t)v;
  else ((fp16_t*)p)[i] = (fp16_t)v;
}

// Largest that keeps a NaN: fmaxf would drop it, and a row that holds one
// must say so.
__device__ __forceinline__ float max_nan(float a, float b) {
  return a != a ? a : (b != b ? b : fmaxf(a, b));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max_nan(v, __shfl_xor(v, o, 64));
  return v;
}

// Sum or largest value over a block of THREADS threads, the same in every
// thread; `red` holds THREADS / 64 floats and is free for reuse afterwards.
template <int THREADS> __device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) v += red[i];
  __syncthreads();
  return v;
}
template <int THREADS> __device__ __forceinline__ float block_max(float v, float* red) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < THREADS / 64; ++i) v = max_nan(v, red[i]);
  __syncthreads();
  return v;
}

}  // namespace dion
