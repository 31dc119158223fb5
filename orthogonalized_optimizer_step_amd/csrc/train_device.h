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

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));
// 16 bytes at the alignment of 16-bit elements (global memory takes them so)
typedef uintx4 uintx4u __attribute__((aligned(2)));

__device__ __forceinline__ float max3(float a, float b, float c) {   // drops NaN, which sums keep
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// A barrier for LDS alone: loads and stores of global memory stay in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory"); }

// 16 bytes of a row
template <typename Z> struct Chunk {
  static constexpr int N = 16 / (int)sizeof(Z);
  static __device__ __forceinline__ void unpack(const uintx4& v, float* f) {
    union { uintx4 u; Z z[N]; } c;
    c.u = v;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = (float)c.z[i];
  }
  static __device__ __forceinline__ uintx4 pack(const float* f) {
    union { uintx4 u; Z z[N]; } c;
#pragma unroll
    for (int i = 0; i < N; ++i) c.z[i] = (Z)f[i];
    return c.u;
  }
  // m, or the largest of the values where that is more
  static __device__ __forceinline__ float largest(float m, const uintx4& v) {
    float f[N];
    unpack(v, f);
#pragma unroll
    for (int i = 0; i < N; i += 2) m = max3(m, f[i], f[i + 1]);
    return m;
  }
  // elements [j, j + N) of a row of n, `fill` past its end
  static __device__ __forceinline__ uintx4 load(const Z* row, int j, int n, float fill) {
    if (j + N <= n) return *(const uintx4u*)(row + j);
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = j + i < n ? (float)row[j + i] : fill;
    return pack(f);
  }
  template <bool PAST_CACHES> static __device__ __forceinline__ void put(Z* row, int j, int n, const float* f) {
    if (j + N <= n) {
      if (PAST_CACHES) __builtin_nontemporal_store(pack(f), (uintx4u*)(row + j));
      else *(uintx4u*)(row + j) = pack(f);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (j + i < n) row[j + i] = (Z)f[i];
    }
  }
  // results larger than the caches, and results that the next operator reads
  static __device__ __forceinline__ void store(Z* row, int j, int n, const float* f) { put<true>(row, j, n, f); }
  static __device__ __forceinline__ void store_near(Z* row, int j, int n, const float* f) { put<false>(row, j, n, f); }
};

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
