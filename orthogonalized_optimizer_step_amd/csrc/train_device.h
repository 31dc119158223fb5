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

// v moved across lanes (a data-parallel primitive of the VALU: no LDS round
// trip), `none` where nothing comes in
template <int CTRL, int ROWS> __device__ __forceinline__ float lane_move(float none, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(v), CTRL, ROWS, 0xf, false));
}

// op over the 64 lanes of a wave, the same in every lane: within rows of 16
// lanes (shifts by 1, 2, 4 and 8), then the rows' last lanes into the next.
template <typename Op> __device__ __forceinline__ float wave_reduce(float v, float none, Op op) {
  v = op(v, lane_move<0x111, 0xf>(none, v));
  v = op(v, lane_move<0x112, 0xf>(none, v));
  v = op(v, lane_move<0x114, 0xf>(none, v));
  v = op(v, lane_move<0x118, 0xf>(none, v));
  v = op(v, lane_move<0x142, 0xa>(none, v));
  v = op(v, lane_move<0x143, 0xc>(none, v));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// the same over the W <= 16 values that lane l < W holds
template <int W, typename Op> __device__ __forceinline__ float row_reduce(float v, float none, Op op) {
  v = op(v, lane_move<0x111, 0xf>(none, v));
  if (W > 2) v = op(v, lane_move<0x112, 0xf>(none, v));
  if (W > 4) v = op(v, lane_move<0x114, 0xf>(none, v));
  if (W > 8) v = op(v, lane_move<0x118, 0xf>(none, v));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), W - 1));
}

// op over each row of 16 lanes by itself, the same in all of them
template <typename Op> __device__ __forceinline__ float row16_reduce(float v, Op op) {
  v = op(v, lane_move<0x128, 0xf>(v, v));   // rotated by 8, 4, 2, 1
  v = op(v, lane_move<0x124, 0xf>(v, v));
  v = op(v, lane_move<0x122, 0xf>(v, v));
  return op(v, lane_move<0x121, 0xf>(v, v));
}

// and over two such rows, which ds_swizzle exchanges (lane xor 16)
template <typename Op> __device__ __forceinline__ float pair_reduce(float v, Op op) {
  return op(v, __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401f)));
}

struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct MaxNan {
  __device__ __forceinline__ float operator()(float a, float b) const { return max_nan(a, b); }
};
// Largest of magnitudes: as unsigned integers they are in order, with NaN above all.
struct MaxAbs {
  __device__ __forceinline__ float operator()(float a, float b) const {
    return __uint_as_float(max(__float_as_uint(a) & 0x7fffffffu, __float_as_uint(b) & 0x7fffffffu));
  }
};

__device__ __forceinline__ float wave_sum(float v) { return wave_reduce(v, 0.f, Add()); }
__device__ __forceinline__ float wave_max(float v) { return wave_reduce(v, -__builtin_inff(), MaxNan()); }

// op over a block of THREADS threads, the same in every thread.  `red` holds
// THREADS / 64 floats; it may be written again once every thread has passed
// another barrier.
template <int THREADS, typename Op> __device__ __forceinline__ float block_reduce(float v, float none, float* red, Op op) {
  constexpr int W = THREADS / 64;
  static_assert(W >= 2 && W <= 16, "a row of lanes holds the waves' values");
  v = wave_reduce(v, none, op);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  lds_barrier();
  const int lane = threadIdx.x & 63;
  return row_reduce<W>(lane < W ? red[lane] : none, none, op);
}

}  // namespace dion
